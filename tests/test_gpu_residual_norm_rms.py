"""residual_norm's gradient with both norms RMS, where one round of sums serves
both gradients: every pair of types, rows side by side, rows shared by several
warps and rows above 4,096 channels."""
import pytest
import torch

import test_gpu_residual_norm as T

BF, F32 = torch.bfloat16, torch.float32
ALL = "y gate scale shift weight bias y_weight"

# rows, channels, rows per group, stream, branch, params, norm, y_norm, parts given
RMS = {
    "rms_frames": (103, 1280, 25, BF, BF, F32, 2, 2, ALL),
    "rms_float_stream": (65, 1000, 13, F32, BF, BF, 2, 2, ALL),
    "rms_all_float": (50, 520, 50, F32, F32, F32, 2, 2, ALL),
    "rms_four_rows_side_by_side": (61, 136, 9, BF, BF, F32, 2, 2, ALL),
    "rms_two_rows_side_by_side": (61, 264, 20, F32, BF, F32, 2, 2, ALL),
    "rms_smallest_row": (300, 8, 100, F32, F32, F32, 2, 2, "y gate scale"),
    "rms_group_a_row": (23, 72, 1, BF, BF, BF, 2, 2, "y gate scale shift"),
    "rms_long_row": (9, 5000, 4, BF, BF, F32, 2, 2, ALL),
    "rms_long_float_stream": (7, 4104, 7, F32, BF, F32, 2, 2, ALL),
    "rms_longest_float": (5, 8192, 2, F32, F32, F32, 2, 2, ALL),
    "rms_plain": (33, 640, 33, BF, BF, F32, 2, 2, "y"),
    "rms_one_row": (1, 1280, 1, BF, BF, BF, 2, 2, ALL),
}
T.CASES.update(RMS)  # Case looks them up by name; the tests there keep their own list


@pytest.mark.gpu
@pytest.mark.parametrize("name", RMS)
def test_forward(bss, name):
    T.test_forward(bss, name)


@pytest.mark.gpu
@pytest.mark.parametrize("name", RMS)
def test_backward(bss, name):
    T.test_backward(bss, name)


@pytest.mark.gpu
@pytest.mark.parametrize("name", ["rms_frames", "rms_float_stream", "rms_long_row"])
def test_one_side_strided_and_in_place(bss, name):
    T.test_backward_of_one_side(bss, name)
    T.test_strided_and_in_place(bss, name)

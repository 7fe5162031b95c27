"""The host side of the operators around the attention step, by a host program
that compiles it alone (``host_checks.cpp``), and through the C ABI on the CPU."""
import os
import subprocess

import pytest

import block_sparse_spatio_gb300 as bss
from block_sparse_spatio_gb300 import build as nb
from test_block_args import INVALID, backward, forward, norm_args, ptr, rotary, tokens

HERE = os.path.dirname(os.path.abspath(__file__))
NO_DEVICE = 3  # BSS_ERR_CUDA: every check passed, there is nothing to launch on


@pytest.fixture(scope="module")
def lib():
    nb.build()
    return bss.load()


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    out = str(tmp_path_factory.mktemp("host") / "host_checks")
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nb.nvcc()))), "include")
    for name in (cuda, "/usr/local/cuda/include"):
        if os.path.exists(os.path.join(name, "cuda_runtime_api.h")):
            cuda = name
    res = subprocess.run(["g++", "-std=c++17", "-O1", "-pthread", "-I", nb.INCLUDE, "-I", nb.CSRC, "-I", cuda,
                          os.path.join(HERE, "host_checks.cpp"), "-o", out], capture_output=True, text=True)
    assert res.returncode == 0, res.stderr[-2000:]
    return out


def run(program, what):
    res = subprocess.run([program, what], capture_output=True, text=True, timeout=300)
    assert res.returncode == 0, res.stdout[-1000:]


def test_overlap_of_strided_tensors(program):
    run(program, "regions")


def test_limits_of_many_launch_sizes(program):
    """More sizes than the library keeps, also from several threads."""
    run(program, "limits")


@pytest.fixture
def no_gpu():
    """Calls that pass every check on made-up addresses: only where nothing can be launched."""
    import torch
    if torch.cuda.is_available():
        pytest.skip("made-up addresses, never on a machine with a GPU")


@pytest.mark.parametrize("H,d", [(1, 128), (2, 128), (10, 64)])
def test_gradients_packed_head_by_head(lib, no_gpu, H, d):
    """dq, dk and dv as views of one [N][H][3][d] or [H][N][3][d] tensor share no byte."""
    p = bss.MaskParams(3, 4, 5, d, 1, 1)
    for ts, hs in ((3 * H * d, 3 * d), (3 * d, p.N * 3 * d), (3 * H * d + 8, 3 * d)):
        views = [tokens(0, data=(1 << 32) + 2 * i * d, token_stride=ts, head_stride=hs) for i in range(3)]
        assert backward(lib, H=H, params=p, outs=views) == NO_DEVICE
        views[1] = tokens(0, data=(1 << 32) + 2 * d - 16, token_stride=ts, head_stride=hs)  # 8 channels into dq
        assert backward(lib, H=H, params=p, outs=views) == INVALID


# Outputs written over their input, with a parameter at the same address: rows would
# read modulations that other rows have overwritten.  bf16 parameters, 64 channels.
OVER_FORWARD = [dict(r=ptr(0), **{k: ptr(0), k + "_stride": 64}) for k in ("gate", "scale", "shift")] + [
    dict(h=ptr(1), **{k: ptr(1), k + "_stride": 64}) for k in ("gate", "scale", "shift")] + [
    dict(r=ptr(0), scale=ptr(0), scale_stride=64, rows_per_group=1), dict(r=ptr(0), weight=ptr(0), rows=1),
    dict(h=ptr(1), y_weight=ptr(1), rows=1), dict(h=ptr(1), bias=ptr(1), rows=1),
    dict(r=ptr(0), h=None, gate=ptr(0), gate_stride=64)]
OVER_BACKWARD = [dict(dx=ptr(2), **{k: ptr(2), k + "_stride": 64}) for k in ("gate", "scale")] + [
    dict(dy=ptr(3), **{k: ptr(3), k + "_stride": 64}) for k in ("gate", "scale")] + [
    dict(dx=ptr(2), weight=ptr(2), rows=1), dict(dy=ptr(3), y_weight=ptr(3), rows=1),
    dict(dx=ptr(2), scale=ptr(2), scale_stride=64, rows_per_group=1), dict(dx=ptr(2), stats=ptr(2)),
    dict(dx=ptr(3), dr=None), dict(dy=ptr(2), dx=ptr(5))]


@pytest.mark.parametrize("kw", OVER_FORWARD)
def test_norm_in_place_refuses_parameters_there(lib, no_gpu, kw):
    assert lib.bss_residual_norm(norm_args(bss._ResidualNormArgs, param_dtype=0, **kw), None) == INVALID


@pytest.mark.parametrize("kw", OVER_BACKWARD)
def test_norm_backward_in_place_refuses_parameters_there(lib, no_gpu, kw):
    assert lib.bss_residual_norm_backward(norm_args(bss._ResidualNormGrads, param_dtype=0, **kw), None) == INVALID


def test_norm_in_place_still_taken(lib, no_gpu):
    """Over the paired input, also where another row input is that same tensor."""
    for kw in (dict(r=ptr(0)), dict(h=ptr(1)), dict(r=ptr(0), h=ptr(1)), dict(y=ptr(0), r=ptr(0)),
               dict(y=ptr(0), h=ptr(0)), dict(r=ptr(0), rows=1, x_stride=8, r_stride=24)):
        assert lib.bss_residual_norm(norm_args(bss._ResidualNormArgs, **kw), None) == NO_DEVICE
    for kw in (dict(dx=ptr(2)), dict(dy=ptr(3)), dict(dx=ptr(2), dy=ptr(3)), dict(r=ptr(2), dx=ptr(2)),
               dict(y=ptr(3), dy=ptr(3)), dict(dr=ptr(3), dx=ptr(3))):
        assert lib.bss_residual_norm_backward(norm_args(bss._ResidualNormGrads, **kw), None) == NO_DEVICE


# heads: addresses 0 .. 2 are the token-major tensors, 3 .. 5 the head-major ones
@pytest.mark.parametrize("norm", [1, 2])
def test_heads_refuse_outputs_over_what_is_read(lib, no_gpu, norm):
    x = (tokens(6), tokens(7))
    near = lambda i: ptr(i) + 64  # noqa: E731  inside the tensor
    rot = lambda a, i: dict(rotary=rotary(tables=[near(i) if k == a else ptr(10 + k) for k in range(3)]))  # noqa: E731
    for i in (3, 4, 5):  # outputs forward
        for kw in (dict(qw=near(i)), dict(kw=near(i)), dict(flags=near(i)), rot(0, i), rot(1, i), rot(2, i)):
            assert forward(lib, norm=norm, **kw) == INVALID
    for i in (0, 1, 2):  # and back
        for kw in (dict(qw=near(i)), dict(kw=near(i)), dict(flags=near(i)), rot(0, i), rot(2, i)):
            assert backward(lib, norm=norm, x=x, **kw) == INVALID
    good = dict(norm=norm, x=x, ws=ptr(22), ws_bytes=1 << 26, qw=ptr(23), kw=ptr(24), flags=ptr(25), rotary=rotary())
    assert backward(lib, dw=(ptr(20), ptr(21)), **good) == NO_DEVICE
    for i in (0, 1, 2, 3, 4, 5, 6, 7, 10, 22, 23, 24, 25):  # weight gradients over anything
        assert backward(lib, dw=(ptr(i), ptr(21)), **good) == INVALID
        assert backward(lib, dw=(ptr(20), ptr(i)), **good) == INVALID
    assert backward(lib, dw=(ptr(20), ptr(20) + 16), **good) == INVALID
    for i in (0, 1, 2, 3, 4, 5, 6, 7, 10, 20, 21, 23, 24, 25):  # the workspace too
        assert backward(lib, dw=(ptr(20), ptr(21)), **{**good, "ws": ptr(i)}) == INVALID
    # what is not read or written may lie anywhere: no weight gradient, no norm, an axis without pairs
    assert backward(lib, **{**good, "ws": ptr(0)}) == NO_DEVICE
    assert forward(lib, norm=0, qw=near(3)) == NO_DEVICE
    r = rotary(pairs=(22, 0, 21), tables=(ptr(10), near(3), ptr(12)))
    assert forward(lib, norm=norm, rotary=r) == NO_DEVICE


@pytest.mark.parametrize("group", [7, 1 << 40, (1 << 63) - 1])
def test_norm_groups_longer_than_the_rows(lib, no_gpu, group):
    """One group, however many rows it could hold: its overlaps are still seen."""
    many = dict(rows_per_group=group)
    assert lib.bss_residual_norm(norm_args(bss._ResidualNormArgs, gate=ptr(8), gate_stride=4, **many), None) == NO_DEVICE
    assert lib.bss_residual_norm(norm_args(bss._ResidualNormArgs, gate=ptr(3) + 256, **many), None) == INVALID
    ws = dict(workspace=ptr(10), workspace_bytes=1 << 24)
    back = lambda **kw: lib.bss_residual_norm_backward(norm_args(bss._ResidualNormGrads, **many, **ws, **kw), None)  # noqa: E731
    assert back(dshift=ptr(9)) == NO_DEVICE
    for over in (ptr(3), ptr(4) + 64, ptr(10)):
        assert back(dshift=over) == INVALID
        assert back(dgate=over) == INVALID

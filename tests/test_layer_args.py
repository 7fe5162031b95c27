"""Refusals of the matrix products and the cross attention, on the CPU: the C ABI
returns its errors before anything is launched."""
import ctypes

import pytest

import block_sparse_spatio_gb300 as bss
from test_block_args import INVALID, UNSUPPORTED, lib, ptr  # noqa: F401

NAN, INF = float("nan"), float("inf")


def linear_args(**kw):
    a = dict(rows=100, rows_per_group=100, in_channels=64, out_channels=128, out_dtype=0, param_dtype=1, activation=0,
             residual_scale=1.0, x=ptr(0), weight=ptr(1), bias=ptr(2), gate=None, residual=None, out=ptr(3), pre=None,
             x_stride=64, weight_stride=64, gate_stride=128, residual_stride=128, out_stride=128, pre_stride=128,
             workspace=ptr(9), workspace_bytes=1 << 40)
    a.update(kw)
    return bss._LinearArgs(**a)


BAD_LINEAR = [
    (dict(rows=0), INVALID), (dict(rows=-1), INVALID), (dict(rows=1 << 31), UNSUPPORTED), (dict(rows_per_group=0), INVALID),
    (dict(in_channels=0), INVALID), (dict(in_channels=60), INVALID), (dict(out_channels=4), INVALID),
    (dict(in_channels=65544), UNSUPPORTED), (dict(out_channels=65544), UNSUPPORTED),
    (dict(out_dtype=2), INVALID), (dict(param_dtype=-1), INVALID), (dict(activation=4), INVALID), (dict(activation=-1), INVALID),
    (dict(x=None), INVALID), (dict(weight=None), INVALID), (dict(out=None), INVALID),
    (dict(residual_scale=0.5), INVALID), (dict(residual=ptr(4), residual_scale=NAN), INVALID),
    (dict(residual=ptr(4), residual_scale=INF), INVALID),
]
BAD_LINEAR_TENSORS = [
    dict(x=ptr(0) + 8), dict(weight=ptr(1) + 4), dict(bias=ptr(2) + 4), dict(out=ptr(3) + 2), dict(gate=ptr(5) + 8),
    dict(x_stride=60), dict(x_stride=-64), dict(x_stride=(1 << 28) + 8), dict(weight_stride=68), dict(out_stride=120),
    dict(out_stride=0), dict(residual=ptr(4), residual_stride=4), dict(pre=ptr(6), pre_stride=64),
    dict(gate=ptr(5), rows_per_group=10, gate_stride=4), dict(out=ptr(0)), dict(out=ptr(1)), dict(out=ptr(2)),
    dict(pre=ptr(3)), dict(pre=ptr(4), residual=ptr(4)), dict(residual=ptr(3), residual_stride=136),
    dict(residual=ptr(3) + 256), dict(gate=ptr(3) + 16),
]


@pytest.mark.parametrize("kw,code", BAD_LINEAR)
def test_linear_refuses(lib, kw, code):  # noqa: F811
    a = linear_args(**kw)
    assert lib.bss_linear(ctypes.byref(a), None) == code
    assert lib.bss_last_error_message() != b""
    need = ctypes.c_int64(7)
    assert lib.bss_linear_workspace(ctypes.byref(a), ctypes.byref(need)) == code and need.value == 0


@pytest.mark.parametrize("kw", BAD_LINEAR_TENSORS)
def test_linear_refuses_tensors(lib, kw):  # noqa: F811
    a = linear_args(**kw)
    assert lib.bss_linear(ctypes.byref(a), None) == INVALID
    assert lib.bss_last_error_message() != b""


def test_linear_refuses_null_and_short_workspaces(lib):  # noqa: F811
    need = ctypes.c_int64()
    assert lib.bss_linear(None, None) == INVALID
    assert lib.bss_linear_workspace(None, ctypes.byref(need)) == INVALID
    assert lib.bss_linear_workspace(ctypes.byref(linear_args()), None) == INVALID
    # a long contraction with one tile: split
    kw = dict(rows=64, rows_per_group=64, in_channels=65536, x_stride=65536, weight_stride=65536, x=ptr(0), weight=ptr(1))
    assert lib.bss_linear_workspace(ctypes.byref(linear_args(**kw)), ctypes.byref(need)) == 0 and need.value > 0
    for bad in (dict(workspace=None), dict(workspace_bytes=need.value - 1), dict(workspace=ptr(9) + 8),
                dict(workspace=ptr(3)), dict(workspace=ptr(0) + 4096)):
        assert lib.bss_linear(ctypes.byref(linear_args(**kw, **bad)), None) == INVALID


def grad_args(**kw):
    a = dict(rows=100, rows_per_group=100, in_channels=64, out_channels=128, dout_dtype=0, param_dtype=1, dweight_dtype=0,
             activation=1, dout=ptr(0), x=ptr(1), weight=ptr(2), pre=ptr(3), gate=None, dx=ptr(4), dweight=ptr(5),
             dbias=ptr(6), dgate=None, dout_stride=128, x_stride=64, weight_stride=64, pre_stride=128, gate_stride=128,
             dx_stride=64, dweight_stride=64, workspace=ptr(20), workspace_bytes=1 << 40)
    a.update(kw)
    return bss._LinearGrads(**a)


BAD_GRADS = [
    (dict(rows=0), INVALID), (dict(rows=1 << 31), UNSUPPORTED), (dict(rows_per_group=-3), INVALID),
    (dict(in_channels=12), INVALID), (dict(out_channels=65544), UNSUPPORTED), (dict(dout_dtype=3), INVALID),
    (dict(dweight_dtype=3), INVALID), (dict(activation=9), INVALID), (dict(dout=None), INVALID),
    (dict(dx=None, dweight=None, dbias=None), INVALID), (dict(weight=None), INVALID), (dict(x=None), INVALID),
    (dict(dgate=ptr(7)), INVALID), (dict(pre=None), INVALID), (dict(activation=0, pre=None, gate=ptr(8), dgate=ptr(7)), INVALID),
    (dict(workspace=None), INVALID), (dict(workspace_bytes=100), INVALID),
]
BAD_GRAD_TENSORS = [
    dict(dout=ptr(0) + 8), dict(dx=ptr(4) + 8), dict(dbias=ptr(6) + 4), dict(dout_stride=100), dict(dx_stride=32),
    dict(dweight_stride=56), dict(dx=ptr(1)), dict(dx=ptr(0)), dict(dweight=ptr(2)), dict(dbias=ptr(3)), dict(dbias=ptr(5)),
    dict(gate=ptr(8), dgate=ptr(8)), dict(gate=ptr(8), dgate=ptr(6)), dict(workspace=ptr(4)), dict(workspace=ptr(0)),
    dict(pre=ptr(3) + 2), dict(x_stride=-8),
]


@pytest.mark.parametrize("kw,code", BAD_GRADS + [(kw, INVALID) for kw in BAD_GRAD_TENSORS])
def test_linear_backward_refuses(lib, kw, code):  # noqa: F811
    assert lib.bss_linear_backward(ctypes.byref(grad_args(**kw)), None) == code
    assert lib.bss_last_error_message() != b""


def tok(i, H=6, d=64, **kw):
    a = dict(data=ptr(i), token_stride=H * d, head_stride=d)
    a.update(kw)
    return bss._TokenTensor(**a)


def states(i, L=33, H=3, d=64, **kw):
    a = dict(data=ptr(i), group_stride=L * H * d, token_stride=H * d, head_stride=d)
    a.update(kw)
    return bss._StateTensor(**a)


def cross_args(**kw):
    a = dict(rows=100, rows_per_group=40, heads=6, kv_heads=3, head_dim=64, keys=33, softmax_scale=0.0, q=tok(0), O=tok(1),
             k=states(2), v=states(3), lengths=ptr(4), lse=ptr(5))
    a.update(kw)
    return bss._CrossArgs(**a)


BAD_CROSS = [
    (dict(rows=0), INVALID), (dict(rows=0x7FFFFFFF), UNSUPPORTED), (dict(rows_per_group=0), INVALID), (dict(heads=0), INVALID),
    (dict(kv_heads=4), INVALID), (dict(kv_heads=-3), INVALID), (dict(heads=65538, kv_heads=3), UNSUPPORTED),
    (dict(head_dim=96), UNSUPPORTED), (dict(head_dim=0), UNSUPPORTED), (dict(keys=0), INVALID),
    (dict(keys=0x7FFFFFFF), UNSUPPORTED), (dict(softmax_scale=NAN), INVALID), (dict(softmax_scale=INF), INVALID),
    (dict(lengths=ptr(4) + 2), INVALID),
    (dict(rows=1 << 30, rows_per_group=1, heads=600, kv_heads=3, q=tok(0, token_stride=600 * 64), O=tok(1 << 20, token_stride=600 * 64),
          lengths=None, lse=None, k=states(2, group_stride=0), v=states(3, group_stride=0)), UNSUPPORTED),
]
BAD_TOKENS = [dict(data=None), dict(data=ptr(0) + 8), dict(token_stride=0), dict(token_stride=-8), dict(token_stride=388),
              dict(token_stride=(1 << 28) + 8), dict(head_stride=0), dict(head_stride=4), dict(head_stride=(1 << 38) + 8)]
BAD_STATES = [dict(data=None), dict(data=ptr(2) + 8), dict(token_stride=0), dict(token_stride=-8), dict(token_stride=4),
              dict(token_stride=(1 << 28) + 8), dict(head_stride=0), dict(head_stride=-64), dict(group_stride=-8),
              dict(group_stride=(1 << 38) + 8)]


@pytest.mark.parametrize("kw,code", BAD_CROSS)
def test_cross_refuses(lib, kw, code):  # noqa: F811
    assert lib.bss_cross_attention(ctypes.byref(cross_args(**kw)), None) == code
    assert lib.bss_last_error_message() != b""


def test_cross_refuses_tensors(lib):  # noqa: F811
    call = lambda **kw: lib.bss_cross_attention(ctypes.byref(cross_args(**kw)), None)  # noqa: E731
    assert lib.bss_cross_attention(None, None) == INVALID
    for kw in BAD_TOKENS:
        assert call(q=tok(0, **kw)) == INVALID, kw
        assert call(O=tok(1, **kw)) == INVALID, kw
    for kw in BAD_STATES:
        assert call(k=states(2, **kw)) == INVALID, kw
        assert call(v=states(3, **kw)) == INVALID, kw
    assert call(k=states(2, group_stride=0)) == UNSUPPORTED  # v has groups of its own
    assert call(lse=ptr(5) + 2) == INVALID
    # outputs over something else: inputs, one another, themselves
    for kw in (dict(O=tok(2)), dict(O=tok(0, data=ptr(0) + 128)), dict(O=tok(0, token_stride=512)), dict(lse=ptr(1)),
               dict(lse=ptr(4)), dict(lse=ptr(0)), dict(O=tok(1, token_stride=320)), dict(O=tok(1, head_stride=32))):
        assert call(**kw) == INVALID, kw


def cross_grads(**kw):
    a = dict(rows=100, rows_per_group=40, heads=6, kv_heads=3, head_dim=64, keys=33, softmax_scale=0.0, dO=tok(0), q=tok(1),
             O=tok(2), dq=tok(3), k=states(4), v=states(5), dk=states(6), dv=states(7), lengths=ptr(8), lse=ptr(9),
             workspace=ptr(20), workspace_bytes=1 << 40)
    a.update(kw)
    return bss._CrossGrads(**a)


def test_cross_backward_refuses(lib):  # noqa: F811
    call = lambda **kw: lib.bss_cross_attention_backward(ctypes.byref(cross_grads(**kw)), None)  # noqa: E731
    need = ctypes.c_int64()
    assert lib.bss_cross_attention_backward(None, None) == INVALID
    assert lib.bss_cross_attention_backward_workspace(None, ctypes.byref(need)) == INVALID
    for kw, code in BAD_CROSS[:-1]:
        if "lengths" not in kw:
            assert call(**kw) == code, kw
    for kw in BAD_TOKENS:
        for name in ("dO", "q", "O", "dq"):
            assert call(**{name: tok(0, **kw)}) == INVALID, (name, kw)
    for kw in BAD_STATES:
        for name in ("k", "v", "dk", "dv"):
            assert call(**{name: states(4, **kw)}) == INVALID, (name, kw)
    for kw in (dict(lse=None), dict(workspace=None), dict(workspace_bytes=1000), dict(workspace=ptr(20) + 8), dict(dq=tok(1)),
               dict(dq=tok(0)), dict(dk=states(7)), dict(dv=states(5)), dict(dk=states(6, group_stride=0)),
               dict(dk=states(6, token_stride=64)), dict(workspace=ptr(3)), dict(dv=states(7, group_stride=64))):
        assert call(**kw) == INVALID, kw
    assert call(k=states(4, group_stride=0), v=states(5, group_stride=0)) == UNSUPPORTED
    # gradients whose groups, tokens and heads all lie apart
    assert call(dk=states(6, group_stride=33 * 1024, token_stride=1000, head_stride=72)) == UNSUPPORTED
    assert lib.bss_cross_attention_backward_workspace(ctypes.byref(cross_grads()), ctypes.byref(need)) == 0
    assert need.value >= 4 * 6 * 100

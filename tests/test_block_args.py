"""Refusals of the operators around the attention step, on the CPU: the C ABI
returns its errors before anything is launched."""
import ctypes

import pytest
import torch

import block_sparse_spatio_gb300 as bss

INVALID, UNSUPPORTED = 1, 2


@pytest.fixture(scope="module")
def lib():
    from block_sparse_spatio_gb300 import build
    build.build()
    return bss.load()


def ptr(i):
    """Made-up device addresses, 4 GiB apart: never touched."""
    return (i + 1) << 32


def tokens(i, H=4, d=128, **kw):
    a = dict(data=ptr(i), token_stride=H * d, head_stride=d)
    a.update(kw)
    return bss._TokenTensor(**a)


def heads_call(lib, backward=False, params=None, H=4, rotary=None, norm=0, eps=1e-6, weight_dtype=1, qw=None, kw=None,
               ins=None, outs=None, x=(None, None), dw=(None, None), ws=None, ws_bytes=0, options=True, flags=None):
    p = bss.MaskParams(3, 4, 5, 128, 1, 1) if params is None else params
    mp = None if p == "null" else ctypes.byref(p.c())
    o = bss._HeadsOptions(norm, eps, weight_dtype, qw, kw, None if rotary is None else ctypes.pointer(rotary))
    op = ctypes.byref(o) if options else None
    tok = [None if t is None else ctypes.byref(t) for t in (ins if not backward else outs)]
    flat = outs if not backward else ins
    if not backward:
        return lib.bss_heads_from_tokens(*tok, *flat, flags, H, mp, op, None)
    xs = [None if t is None else ctypes.byref(t) for t in x]
    return lib.bss_heads_from_tokens_backward(*flat, *xs, *tok, *dw, flags, H, mp, op, ws, ws_bytes, None)


def forward(lib, **kw):
    a = dict(ins=[tokens(i) for i in range(3)], outs=[ptr(i + 3) for i in range(3)])
    a.update(kw)
    return heads_call(lib, **a)


def backward(lib, **kw):
    a = dict(ins=[ptr(i + 3) for i in range(3)], outs=[tokens(i) for i in range(3)])
    a.update(kw)
    return heads_call(lib, backward=True, **a)


def rotary(pairs=(22, 21, 21), length=(3, 4, 5), offset=(0, 0, 0), pairing=0, tables=(ptr(10), ptr(11), ptr(12))):
    r = bss._Rotary()
    for i in range(3):
        r.table[i], r.pairs[i], r.length[i], r.offset[i] = tables[i], pairs[i], length[i], offset[i]
    r.pairing = pairing
    return r


BAD_OPTIONS = [
    (dict(params="null"), INVALID),
    (dict(options=False), INVALID),
    (dict(params=bss.MaskParams(0, 4, 5, 128, 1, 1)), INVALID),
    (dict(params=bss.MaskParams(3, 4, 5, 96, 1, 1)), UNSUPPORTED),
    (dict(H=0), INVALID),
    (dict(H=65536), UNSUPPORTED),
    (dict(norm=3), INVALID),
    (dict(norm=-1), INVALID),
    (dict(norm=1, eps=-1.0), INVALID),
    (dict(norm=1, eps=float("nan")), INVALID),
    (dict(norm=1, eps=float("inf")), INVALID),
    (dict(norm=1, weight_dtype=2), INVALID),
    (dict(norm=1, qw=ptr(9) + 4), INVALID),
    (dict(norm=2, H=65), UNSUPPORTED),  # 8320 channels a token
    (dict(rotary=rotary(pairing=2)), INVALID),
    (dict(rotary=rotary(pairs=(22, 21, 22))), INVALID),
    (dict(rotary=rotary(pairs=(22, -1, 21))), INVALID),
    (dict(rotary=rotary(length=(2, 4, 5))), INVALID),
    (dict(rotary=rotary(offset=(0, 1, 0))), INVALID),
    (dict(rotary=rotary(offset=(0, 0, -1))), INVALID),
    (dict(rotary=rotary(tables=(ptr(10), None, ptr(12)))), INVALID),
    (dict(rotary=rotary(tables=(ptr(10) + 8, ptr(11), ptr(12)))), INVALID),
    (dict(rotary=rotary(pairs=(22, 21, 20), pairing=1)), UNSUPPORTED),  # 126 channels in halves
]


@pytest.mark.parametrize("kw,code", BAD_OPTIONS)
def test_heads_refuse_bad_options_both_ways(lib, kw, code):
    assert forward(lib, **kw) == code
    assert lib.bss_last_error_message() != b""
    extra = dict(x=(tokens(6), tokens(7))) if kw.get("norm") else {}
    assert backward(lib, **kw, **extra) == code


def test_heads_refuse_bad_tensors(lib):
    good_in, good_out = [tokens(i) for i in range(3)], [ptr(i + 3) for i in range(3)]

    def one(i, t, lst):
        lst = list(lst)
        lst[i] = t
        return lst
    for t in (tokens(0, data=ptr(0) + 8), tokens(0, token_stride=514), tokens(0, head_stride=-8),
              tokens(0, head_stride=1 << 60)):
        assert forward(lib, ins=one(0, t, good_in)) == INVALID
        assert backward(lib, outs=one(0, t, good_in)) == INVALID
    assert forward(lib, outs=one(1, ptr(4) + 8, good_out)) == INVALID
    assert forward(lib, outs=one(1, None, good_out)) == INVALID       # k without Kh
    assert forward(lib, ins=one(1, None, good_in)) == INVALID
    assert forward(lib, ins=[None] * 3, outs=[None] * 3) == INVALID
    assert forward(lib, outs=one(1, ptr(3) + 4096, good_out)) == INVALID   # outputs overlap
    assert forward(lib, outs=one(0, ptr(2) + 16, good_out)) == INVALID     # over an input
    # gradients: outputs that overlap themselves, each other or an input
    assert backward(lib, outs=one(0, tokens(0, head_stride=0), good_in)) == INVALID
    assert backward(lib, outs=one(0, tokens(0, token_stride=384), good_in)) == INVALID
    assert backward(lib, outs=one(0, tokens(1), good_in)) == INVALID
    assert backward(lib, outs=one(0, tokens(3), good_in)) == INVALID
    assert backward(lib, norm=1, x=(tokens(0), tokens(7))) == INVALID      # dq over q
    assert backward(lib, norm=1) == INVALID                                # no q
    assert backward(lib, norm=1, x=(tokens(6), None)) == INVALID
    assert backward(lib, dw=(ptr(20), None)) == INVALID                    # a weight gradient without a norm
    assert backward(lib, norm=1, x=(tokens(6), tokens(7)), dw=(ptr(20), None)) == INVALID  # no workspace


def test_heads_workspace_query(lib):
    n = ctypes.c_int64(-1)
    p = bss.MaskParams(3, 4, 5, 128, 1, 1).c()
    assert lib.bss_heads_from_tokens_backward_workspace(4, ctypes.byref(p), 0, ctypes.byref(n)) == 0 and n.value == 0
    assert lib.bss_heads_from_tokens_backward_workspace(4, ctypes.byref(p), 1, ctypes.byref(n)) == 0 and n.value > 0
    need = n.value
    assert lib.bss_heads_from_tokens_backward_workspace(4, ctypes.byref(p), 7, ctypes.byref(n)) == INVALID
    assert lib.bss_heads_from_tokens_backward_workspace(4, ctypes.byref(p), 1, None) == INVALID
    assert lib.bss_heads_from_tokens_backward_workspace(4, None, 1, ctypes.byref(n)) == INVALID
    assert backward(lib, norm=1, x=(tokens(6), tokens(7)), dw=(ptr(20), None), ws=ptr(21), ws_bytes=need - 1) == INVALID
    assert backward(lib, norm=1, x=(tokens(6), tokens(7)), dw=(ptr(20), None), ws=ptr(21) + 8, ws_bytes=need) == INVALID


def test_step_from_tokens_refuses_a_stale_map(lib):
    t = ctypes.byref(tokens(0))
    o = bss._HeadsOptions(0, 1e-6, 1, None, None, None)
    assert lib.bss_attention_step_tokens(t, t, t, ptr(5), None, ctypes.c_void_p(0x1234), None, 4, ctypes.byref(o),
                                         ptr(6), ptr(7), ptr(8), None) == INVALID


@pytest.mark.parametrize("kw", [dict(length=0), dict(pairs=0), dict(dim=0), dict(base=0.0), dict(base=-2.0),
                                dict(base=float("nan")), dict(base=float("inf")), dict(out=None),
                                dict(out=ptr(0) + 8), dict(positions=ptr(1) + 4)])
def test_rotary_table_refuses(lib, kw):
    a = dict(positions=None, length=4, pairs=3, dim=6, base=100.0, out=ptr(0))
    a.update(kw)
    assert lib.bss_rotary_table(a["positions"], a["length"], a["pairs"], a["dim"], a["base"], a["out"], None) == INVALID


def test_rotary_table_refuses_too_many_entries(lib):
    assert lib.bss_rotary_table(None, 1 << 20, 1 << 11, 6, 100.0, ptr(0), None) == UNSUPPORTED


def norm_args(cls, **kw):
    a = dict(rows=6, rows_per_group=2, channels=64, stream_dtype=0, branch_dtype=0, param_dtype=1, norm=1, y_norm=0,
             residual_scale=1.0)
    if cls is bss._ResidualNormArgs:
        a.update(eps=1e-6, x=ptr(0), y=ptr(1), r=ptr(2), h=ptr(3), x_stride=64, y_stride=64, r_stride=64, h_stride=64)
    else:
        a.update(r=ptr(0), y=ptr(1), dr=ptr(2), dh=ptr(3), dx=ptr(4), dy=ptr(5), stats=ptr(6), r_stride=64, y_stride=64,
                 dr_stride=64, dh_stride=64, dx_stride=64, dy_stride=64)
    a.update(kw)
    return ctypes.byref(cls(**a))


COMMON = [
    (dict(rows=0), INVALID), (dict(rows=-1), INVALID), (dict(rows=1 << 31), UNSUPPORTED),
    (dict(rows_per_group=0), INVALID), (dict(channels=0), INVALID), (dict(channels=60), INVALID),
    (dict(channels=8200), UNSUPPORTED), (dict(stream_dtype=2), INVALID), (dict(branch_dtype=-1), INVALID),
    (dict(param_dtype=5), INVALID), (dict(branch_dtype=1), UNSUPPORTED), (dict(norm=3), INVALID),
    (dict(y_norm=-1), INVALID), (dict(residual_scale=float("inf")), INVALID),
    (dict(residual_scale=float("nan")), INVALID), (dict(gate=ptr(8) + 4, gate_stride=64), INVALID),
    (dict(scale=ptr(8), scale_stride=4), INVALID), (dict(weight=ptr(8) + 8), INVALID),
]
FORWARD = [
    (dict(eps=-1e-6), INVALID), (dict(eps=float("nan")), INVALID), (dict(x=None), INVALID), (dict(r=None, h=None), INVALID),
    (dict(y=None), INVALID), (dict(y=None, r=None, gate=ptr(8)), INVALID),
    (dict(y=None, r=None, residual_scale=0.5), INVALID), (dict(y=None, r=None, y_norm=1), INVALID),
    (dict(h=None, scale=ptr(8), scale_stride=64), INVALID), (dict(h=None, stats=ptr(8)), INVALID),
    (dict(norm=0, stats=ptr(8)), INVALID), (dict(y_stats=ptr(8)), INVALID), (dict(stats=ptr(8) + 4), INVALID),
    (dict(x=ptr(0) + 8), INVALID), (dict(x_stride=68), INVALID), (dict(h_stride=56), INVALID),
    (dict(h_stride=-64), INVALID), (dict(r=ptr(0) + 16), INVALID), (dict(r=ptr(0), r_stride=128), INVALID),
    (dict(h=ptr(0)), INVALID), (dict(r=ptr(1)), INVALID), (dict(h=ptr(2)), INVALID), (dict(stats=ptr(3)), INVALID),
    (dict(r=ptr(0), x_stride=0, r_stride=64), INVALID),
]
BACKWARD = [
    (dict(dx=None), INVALID), (dict(dr=None, dh=None), INVALID), (dict(r=None), INVALID), (dict(stats=None), INVALID),
    (dict(dy=None), INVALID), (dict(y=None), INVALID), (dict(y_norm=1), INVALID),
    (dict(y=None, dy=None, dgate=ptr(9)), INVALID), (dict(y=None, dy=None, residual_scale=2.0), INVALID),
    (dict(dh=None, dscale=ptr(9)), INVALID), (dict(dh=None, dbias=ptr(9)), INVALID), (dict(stats=ptr(6) + 4), INVALID),
    (dict(dshift=ptr(9) + 4), INVALID), (dict(dshift=ptr(9)), INVALID),            # no workspace
    (dict(dshift=ptr(9), workspace=ptr(10), workspace_bytes=64), INVALID),
    (dict(dshift=ptr(9), workspace=ptr(10) + 8, workspace_bytes=1 << 24), INVALID),
    (dict(dshift=ptr(9), workspace=ptr(0), workspace_bytes=1 << 24), INVALID),
    (dict(dshift=ptr(3), workspace=ptr(10), workspace_bytes=1 << 24), INVALID),
    (dict(dx=ptr(2), dx_stride=128), INVALID), (dict(dx=ptr(2) + 64), INVALID), (dict(dx=ptr(0)), INVALID),
    (dict(dy=ptr(1)), INVALID), (dict(dy=ptr(4)), INVALID), (dict(dx_stride=32), INVALID),
]


@pytest.mark.parametrize("kw,code", COMMON + FORWARD)
def test_residual_norm_refuses(lib, kw, code):
    assert lib.bss_residual_norm(norm_args(bss._ResidualNormArgs, **kw), None) == code
    assert lib.bss_last_error_message() != b""


@pytest.mark.parametrize("kw,code", COMMON + BACKWARD)
def test_residual_norm_backward_refuses(lib, kw, code):
    assert lib.bss_residual_norm_backward(norm_args(bss._ResidualNormGrads, **kw), None) == code


def test_residual_norm_null_and_workspace(lib):
    n = ctypes.c_int64(-1)
    assert lib.bss_residual_norm(None, None) == INVALID
    assert lib.bss_residual_norm_backward(None, None) == INVALID
    assert lib.bss_residual_norm_backward_workspace(None, ctypes.byref(n)) == INVALID
    g = norm_args(bss._ResidualNormGrads)
    assert lib.bss_residual_norm_backward_workspace(g, None) == INVALID
    assert lib.bss_residual_norm_backward_workspace(g, ctypes.byref(n)) == 0 and n.value == 0
    g = norm_args(bss._ResidualNormGrads, dshift=ptr(9))
    assert lib.bss_residual_norm_backward_workspace(g, ctypes.byref(n)) == 0 and n.value > 0


def test_binding_refuses_cpu_tensors_and_bad_shapes():
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        bss.residual_norm(x, h=x)
    with pytest.raises(ValueError):
        bss.residual_norm_backward(x, dh=x, dx=x)
    with pytest.raises(ValueError):
        bss.Rotary(torch.zeros(4, 64))
    with pytest.raises(ValueError):
        bss.Rotary(torch.zeros(4, 8, 2))
    with pytest.raises(ValueError):
        bss.heads_from_tokens(None, None, None, None, None, None, bss.MaskParams(1, 1, 1, 64, 0, 0))
    with pytest.raises(ValueError):
        bss.rotary_table(0, 4)


def test_step_from_tokens_refuses_before_the_first_launch(lib):
    """With a map that is never dereferenced on the device: a stale one only, on the CPU."""
    o = bss._HeadsOptions(0, 1e-6, 1, None, None, None)
    t = ctypes.byref(tokens(0))
    for m in (None, ctypes.c_void_p(0x40)):
        assert lib.bss_attention_step_tokens(t, t, t, ptr(5), None, m, None, 4, ctypes.byref(o), ptr(6), ptr(7), ptr(8),
                                             None) == INVALID

"""linear and its gradients on the GPU against the 64-bit formulas: sizes around
the tiles and vectors, one row to many, strides, types, groups, in place, captured."""
import pytest
import torch

import _layers_ref as L
from _block_ref import check

DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32
# (rows, in, out): one element of everything, ragged tiles on each side, several tiles, a long contraction
SIZES = [(1, 8, 8), (1, 64, 7680), (2, 72, 136), (7, 1000, 24), (16, 1280, 264), (17, 136, 520), (33, 8, 264), (64, 2056, 40),
         (65, 128, 128), (127, 64, 256), (128, 200, 256), (129, 264, 264), (255, 72, 8), (256, 128, 512), (300, 520, 328),
         (513, 64, 776), (1001, 248, 136), (40, 20480, 64)]


def strided(t, pad):
    """The same values in rows `pad` elements further apart."""
    if t is None or not pad:
        return t
    wide = torch.full((t.shape[0], t.shape[1] + pad), float("nan"), dtype=t.dtype, device=t.device)
    wide[:, :t.shape[1]] = t
    return wide[:, :t.shape[1]]


def rnd(g, *s, dtype=F32, scale=1.0):
    return (torch.randn(*s, generator=g) * scale).to(dtype)


def dev(t, pad=0):
    return None if t is None else strided(t.to(DEV), pad)


def forward(bss, rows, inner, outer, kind=0, out=BF, params=F32, bias=True, gate=False, residual=False, a=1.0, group=None,
            pre=False, pad=0, inplace=False, seed=0, x=None):
    g = torch.Generator().manual_seed(seed)
    x = rnd(g, rows, inner, dtype=BF) if x is None else x
    w = rnd(g, outer, inner, dtype=BF, scale=2.0 * inner ** -0.5)
    group = group or rows
    G = -(-rows // group)
    b = rnd(g, outer, dtype=params) if bias else None
    ga = rnd(g, G, outer, dtype=params) if gate else None
    r = rnd(g, rows, outer, dtype=out) if residual else None
    ref = L.linear(x, w, b, kind, ga, r, group, a)
    rd = dev(r, pad)
    o = rd if inplace else dev(torch.full((rows, outer), float("nan"), dtype=out), pad)
    p = dev(torch.full((rows, outer), float("nan"), dtype=BF), pad) if pre else None
    bss.linear(dev(x, pad), dev(w, pad), o, bias=dev(b), activation=kind, gate=dev(ga, pad), residual=rd,
               rows_per_group=group, residual_scale=a, pre=p)
    torch.cuda.synchronize()
    assert bss.get_device_status() == 0
    check(o, *ref["out"], 1, "out")
    if pre:
        check(p, *ref["pre"], 1, "pre")
    for t in (o, p):  # what lies between the rows stays
        if t is not None and pad and rows > 1:
            gap = t.as_strided((rows - 1, pad), (outer + pad, 1), t.storage_offset() + outer)
            assert torch.isnan(gap).all()
    return o


@pytest.mark.gpu
@pytest.mark.parametrize("rows,inner,outer", SIZES)
def test_sizes(bss, rows, inner, outer):
    forward(bss, rows, inner, outer)
    forward(bss, rows, inner, outer, kind=1, out=F32, pre=True, pad=8, gate=True, residual=True, group=max(1, rows // 3))


@pytest.mark.gpu
@pytest.mark.parametrize("rows", [1, 5, 130, 520])
@pytest.mark.parametrize("kind", [0, 1, 2, 3])
@pytest.mark.parametrize("out,params", [(BF, F32), (F32, BF)])
def test_activations_and_types(bss, rows, kind, out, params):
    forward(bss, rows, 96, 136, kind=kind, out=out, params=params, pre=True)
    forward(bss, rows, 96, 136, kind=kind, out=out, params=params, bias=False, gate=True, residual=True, a=0.5,
            group=max(1, rows // 4), pad=24, inplace=True)


@pytest.mark.gpu
@pytest.mark.parametrize("group", [1, 2, 31, 129, 400])
@pytest.mark.parametrize("rows", [11, 387])
def test_groups(bss, rows, group):
    forward(bss, rows, 64, 264, gate=True, group=group)


@pytest.mark.gpu
def test_one_row_repeated(bss):
    """A broadcast input (row stride 0)."""
    g = torch.Generator().manual_seed(1)
    x = rnd(g, 1, 128, dtype=BF)
    w = rnd(g, 64, 128, dtype=BF)
    o = torch.empty(200, 64, dtype=BF, device=DEV)
    bss.linear(x.to(DEV).expand(200, 128), w.to(DEV), o)
    check(o, *L.linear(x.expand(200, 128), w)["out"], 1)


@pytest.mark.gpu
def test_extreme_values(bss):
    """Large and infinite pre-activations meet their limits; NaN stays in its row."""
    x = torch.zeros(5, 8, dtype=BF)
    x[0, 0], x[1, 0], x[2, 0], x[3, 0], x[4, 0] = 3e38, -3e38, 100, -100, float("nan")
    w = torch.zeros(8, 8, dtype=BF)
    w[:, 0] = 1
    for kind in (1, 2, 3):
        o = torch.empty(5, 8, dtype=F32, device=DEV)
        bss.linear(x.to(DEV), w.to(DEV), o, activation=kind)
        want = L.act(x[:4, 0].double(), 3)[0]
        got = o.double().cpu()
        assert torch.equal(got[0], want[0].expand(8)) and torch.equal(got[2], want[2].expand(8))
        assert (got[1].abs() == 0).all() and (got[3].abs() < 1e-30).all()
        assert torch.isnan(got[4]).all()
        # slopes: 1 and 0
        dx = torch.empty(4, 8, dtype=BF, device=DEV)
        pre = x[:4, :1].expand(4, 8).contiguous().to(DEV)
        eye = torch.eye(8, dtype=BF, device=DEV)
        bss.linear_backward(torch.ones(4, 8, dtype=BF, device=DEV), weight=eye, dx=dx, activation=kind, pre=pre)
        assert torch.equal(dx.float().cpu(), torch.tensor([1.0, 0, 1, 0])[:, None].expand(4, 8))


def backward(bss, rows, inner, outer, kind=0, dtype=BF, dw=F32, params=F32, gate=False, group=None, pad=0, seed=0,
             want=("dx", "dweight", "dbias", "dgate"), workspace=None):
    g = torch.Generator().manual_seed(seed)
    x, w = rnd(g, rows, inner, dtype=BF), rnd(g, outer, inner, dtype=BF, scale=2.0 * inner ** -0.5)
    group = group or rows
    G = -(-rows // group)
    ga = rnd(g, G, outer, dtype=params) if gate else None
    d = rnd(g, rows, outer, dtype=dtype)
    pre = rnd(g, rows, outer, dtype=BF, scale=2.0) if kind or gate else None
    ref = L.linear_grad(d, x, w, pre, kind, ga, group)
    outs = {"dx": dev(torch.full((rows, inner), float("nan"), dtype=BF), pad),
            "dweight": dev(torch.full((outer, inner), float("nan"), dtype=dw), pad),
            "dbias": torch.full((outer,), float("nan"), device=DEV),
            "dgate": torch.full((G, outer), float("nan"), device=DEV) if gate else None}
    outs = {k: t for k, t in outs.items() if k in want and t is not None}
    bss.linear_backward(dev(d, pad), dev(x, pad), dev(w, pad), activation=kind, pre=dev(pre, pad), gate=dev(ga, pad),
                        rows_per_group=group, workspace=workspace, **outs)
    torch.cuda.synchronize()
    assert bss.get_device_status() == 0
    for k, t in outs.items():
        check(t, *ref[k], 1, k)
    return outs


@pytest.mark.gpu
@pytest.mark.parametrize("rows,inner,outer", SIZES)
def test_backward_sizes(bss, rows, inner, outer):
    backward(bss, rows, inner, outer)
    backward(bss, rows, inner, outer, kind=3, dw=BF, gate=True, group=max(1, rows // 3), pad=8)


@pytest.mark.gpu
@pytest.mark.parametrize("rows", [1, 6, 300])
@pytest.mark.parametrize("kind", [0, 1, 2, 3])
@pytest.mark.parametrize("dtype,params", [(BF, F32), (F32, BF)])
def test_backward_types(bss, rows, kind, dtype, params):
    backward(bss, rows, 136, 200, kind=kind, dtype=dtype, params=params, gate=kind % 2 == 0, group=max(1, rows // 4))


@pytest.mark.gpu
@pytest.mark.parametrize("group", [1, 2, 5, 31, 32, 33, 129, 700, 2000])
def test_backward_groups(bss, group):
    backward(bss, 1400, 16, 264, kind=1, gate=True, group=group)
    backward(bss, 1400, 16, 8, gate=True, group=group, want=("dgate",))


@pytest.mark.gpu
@pytest.mark.parametrize("want", [("dx",), ("dweight",), ("dbias",), ("dgate",), ("dbias", "dgate"), ("dx", "dbias")])
def test_backward_parts(bss, want):
    backward(bss, 260, 72, 136, kind=2, gate=True, group=100, want=want)
    if want[0] != "dgate":
        backward(bss, 260, 72, 136, want=want)


@pytest.mark.gpu
def test_same_bits_again(bss):
    for rows, inner, outer in ((3000, 128, 264), (20000, 64, 128)):
        a = backward(bss, rows, inner, outer, kind=1, gate=True, group=rows // 3)
        b = backward(bss, rows, inner, outer, kind=1, gate=True, group=rows // 3)
        for k in a:
            assert torch.equal(a[k].view(torch.int16), b[k].view(torch.int16)), k


@pytest.mark.gpu
@pytest.mark.parametrize("kind", [0, 1])
def test_pairs_of_ctas(bss, kind):
    """Results of many 256 x 256 tiles, ragged at every end."""
    forward(bss, 20003, 72, 264, kind=kind, pre=True, gate=True, residual=True, group=777, pad=8)
    backward(bss, 20003, 264, 72, kind=kind)
    backward(bss, 70, 2056, 2568, kind=kind, dw=F32 if kind else BF, pad=8)


@pytest.mark.gpu
@pytest.mark.parametrize("rows,inner,outer", [(20, 4096, 136), (130, 3000, 264), (512, 4096, 640)])
@pytest.mark.parametrize("out", [BF, F32])
def test_split_contraction(bss, rows, inner, outer, out):
    forward(bss, rows, inner, outer, kind=1, out=out, pre=True, gate=True, residual=True, a=0.5, group=max(1, rows // 3), pad=8)
    forward(bss, rows, inner, outer, out=out, bias=False, residual=True, inplace=True)
    backward(bss, inner, rows // 4 * 8, outer, dw=out)


@pytest.mark.gpu
def test_error_function(bss):
    """GELU by the error function in 32 bits over its whole range.  In units of 2^-24 of the
    share: its fit and the polynomial's roundings 5, the quotient 3, two products 2, the
    exponential 4 and three roundings of its argument z^2 / 2, the last steps 2."""
    n = 4096
    z = torch.linspace(-12.5, 12.5, n).to(BF)
    w = torch.zeros(n, 8, dtype=BF)
    w[:, 0] = z
    x = torch.zeros(1, 8, dtype=BF)
    x[0, 0] = 1
    o, slope = torch.empty(1, n, dtype=F32, device=DEV), torch.empty(n, dtype=F32, device=DEV)
    bss.linear(x.to(DEV), w.to(DEV), o, activation=2)
    bss.linear_backward(torch.ones(1, n, dtype=BF, device=DEV), pre=z[None].to(DEV), dbias=slope, activation=2)
    z = z.double()
    value, want = L.act(z, 2)
    units = 16 + 1.5 * z * z
    share = 0.5 * torch.erfc(-z / 2 ** 0.5)
    assert ((o[0].double().cpu() - value).abs() <= units * 2.0 ** -24 * value.abs()).all()
    phi = (want - share).abs()
    assert ((slope.double().cpu() - want).abs() <= units * 2.0 ** -24 * (share + phi) + 2.0 ** -24 * want.abs()).all()


@pytest.mark.gpu
@pytest.mark.parametrize("kind", [0, 2])
def test_many_splits(bss, kind):
    """A long contraction of few results: more splits than a cluster's or a pair's."""
    backward(bss, 20011, 64, 72, kind=kind)

"""linear on the GPU with infinities, NaN and the ends of the range amid ordinary rows, in
each of its kernels: a few rows, tiles, joined by a cluster, summed from memory, pairs."""
import math

import pytest
import torch

import _layers_ref as L
from _block_ref import check
from test_gpu_linear import BF, DEV, F32, rnd

pytestmark = pytest.mark.gpu

SIZES = [(9, 96, 136), (130, 96, 136), (130, 3000, 264), (50, 4096, 72), (20003, 72, 1032)]
ODD = [3e38, -3e38, 100.0, -100.0, math.inf, math.nan]  # the pre-activation of a row each


def inputs(rows, inner, outer):
    """Rows of ODD (by their first channel, whose weights are 1) amid ordinary ones."""
    g = torch.Generator().manual_seed(rows)
    x, w = rnd(g, rows, inner, dtype=BF), rnd(g, outer, inner, dtype=BF, scale=inner ** -0.5)
    w[:, 0] = 1
    at = [(rows - 1) * i // 5 for i in range(6)]
    x[at] = 0
    x[at, 0] = torch.tensor(ODD).to(BF)
    rest = torch.ones(rows, dtype=torch.bool)
    rest[at] = False
    return g, x, w, at, rest


@pytest.mark.parametrize("rows,inner,outer", SIZES)
@pytest.mark.parametrize("kind", [0, 1, 2, 3])
def test_rows_stay_apart(bss, rows, inner, outer, kind):
    g, x, w, at, rest = inputs(rows, inner, outer)
    z = x[at[:5], 0].double()
    value = z if kind == 0 else torch.tensor([z[0], 0, 100, 0, math.inf])
    o, pre = torch.empty(rows, outer, dtype=F32, device=DEV), torch.empty(rows, outer, dtype=BF, device=DEV)
    bss.linear(x.to(DEV), w.to(DEV), o, activation=kind, pre=pre)
    got = o.double().cpu()
    assert torch.isnan(got[at[5]]).all() and torch.isnan(pre[at[5]]).all()
    assert torch.equal(pre[at[:5]].double().cpu(), z[:, None].expand(5, outer))
    assert ((got[at[:5]] == value[:, None]) | ((got[at[:5]] - value[:, None]).abs() < 1e-30)).all()
    check(o[rest.to(DEV)], *L.linear(x[rest], w, kind=kind)["out"], 1, "out")

    # with a gate and a residual, whose own NaN and infinity stay in their rows too
    r = rnd(g, rows, outer)
    bad = next(i for i in range(rows) if rest[i])
    r[bad, :8], r[bad, 8:] = math.inf, math.nan
    gate = torch.full((1, outer), 0.5)
    bss.linear(x.to(DEV), w.to(DEV), o, activation=kind, gate=gate.to(DEV), residual=r.to(DEV))
    got = o.double().cpu()
    assert torch.isnan(got[at[5]]).all()
    assert (got[bad, :8] == math.inf).all() and torch.isnan(got[bad, 8:]).all()
    want = (0.5 * value[:, None] + r[at[:5]].double()).float().double()
    assert torch.equal(got[at[:5]], want)
    rest[bad] = False
    check(o[rest.to(DEV)], *L.linear(x[rest], w, None, kind, gate, r[rest], rows)["out"], 1, "out")


@pytest.mark.parametrize("rows", [9, 130, 2000])
@pytest.mark.parametrize("kind", [1, 2, 3])
def test_slopes_at_the_ends(bss, rows, kind):
    """dx through a weight of ones and zeros: slopes of 1 and 0, NaN in its row alone."""
    g = torch.Generator().manual_seed(rows)
    n = 136
    at = [(rows - 1) * i // 5 for i in range(6)]
    pre = rnd(g, rows, n, dtype=BF, scale=2.0)
    pre[at] = torch.tensor(ODD).to(BF)[:, None].expand(6, n)
    d, w = rnd(g, rows, n, dtype=BF), torch.eye(n, dtype=BF)
    d[at] = 1
    dx = torch.empty(rows, n, dtype=BF, device=DEV)
    bss.linear_backward(d.to(DEV), weight=w.to(DEV), dx=dx, activation=kind, pre=pre.to(DEV))
    got = dx.float().cpu()
    assert torch.equal(got[at[:5]], torch.tensor([1.0, 0, 1, 0, 1])[:, None].expand(5, n))
    assert torch.isnan(got[at[5]]).all()
    rest = torch.ones(rows, dtype=torch.bool)
    rest[at] = False
    check(dx[rest.to(DEV)], *L.linear_grad(d[rest], None, w, pre[rest], kind)["dx"], 1, "dx")

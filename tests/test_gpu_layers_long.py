"""The matrix products and the cross attention on the GPU where elements lie more than
2^32 bytes (and 2^31 elements) from their tensor's start: the last rows, states and heads
against the 64-bit formulas."""
import pytest
import torch

import _layers_ref as L
from _block_ref import check
from test_gpu_linear import BF, DEV, F32

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def seeded():
    torch.manual_seed(5)


def rnd(*s, dtype=BF, scale=1.0):
    t = torch.empty(*s, dtype=dtype, device=DEV)
    t.view(-1).normal_()
    return t.mul_(scale) if scale != 1.0 else t


@pytest.mark.parametrize("kind", [0, 2])
def test_many_rows(bss, kind):
    rows, inner, outer = 450_000, 64, 5120  # 2.3e9 results
    x, w, b, gate = rnd(rows, inner), rnd(outer, inner, scale=inner ** -0.5), rnd(outer, dtype=F32), rnd(3, outer, dtype=F32)
    out, pre = (torch.empty(rows, outer, dtype=BF, device=DEV) for _ in range(2))
    group = 200_000
    bss.linear(x, w, out, bias=b, activation=kind, gate=gate, rows_per_group=group, pre=pre)
    dx, dw, db = torch.empty_like(x), torch.empty(outer, inner, device=DEV), torch.empty(outer, device=DEV)
    assert bss.get_device_status() == 0
    at = torch.cat([torch.arange(3), torch.arange(group - 2, group + 2), torch.arange(rows - 200, rows)])
    g = gate.cpu()[at // group]
    ref = L.linear(x[at].cpu(), w.cpu(), b.cpu(), kind, g, None, 1)
    check(out[at], *ref["out"], 1, "out")
    check(pre[at], *ref["pre"], 1, "pre")
    # backward, with dout in out's place
    bss.linear_backward(out, x, w, dx, dw, db, activation=kind, pre=pre, gate=gate, rows_per_group=group)
    torch.cuda.synchronize()
    assert bss.get_device_status() == 0
    ref = L.linear_grad(out[at].cpu(), None, w.cpu(), pre[at].cpu(), kind, g, 1)
    check(dx[at], *ref["dx"], 1, "dx")
    # a column of the sums over all rows
    col = [0, 5119]
    ref = L.linear_grad(out[:, col].cpu(), x.cpu(), None, pre[:, col].cpu(), kind, gate[:, col].cpu(), group)
    check(dw[col], *ref["dweight"], 1, "dweight")
    check(db[col], *ref["dbias"], 1, "dbias")


@pytest.mark.parametrize("rows", [1, 17, 300])
def test_widest_layer(bss, rows):
    inner = outer = 65536  # 4.3e9 weights
    x, w = rnd(rows, inner), rnd(outer, inner, scale=inner ** -0.5)
    out = torch.empty(rows, outer, dtype=F32, device=DEV)
    bss.linear(x, w, out)
    at = torch.cat([torch.arange(9), torch.arange(outer - 200, outer)])
    check(out[:, at.to(DEV)], *L.linear(x.cpu(), w[at].cpu())["out"], 1, "out")
    del w
    d, dw = rnd(rows, outer), torch.empty(outer, inner, dtype=BF, device=DEV)
    bss.linear_backward(d, x=x, dweight=dw)
    torch.cuda.synchronize()
    assert bss.get_device_status() == 0
    check(dw[at], *L.linear_grad(d[:, at.to(DEV)].cpu(), x.cpu(), None)["dweight"], 1, "dweight")


@pytest.mark.parametrize("rows,H,d", [(1_700_000, 10, 128), (3_400_000, 10, 64)])
def test_many_tokens(bss, rows, H, d):
    keys, group = 20, 850_001  # 2.2e9 elements of q
    G = -(-rows // group)
    q, k, v, do = rnd(rows, H, d), rnd(G, keys, H, d), rnd(G, keys, H, d), rnd(rows, H, d)
    O, lse, dq = torch.empty_like(q), torch.empty(H, rows, device=DEV), torch.empty_like(q)
    dk, dv = torch.empty_like(k), torch.empty_like(v)
    bss.cross_attention(q, k, v, O, lse=lse, rows_per_group=group)
    bss.cross_attention_backward(do, q, k, v, O, lse, dq, dk, dv, rows_per_group=group)
    torch.cuda.synchronize()
    assert bss.get_device_status() == 0
    n = 300  # the last rows, as a group of their own
    at, last = slice(rows - n, rows), slice(G - 1, G)
    part = [t.cpu() for t in (q[at], k[last], v[last])]
    ref = L.cross(*part, [keys], n)
    check(O[at], *ref["O"], 1, "O")
    check(lse[:, at], *ref["lse"], 1, "lse")
    ref = L.cross_grad(do[at].cpu(), *part, O[at].cpu(), lse[:, at].cpu(), [keys], n)
    check(dq[at], *ref["dq"], 1, "dq")
    assert torch.isfinite(dk).all() and torch.isfinite(dv).all()


@pytest.mark.parametrize("rows", [2, 40])
@pytest.mark.parametrize("layout", ["tokens", "heads"])
def test_many_states(bss, rows, layout):
    keys, H, d = 1_100_000, 16, 128  # 2.25e9 elements of K
    make = (lambda: rnd(1, keys, H, d)) if layout == "tokens" else (lambda: rnd(1, H, keys, d).transpose(1, 2))
    k, v = make(), make()
    q, do = rnd(rows, H, d), rnd(rows, H, d)
    O, lse, dq = torch.empty_like(q), torch.empty(H, rows, device=DEV), torch.empty_like(q)
    dk, dv = torch.empty_like(k), torch.empty_like(v)
    lengths = torch.tensor([keys - 5], dtype=torch.int32, device=DEV)
    bss.cross_attention(q, k, v, O, lengths=lengths, lse=lse)
    bss.cross_attention_backward(do, q, k, v, O, lse, dq, dk, dv, lengths=lengths)
    torch.cuda.synchronize()
    assert bss.get_device_status() == 0
    for h in (0, H - 1):
        one = slice(h, h + 1)
        part = [t.cpu() for t in (q[:, one], k[:, :, one], v[:, :, one])]
        ref = L.cross(*part, [keys - 5], rows)
        check(O[:, one], *ref["O"], 1, "O")
        check(lse[one], *ref["lse"], 1, "lse")
        ref = L.cross_grad(do[:, one].cpu(), *part, O[:, one].cpu(), lse[one].cpu(), [keys - 5], rows)
        check(dq[:, one], *ref["dq"], 1, "dq")
        check(dk[:, :, one], *ref["dk"], 1, "dk")
        check(dv[:, :, one], *ref["dv"], 1, "dv")

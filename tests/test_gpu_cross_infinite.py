"""cross_attention on the GPU where scores are minus infinity without being masked."""
import math

import pytest
import torch

import _layers_ref as L
from _block_ref import check
from test_gpu_cross import BF, DEV, rnd

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("rows,H", [(3, 2), (200, 2)])
@pytest.mark.parametrize("keys,first,length", [(300, 128, 300), (400, 130, 390), (700, 600, 601), (90, 40, 77)])
def test_finite_scores_behind_infinite_ones(bss, rows, H, d, keys, first, length):
    """The first states' scores are minus infinity, the others' far below 0 (about -150):
    their weights are those of the others alone."""
    g = torch.Generator().manual_seed(3)
    q = (rnd(g, rows, H, d).abs() + 0.5).to(BF)
    k = (rnd(g, 1, keys, H, d) - 120 * d ** -0.5).to(BF)
    v = rnd(g, 1, keys, H, d)
    ref = L.cross(q, k[:, first:], v[:, first:], [length - first], rows)
    k[:, :first] = -math.inf
    O, lse = torch.full_like(q, float("nan")).to(DEV), torch.full((H, rows), float("nan"), device=DEV)
    bss.cross_attention(q.to(DEV), k.to(DEV), v.to(DEV), O, lse=lse,
                        lengths=torch.tensor([length], dtype=torch.int32, device=DEV))
    torch.cuda.synchronize()
    assert bss.get_device_status() == 0
    check(lse, *ref["lse"], 1, "lse")
    check(O, *ref["O"], 1, "O")


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("rows,H", [(3, 2), (200, 2), (300, 3)])
@pytest.mark.parametrize("keys", [40, 200])
def test_rows_without_a_finite_score(bss, rows, H, d, keys):
    """A row whose scores all leave the float range downwards has O = 0 and lse = -inf, and
    brings nothing to a gradient; the other rows' and the states' gradients are theirs."""
    g = torch.Generator().manual_seed(4)
    q, k = (rnd(g, rows, H, d) * 1e-25).to(BF), ((rnd(g, 1, keys, H, d).abs() + 1) * -1e25).to(BF)
    v, do = rnd(g, 1, keys, H, d), rnd(g, rows, H, d)
    lost = [0, 2, rows - 1]
    q[lost] = (q[lost].float().abs() * 1e30 + 1e25).to(BF)
    qd, kd, vd, dod = (t.to(DEV) for t in (q, k, v, do))
    O, lse = torch.full_like(qd, float("nan")), torch.full((H, rows), float("nan"), device=DEV)
    bss.cross_attention(qd, kd, vd, O, lse=lse)
    assert (O[lost] == 0).all() and (lse[:, lost] == -math.inf).all()
    rest = [i for i in range(rows) if i not in lost]
    dq, dk, dv = (torch.full_like(t, float("nan")) for t in (qd, kd, vd))
    bss.cross_attention_backward(dod, qd, kd, vd, O, lse, dq, dk, dv)
    torch.cuda.synchronize()
    assert bss.get_device_status() == 0
    assert (dq[lost] == 0).all()
    if not rest:
        assert (dk == 0).all() and (dv == 0).all()
        return
    ref = L.cross(q[rest], k, v, [keys], len(rest))
    check(O[rest], *ref["O"], 1, "O")
    ref = L.cross_grad(do[rest], q[rest], k, v, O[rest].cpu(), lse[:, rest].cpu(), [keys], len(rest))
    # sums of as many rows as before: the ones left out are zeros
    for name, t in (("dq", dq[rest]), ("dk", dk), ("dv", dv)):
        check(t, *ref[name], 1, name)

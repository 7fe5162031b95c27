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

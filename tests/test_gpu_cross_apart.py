"""cross_attention on the GPU: a group's results have the same bits whatever the rows of
the group behind it hold, and whether or not these are being written over."""
import pytest
import torch

import _layers_ref as L
from _block_ref import check
from test_gpu_cross import BF, DEV, case

pytestmark = pytest.mark.gpu


def growing(rows, group, H, d, keys, scale=0.3):
    """Keys that grow along the states: a row of large queries moves its references in
    the later tiles, one of small queries does not."""
    q, k, v, group, G = case(rows, H, d, keys, group=group, scale=scale)
    return q, (k.float() * torch.linspace(0.01, 8, keys)[None, :, None, None]).to(BF), v, group, G


def call(bss, q, k, v, group, O=None):
    O = torch.full_like(q, float("nan")) if O is None else O
    lse = torch.full((q.shape[1], q.shape[0]), float("nan"), device=DEV)
    bss.cross_attention(q, k, v, O, lse=lse, rows_per_group=group)
    torch.cuda.synchronize()
    assert bss.get_device_status() == 0
    return O, lse


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("group", [1, 33, 100, 129, 200, 300])
def test_bits_do_not_depend_on_the_next_group(bss, group, d):
    H, keys = 4, 300
    rows = max(2 * group, 160)
    q, k, v, group, G = growing(rows, group, H, d, keys)
    small, k, v = q.to(DEV), k.to(DEV), v.to(DEV)
    O, lse = call(bss, small, k, v, group)
    at = torch.arange(rows, device=DEV) // group % 2 == 0  # every other group keeps its queries
    for content in (small * 30, torch.full_like(small, float("nan")), torch.full_like(small, 3e38)):
        other = torch.where(at[:, None, None], small, content)
        x, y = call(bss, other, k, v, group)
        assert torch.equal(x[at], O[at]) and torch.equal(y[:, at], lse[:, at])
    even = L.cross(q, k.cpu(), v.cpu(), [keys] * G, group)
    check(O, *even["O"], 1, "O")


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("rows,group,H,keys", [(700, 33, 10, 300), (5000, 300, 6, 300), (3001, 1000, 10, 513)])
def test_in_place_has_the_same_bits(bss, rows, group, H, keys, d):
    q, k, v, group, G = growing(rows, group, H, d, keys, scale=1.0)
    q, k, v = (t.to(DEV) for t in (q, k, v))
    O, lse = call(bss, q, k, v, group)
    for _ in range(5):
        over = q.clone()
        x, y = call(bss, over, k, v, group, O=over)
        assert torch.equal(x, O) and torch.equal(y, lse)

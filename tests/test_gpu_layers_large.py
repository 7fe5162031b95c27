"""The matrix products and the cross attention on the GPU at sizes whose CTAs take many
tiles or items each, one after another, and by pairs of CTAs."""
import pytest
import torch

import _layers_ref as L
import test_gpu_cross_grad as grad
from test_gpu_cross import DEV, case, run
from test_gpu_linear import BF, F32, backward, forward

pytestmark = pytest.mark.gpu

LENGTHS = [300, 0, 1, 128, 299, 129, 17, 256, 257, 77, 0, 300, 64, 200, 130]
# rows, group, heads, key heads: halves of 128 rows both there and not, groups smaller than a warp
MANY = [(20000, 1000, 8, 8), (12001, 300, 9, 3), (6005, 77, 8, 1), (700, 1, 2, 2), (1000, 3, 4, 2), (40001, 40001, 5, 5)]


def lengths_of(group, rows):
    return [LENGTHS[i % len(LENGTHS)] for i in range(-(-rows // group))]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("rows,group,H,Hk", MANY)
def test_cross_many_items(bss, rows, group, H, Hk, d):
    """More items than CTAs: several times as many, of all lengths, one behind another."""
    q, k, v, group, _ = case(rows, H, d, 300, group=group, Hk=Hk)
    first = run(bss, q, k, v, group, lengths_of(group, rows))
    again = run(bss, q, k, v, group, lengths_of(group, rows), in_place=True)
    assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_cross_many_items_whose_references_move(bss):
    q, k, v, group, _ = case(9000, 10, 64, 400, group=450)
    k = (k.float() * torch.linspace(0.01, 8, 400)[None, :, None, None]).to(BF)
    run(bss, q, k, v, group)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("rows,group,H,Hk", MANY)
def test_cross_backward_many_items(bss, rows, group, H, Hk, d):
    q, k, v, group, _ = case(rows, H, d, 300, group=group, Hk=Hk)
    grad.run(bss, q, k, v, group, lengths_of(group, rows), layout="packed")


@pytest.mark.parametrize("rows,group,H,Hk", [(1, 1, 3, 3), (8, 4, 4, 2), (16, 16, 2, 2)])
@pytest.mark.parametrize("keys", [31, 32, 33, 63, 64, 65, 127, 128, 129])
def test_cross_backward_few_rows_blocks_of_keys(bss, rows, group, H, Hk, keys):
    """Around the keys of a block of the kernel without tiles."""
    q, k, v, group, G = case(rows, H, 64, keys, group=group, Hk=Hk)
    grad.run(bss, q, k, v, group)
    grad.run(bss, q, k, v, group, [keys - 1] * G)


@pytest.mark.parametrize("out", [BF, F32])
@pytest.mark.parametrize("kind", [0, 1, 3])
def test_linear_by_pairs(bss, out, kind):
    """395 tiles of 256 x 256 for 76 pairs of CTAs, ragged at every end, with every part."""
    forward(bss, 20003, 72, 1032, kind=kind, out=out, pre=True, gate=True, residual=True, a=0.5, group=777, pad=8)


def test_linear_by_pairs_in_place_and_with_a_gate_a_row(bss):
    forward(bss, 20003, 72, 1032, residual=True, inplace=True)
    forward(bss, 20003, 72, 1032, out=F32, params=BF, gate=True, group=1, residual=True, inplace=True)


@pytest.mark.parametrize("rows,inner,outer", [(20003, 1032, 72),     # dx by pairs
                                              (70, 4104, 4104),      # dW by pairs
                                              (12001, 1288, 1288)])  # dW by pairs, two splits of the rows
def test_linear_backward_by_pairs(bss, rows, inner, outer):
    for dw in (BF, F32):
        backward(bss, rows, inner, outer, dw=dw, pad=8 if dw == BF else 0)


def test_linear_rows_beside_one_another(bss):
    """The last sizes without tiles and the first with them; whole tiles and one row more."""
    for rows in (16, 17, 128, 129, 256, 257, 1024, 1025):
        forward(bss, rows, 264, 136, kind=2, gate=True, group=5)
        backward(bss, rows, 264, 136, kind=2, gate=True, group=5)

"""cross_attention on the GPU against the 64-bit formulas: lengths from none to
several tiles, groups, shared heads, strides, masked states of any content."""
import math

import pytest
import torch

import _layers_ref as L
from _block_ref import check

DEV = "cuda"
BF = torch.bfloat16


def rnd(g, *s, scale=1.0):
    return (torch.randn(*s, generator=g) * scale).to(BF)


def case(rows, H, d, keys, group=None, Hk=None, seed=0, scale=1.5, k_scale=1.0):
    g = torch.Generator().manual_seed(seed)
    group = group or rows
    G, Hk = -(-rows // group), Hk or H
    return rnd(g, rows, H, d, scale=scale), rnd(g, G, keys, Hk, d, scale=k_scale), rnd(g, G, keys, Hk, d), group, G


def place(t, how):
    """The same values on the device in another layout."""
    t = t.to(DEV)
    if how == "packed":  # one tensor's slices, as a projection gives them
        wide = torch.full((*t.shape[:-2], 3, *t.shape[-2:]), float("nan"), dtype=t.dtype, device=DEV)
        wide[..., 1, :, :] = t
        return wide[..., 1, :, :]
    if how == "heads":  # head-major
        return t.transpose(-3, -2).contiguous().transpose(-3, -2)
    if how == "by_head":  # packed head by head
        wide = torch.full((*t.shape[:-1], 2, t.shape[-1]), float("nan"), dtype=t.dtype, device=DEV)
        wide[..., 1, :] = t
        return wide[..., 1, :]
    return t


def run(bss, q, k, v, group, lengths=None, layout="plain", scale=None, want_lse=True, in_place=False, poison=True):
    rows, H, d = q.shape
    G, keys = k.shape[:2]
    valid = [keys] * G if lengths is None else [min(max(n, 0), keys) for n in lengths]
    ref = L.cross(q, k, v, valid, group, scale)
    kd, vd = k.clone(), v.clone()
    if poison:  # what is masked is not looked at
        for i, n in enumerate(valid):
            kd[i, n:], vd[i, n:] = float("nan"), float("inf")
    qd = place(q, layout)
    O = qd if in_place else place(torch.full_like(q, float("nan")), layout)
    lse = torch.full((H, rows), float("nan"), device=DEV) if want_lse else None
    ln = None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device=DEV)
    bss.cross_attention(qd, place(kd, layout), place(vd, layout), O, lengths=ln, lse=lse, rows_per_group=group,
                        softmax_scale=scale)
    torch.cuda.synchronize()
    assert bss.get_device_status() == 0
    check(O, *ref["O"], 1, "O")
    if want_lse:
        value, slack = ref["lse"]
        empty = value == -math.inf
        assert (lse.cpu()[empty] == -math.inf).all()
        check(lse.cpu()[~empty], value[~empty], slack[~empty], 1, "lse")
    return O, lse


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("rows", [1, 2, 127, 128, 129, 256, 257, 700])
@pytest.mark.parametrize("keys", [1, 77, 129])
def test_rows(bss, rows, keys, d):
    run(bss, *case(rows, 2, d, keys)[:4])


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("keys", [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 95, 97, 112, 113, 127, 128, 129, 255, 256, 257, 383, 512, 1000])
def test_keys(bss, keys, d):
    run(bss, *case(150, 2, d, keys)[:4])


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
def test_lengths_of_padded_states(bss, d):
    lengths = [0, 1, 300, 15, 16, 17, 0, 128, 129, 256, 299, -5, 1000, 2]
    q, k, v, group, G = case(14 * 33 - 20, 3, d, 300, group=33)
    assert G == len(lengths)
    run(bss, q, k, v, group, lengths)
    run(bss, q, k, v, group, lengths[::-1], layout="packed", want_lse=False)


@pytest.mark.gpu
@pytest.mark.parametrize("lengths", [[0], [0, 0, 0], [0, 40, 0]])
def test_no_states(bss, lengths):
    q, k, v, group, _ = case(300 * len(lengths), 2, 64, 64, group=300)
    run(bss, q, k, v, group, lengths)


@pytest.mark.gpu
@pytest.mark.parametrize("group", [1, 3, 128, 200, 256, 300, 999])
def test_groups(bss, group):
    q, k, v, group, _ = case(1000 if group > 3 else 40, 2, 64, 40, group=group)
    run(bss, q, k, v, group)


@pytest.mark.gpu
@pytest.mark.parametrize("H,Hk", [(1, 1), (6, 2), (8, 1), (5, 5)])
@pytest.mark.parametrize("layout", ["plain", "packed", "heads", "by_head"])
def test_heads_and_layouts(bss, H, Hk, layout):
    q, k, v, group, _ = case(333, H, 64, 150, group=120, Hk=Hk)
    run(bss, q, k, v, group, [150, 70, 3], layout=layout)


@pytest.mark.gpu
def test_in_place_and_scale(bss):
    q, k, v, group, _ = case(700, 3, 128, 200, group=300)
    run(bss, q, k, v, group, layout="packed", in_place=True, scale=0.3)


@pytest.mark.gpu
def test_states_shared_by_groups(bss):
    q, k, v, group, G = case(500, 2, 64, 90, group=100)
    k, v = k[:1].expand(G, -1, -1, -1), v[:1].expand(G, -1, -1, -1)
    ref = L.cross(q, k, v, [90, 40, 0, 1, 90], group)
    O = torch.full_like(q, float("nan")).to(DEV)
    kd, vd = (t[:1].to(DEV).expand(G, -1, -1, -1) for t in (k, v))
    bss.cross_attention(q.to(DEV), kd, vd, O, lengths=torch.tensor([90, 40, 0, 1, 90], dtype=torch.int32, device=DEV),
                        rows_per_group=group)
    check(O, *ref["O"], 1, "O")


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
def test_scores_that_grow(bss, d):
    """Keys that grow along the states: references move in later tiles."""
    q, k, v, group, _ = case(400, 2, d, 600)
    k = (k.float() * torch.linspace(0.01, 8, 600)[None, :, None, None]).to(BF)
    run(bss, q, k, v, group)
    run(bss, q, k.flip(1).contiguous(), v, group)


@pytest.mark.gpu
def test_rows_stay_apart(bss):
    """NaN and infinities in one row of q, and in one group's states, stay there."""
    q, k, v, group, _ = case(600, 2, 64, 100, group=200)
    q[3, 0], q[250, 1] = float("nan"), float("inf")
    k[2, 5], v[2, 7] = float("nan"), float("inf")
    O = torch.empty_like(q).to(DEV)
    bss.cross_attention(q.to(DEV), k.to(DEV), v.to(DEV), O, rows_per_group=group)
    clean = q.clone()
    clean[3, 0], clean[250, 1] = 0, 0
    ref, slack = L.cross(clean[:400], k[:2], v[:2], [100, 100], group)["O"]
    good = torch.ones(400, 2, dtype=torch.bool)
    good[3, 0] = good[250, 1] = False
    check(O[:400].cpu()[good], ref[good], slack[good], 1, "O")
    assert torch.isnan(O[3, 0]).all() and torch.isnan(O[400:]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("rows,group,H,Hk,d,keys", [
    (1, 1, 1, 1, 64, 1), (1, 1, 10, 10, 128, 512), (1, 1, 6, 3, 128, 20), (5, 5, 4, 1, 64, 333), (8, 8, 2, 2, 128, 2048),
    (7, 2, 6, 2, 64, 33), (23, 8, 8, 1, 128, 63), (64, 1, 2, 2, 64, 129), (8, 8, 8, 8, 64, 4096), (16, 16, 2, 1, 64, 65)])
@pytest.mark.parametrize("layout", ["plain", "packed", "heads", "by_head"])
def test_few_rows(bss, rows, group, H, Hk, d, keys, layout):
    q, k, v, group, G = case(rows, H, d, keys, group=group, Hk=Hk)
    run(bss, q, k, v, group, layout=layout)
    run(bss, q, k, v, group, [(keys, 0, (keys + 1) // 2, 1, max(keys - 3, 0))[(i + 2) % 5] for i in range(G)], layout=layout,
        in_place=True)


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
def test_few_rows_in_32_bits(bss, d, monkeypatch):
    """A few rows' P is not rounded on the way: nothing but the result's own rounding."""
    monkeypatch.setattr(L, "BF16", 0)
    q, k, v, group, _ = case(6, 6, d, 75, group=2, Hk=3)
    run(bss, q, k, v, group, [75, 10, 1])
    run(bss, 8 * q, k, v, group, [75, 10, 1])


@pytest.mark.gpu
def test_few_rows_beside_tiles(bss):
    """The largest calls without tiles and the smallest with them."""
    for rows, keys in ((19, 64), (20, 64), (19, 300), (1, 5000)):
        q, k, v, group, _ = case(rows, 8, 64, keys, Hk=4)
        run(bss, q, k, v, group)


@pytest.mark.gpu
def test_few_rows_share_states(bss):
    """One set of states for all groups, by a group stride of 0."""
    q, k, v, _, _ = case(6, 2, 64, 70)
    O = torch.empty_like(q).to(DEV)
    kd, vd = (t.to(DEV).expand(3, -1, -1, -1) for t in (k, v))
    bss.cross_attention(q.to(DEV), kd, vd, O, rows_per_group=2)
    check(O, *L.cross(q, k, v, [70], 6)["O"], 1, "O")

"""cross_attention_backward on the GPU against the 64-bit formulas, from the O and
lse that the forward call wrote."""
import pytest
import torch

import _layers_ref as L
from _block_ref import check
from test_gpu_cross import BF, DEV, case, place, rnd

pytestmark = pytest.mark.gpu


def run(bss, q, k, v, group, lengths=None, layout="plain", scale=None, seed=9, workspace=None):
    rows, H, d = q.shape
    G, keys, Hk = k.shape[:3]
    valid = [keys] * G if lengths is None else [min(max(n, 0), keys) for n in lengths]
    do = rnd(torch.Generator().manual_seed(seed), rows, H, d)
    kd, vd = k.clone(), v.clone()
    for i, n in enumerate(valid):  # what is masked is not looked at
        kd[i, n:], vd[i, n:] = float("nan"), float("inf")
    ln = None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device=DEV)
    qd, kd, vd, dod = (place(t, layout) for t in (q, kd, vd, do))
    O, lse = torch.empty_like(q).to(DEV), torch.empty(H, rows, device=DEV)
    bss.cross_attention(qd, kd, vd, O, lengths=ln, lse=lse, rows_per_group=group, softmax_scale=scale)
    if layout == "packed":  # the gradients of k and v as views of one tensor
        dkv = torch.full((G, keys, 2, Hk, d), float("nan"), dtype=BF, device=DEV)
        dk, dv = dkv.unbind(2)
    else:
        dk, dv = (place(torch.full_like(k, float("nan")), layout) for _ in range(2))
    dq = place(torch.full_like(q, float("nan")), layout)
    bss.cross_attention_backward(dod, qd, kd, vd, O, lse, dq, dk, dv, lengths=ln, rows_per_group=group,
                                 softmax_scale=scale, workspace=workspace)
    torch.cuda.synchronize()
    assert bss.get_device_status() == 0
    ref = L.cross_grad(do, q, k, v, O.cpu(), lse.cpu(), valid, group, scale)
    for name, t in (("dq", dq), ("dk", dk), ("dv", dv)):
        check(t, *ref[name], 1, name)
    return dq, dk, dv


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("rows", [1, 2, 15, 17, 127, 128, 129, 257, 700])
@pytest.mark.parametrize("keys", [1, 77, 129])
def test_rows(bss, rows, keys, d):
    run(bss, *case(rows, 2, d, keys)[:4])


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("keys", [1, 15, 16, 17, 63, 64, 65, 80, 97, 127, 128, 129, 256, 257, 512, 700])
def test_keys(bss, keys, d):
    run(bss, *case(150, 2, d, keys)[:4])


@pytest.mark.parametrize("d", [64, 128])
def test_lengths_of_padded_states(bss, d):
    lengths = [0, 1, 300, 15, 16, 17, 0, 128, 129, 256, 299, -5, 1000, 2]
    q, k, v, group, G = case(14 * 33 - 20, 3, d, 300, group=33)
    run(bss, q, k, v, group, lengths)
    run(bss, q, k, v, group, lengths[::-1], layout="packed")


@pytest.mark.parametrize("lengths", [[0], [0, 0, 0], [0, 40, 0]])
def test_no_states(bss, lengths):
    q, k, v, group, _ = case(300 * len(lengths), 2, 64, 64, group=300)
    run(bss, q, k, v, group, lengths)


@pytest.mark.parametrize("group", [1, 3, 128, 200, 300, 999])
def test_groups(bss, group):
    q, k, v, group, _ = case(1000 if group > 3 else 40, 2, 64, 40, group=group)
    run(bss, q, k, v, group)


@pytest.mark.parametrize("H,Hk", [(1, 1), (6, 2), (8, 1), (5, 5)])
@pytest.mark.parametrize("layout", ["plain", "packed", "heads", "by_head"])
def test_heads_and_layouts(bss, H, Hk, layout):
    q, k, v, group, _ = case(333, H, 64, 150, group=120, Hk=Hk)
    run(bss, q, k, v, group, [150, 70, 3], layout=layout)


@pytest.mark.parametrize("d", [64, 128])
def test_long(bss, d):
    """More pairs of tiles than CTAs: runs that begin and end inside key tiles."""
    run(bss, *case(7000, 3, d, 200)[:4], scale=0.2)
    q, k, v, group, _ = case(9000, 2, d, 260, group=4000, Hk=1)
    run(bss, q, k, v, group, [260, 129, 30])


def test_more_key_tiles_than_ctas(bss):
    run(bss, *case(130, 1, 64, 20000)[:4])
    q, k, v, group, _ = case(40, 2, 64, 20100, group=20, Hk=1)
    run(bss, q, k, v, group, [20100, 300])


def test_same_bits_again(bss):
    a = case(5000, 2, 128, 200)[:4]
    for x, y in zip(run(bss, *a), run(bss, *a)):
        assert torch.equal(x.view(torch.int16), y.view(torch.int16))


def test_rows_stay_apart(bss):
    """NaN and infinities of one group's rows and states stay in it."""
    q, k, v, group, _ = case(300, 2, 64, 100, group=100)
    do = rnd(torch.Generator().manual_seed(2), 300, 2, 64)
    O, lse = torch.empty_like(q).to(DEV), torch.empty(2, 300, device=DEV)
    clean = [t.clone() for t in (do, q, k, v)]
    do[100, 0], q[101, 1], k[1, 5], v[1, 99] = float("nan"), float("inf"), float("nan"), float("inf")
    args = [t.to(DEV) for t in (do, q, k, v)]
    bss.cross_attention(*args[1:], O, lse=lse, rows_per_group=group)
    dq, dk, dv = torch.empty_like(O), *(torch.empty_like(args[2]) for _ in range(2))
    bss.cross_attention_backward(*args, O, lse, dq, dk, dv, rows_per_group=group)
    o = L.cross(*clean[1:], [100] * 3, group)
    for rows, g in ((slice(0, 100), 0), (slice(200, 300), 2)):
        part = [clean[0][rows], clean[1][rows], clean[2][g:g + 1], clean[3][g:g + 1]]
        check(O[rows], o["O"][0][rows], o["O"][1][rows], 1, "O")
        ref = L.cross_grad(*part, O[rows].cpu(), lse[:, rows].cpu(), [100], 100)
        check(dq[rows], *ref["dq"], 1, "dq")
        check(dk[g:g + 1], *ref["dk"], 1, "dk")
        check(dv[g:g + 1], *ref["dv"], 1, "dv")


@pytest.mark.parametrize("rows,group,H,Hk,d,keys", [
    (1, 1, 1, 1, 64, 1), (1, 1, 10, 10, 128, 512), (1, 1, 6, 3, 128, 20), (5, 5, 4, 1, 64, 333), (8, 8, 2, 2, 128, 2048),
    (7, 2, 6, 2, 64, 33), (23, 8, 8, 1, 128, 31), (64, 1, 2, 2, 64, 129), (8, 8, 8, 8, 64, 4096), (16, 16, 2, 1, 64, 40)])
@pytest.mark.parametrize("layout", ["plain", "packed", "heads", "by_head"])
def test_few_rows(bss, rows, group, H, Hk, d, keys, layout):
    q, k, v, group, G = case(rows, H, d, keys, group=group, Hk=Hk)
    run(bss, q, k, v, group, layout=layout)
    run(bss, q, k, v, group, [(keys, 0, (keys + 1) // 2, 1, max(keys - 3, 0))[(i + 2) % 5] for i in range(G)], layout=layout)


@pytest.mark.parametrize("d", [64, 128])
def test_few_rows_in_32_bits(bss, d, monkeypatch):
    """A few rows' P and dS are not rounded on the way: nothing but the results' own rounding."""
    monkeypatch.setattr(L, "BF16", 0)
    q, k, v, group, _ = case(6, 6, d, 75, group=2, Hk=3)
    run(bss, q, k, v, group, [75, 10, 1])


def test_few_rows_beside_tiles(bss):
    """The largest calls without tiles and the smallest with them."""
    for rows, keys in ((8, 2048), (8, 2049), (9, 64), (1, 5000)):
        q, k, v, group, _ = case(rows, 8, 64, keys, Hk=4)
        run(bss, q, k, v, group)

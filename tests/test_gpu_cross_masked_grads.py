"""cross_attention_backward on the GPU: masked states' gradients are zeros whatever the
rows hold."""
import pytest
import torch

from test_gpu_cross import DEV, case, rnd

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("rows,group,H,Hk,keys,lengths", [
    (6, 3, 2, 2, 75, [40, 0]),                    # few rows: no tiles
    (200, 100, 4, 2, 300, [140, 7]),              # a head's rows in one run
    (9000, 4000, 2, 1, 260, [200, 129, 30]),      # runs that end inside a head's rows
])
@pytest.mark.parametrize("what", ["dO", "q"])
def test_zeros_beside_infinite_rows(bss, rows, group, H, Hk, keys, lengths, d, what):
    q, k, v, group, G = case(rows, H, d, keys, group=group, Hk=Hk)
    do = rnd(torch.Generator().manual_seed(1), rows, H, d)
    bad = do if what == "dO" else q
    bad[0::997] = float("inf")
    bad[group - 1::group] = float("nan")
    q, k, v, do = (t.to(DEV) for t in (q, k, v, do))
    ln = torch.tensor(lengths, dtype=torch.int32, device=DEV)
    O, lse = torch.empty_like(q), torch.empty(H, rows, device=DEV)
    bss.cross_attention(q, k, v, O, lengths=ln, lse=lse, rows_per_group=group)
    dq, dk, dv = (torch.full_like(t, float("nan")) for t in (q, k, v))
    bss.cross_attention_backward(do, q, k, v, O, lse, dq, dk, dv, lengths=ln, rows_per_group=group)
    torch.cuda.synchronize()
    assert bss.get_device_status() == 0
    for i, n in enumerate(lengths):
        for name, t in (("dk", dk), ("dv", dv)):
            assert (t[i, n:] == 0).all(), (name, i)

"""attention_step_tokens refuses tensors of its two launches that overlap, before the first."""
import pytest
import torch

DEV = "cuda"


@pytest.mark.gpu
@pytest.mark.parametrize("permuted", [1, 0])
def test_step_refuses_overlapping_tensors(bss, permuted):
    H, d = 4, 64
    p = bss.MaskParams(2, 3, 5, d, 1, 2, temporal_permuted=permuted)
    N = p.N
    q = torch.randn(N, H, d, device=DEV).to(torch.bfloat16)
    O, *ws = (torch.full((H, N, d), -7.0, dtype=torch.bfloat16, device=DEV) for _ in range(4))
    fl = torch.tensor([1, 0, 0, 1], dtype=torch.uint8, device=DEV)
    floats = lambda t: t.view(-1)[:2 * H * N].view(torch.float32).view(H, N)  # noqa: E731
    bytes_ = lambda t: t.view(-1).view(torch.uint8)[64:64 + H]  # noqa: E731
    lse = torch.full((H, N), -7.0, device=DEV)
    keep = [t.clone() for t in (O, *ws, lse)]
    with bss.build_tile_map(p) as tm:
        calls = [(fl, [O, *ws], floats(t)) for t in (O, *ws)]                           # lse over a tensor
        calls += [(bytes_(t), [O, *ws], None) for t in (O, *ws)]                        # flags inside one
        calls += [(bytes_(lse), [O, *ws], lse)]
        calls += [(fl, [O, ws[0], ws[0], ws[2]], None), (fl, [O, O, ws[1], ws[2]], None)]
        for flags, (o, a, b, c), out in calls:
            with pytest.raises(bss.BssError) as e:
                bss.attention_step_tokens(q, q, q, o, tm, flags, a, b, c, lse=out)
            assert e.value.status == 1
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip((O, *ws, lse), keep))
        bss.attention_step_tokens(q, q, q, O, tm, fl, *ws, lse=lse)
        torch.cuda.synchronize()
    assert torch.isfinite(lse).all() and not torch.equal(O, keep[0])

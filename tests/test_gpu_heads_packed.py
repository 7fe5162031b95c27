"""heads_from_tokens on projections packed head by head, [N][H][3][d]: forward as
views of the packed projection, backward into views of one packed gradient."""
import pytest
import torch

DEV = "cuda"


@pytest.mark.gpu
@pytest.mark.parametrize("norm", [0, 1, 2])
@pytest.mark.parametrize("H,d", [(2, 128), (3, 64), (10, 128)])
def test_heads_packed_one_by_one(bss, H, d, norm):
    F, Hs, Ws = 3, 5, 7
    p = bss.MaskParams(F, Hs, Ws, d, 1, 1)
    N = p.N
    g = torch.Generator().manual_seed(H + norm)
    qkv = torch.randn(N, H, 3, d, generator=g).to(torch.bfloat16).to(DEV)
    w = (1 + 0.2 * torch.randn({0: 1, 1: d, 2: H * d}[norm], generator=g)).to(DEV) if norm else None
    fl = torch.randint(0, 2, (H,), generator=g, dtype=torch.uint8).to(DEV)
    kw = dict(q_weight=w, k_weight=w, norm=norm)
    apart = [t.contiguous() for t in qkv.unbind(2)]
    make = lambda: [torch.full((H, N, d), -7.0, dtype=torch.bfloat16, device=DEV) for _ in range(3)]  # noqa: E731
    got, want = make(), make()
    bss.heads_from_tokens(*qkv.unbind(2), *got, p, fl, **kw)
    bss.heads_from_tokens(*apart, *want, p, fl, **kw)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    grads = [torch.randn(H, N, d, generator=g).to(torch.bfloat16).to(DEV) for _ in range(3)]
    x = dict(q=apart[0], k=apart[1]) if norm else {}
    ref = [torch.full_like(t, -7.0) for t in apart]
    bss.heads_from_tokens_backward(*grads, *ref, p, fl, **x, **kw)
    # a fourth slot a head and rows around: left as they were; head by head, and tokens inside heads
    for shape, view in (((N + 2, H, 4, d), lambda b: b[1:-1]), ((H, N + 2, 4, d), lambda b: b[:, 1:-1].transpose(0, 1))):
        buf = torch.full(shape, -7.0, dtype=torch.bfloat16, device=DEV)
        dqkv = view(buf)
        bss.heads_from_tokens_backward(*grads, *(dqkv[:, :, i] for i in range(3)), p, fl, **x, **kw)
        torch.cuda.synchronize()
        assert all(torch.equal(dqkv[:, :, i], ref[i]) for i in range(3))
        assert torch.all(buf[:, :, 3] == -7.0)
        ends = (buf[0], buf[-1]) if shape[0] == N + 2 else (buf[:, 0], buf[:, -1])
        assert all(torch.all(t == -7.0) for t in ends)

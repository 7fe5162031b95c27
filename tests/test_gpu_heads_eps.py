"""heads_from_tokens with eps = 0: lanes without a piece of a head hold zeros,
whose root is infinite, and must leave no trace in the weights' gradients."""
import pytest
import torch

import _block_ref as R
from test_gpu_heads import DEV, K_GRAD, K_HEADS

F, Hs, Ws = 3, 5, 7
N, S = F * Hs * Ws, Hs * Ws


# Head counts that leave pieces of the last heads out (1, 3, 5, 17), that run an
# instance with more pieces than there are (8, 16) and that fill theirs (10).
@pytest.mark.gpu
@pytest.mark.parametrize("norm", [1, 2])
@pytest.mark.parametrize("H,d", [(1, 64), (1, 128), (3, 64), (5, 128), (8, 128), (10, 128), (16, 128), (17, 64)])
def test_weight_gradients_without_eps(bss, H, d, norm):
    g = torch.Generator().manual_seed(H)
    p = bss.MaskParams(F, Hs, Ws, d, 1, 1)
    x = [torch.randn(N, H, d, generator=g).to(torch.bfloat16) for _ in range(2)]
    dy = [torch.randn(H, N, d, generator=g).to(torch.bfloat16) for _ in range(2)]
    w = [1 + 0.3 * torch.randn(d if norm == 1 else H * d, generator=g) for _ in range(2)]
    flags = torch.randint(0, 2, (H,), generator=g, dtype=torch.uint8)
    X, W, D = ([t.to(DEV) for t in ts] for ts in (x, w, dy))
    kw = dict(q_weight=W[0], k_weight=W[1], norm=norm, eps=0.0)
    out = [torch.full((H, N, d), -7.0, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    bss.heads_from_tokens(*X, None, *out, None, p, flags.to(DEV), **kw)
    dx = [torch.full_like(t, -7.0) for t in X]
    dw = [torch.full_like(t, -7.0) for t in W]
    bss.heads_from_tokens_backward(*D, None, *dx, None, p, flags.to(DEV), q=X[0], k=X[1], dq_weight=dw[0],
                                   dk_weight=dw[1], **kw)
    torch.cuda.synchronize()
    for i in range(2):
        R.check(out[i], *R.heads(x[i].double(), w[i], norm, 0.0, None, False, flags, F, S), K_HEADS, "heads")
        ref, mag, rw, rwmag = R.heads_grad(dy[i].double(), x[i].double(), w[i], norm, 0.0, None, False, flags, F, S)
        R.check(dx[i], ref, mag, K_GRAD, "dx")
        # 48 roundings of a term; at most 105 tokens and 5 heads a lane in a row, 32 lanes' sums after them
        R.check(dw[i], rw, rwmag, 300, "dw")

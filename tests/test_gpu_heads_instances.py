"""The forms of heads_from_tokens under the norm over a token that share a token
between 2, 4, 6 and 8 warps or hold 2 and 6 to 8 pieces a lane, both ways, and
the gradients of zero tokens and of heads that share their input."""
import pytest
import torch

import _block_ref as R
import test_gpu_heads as T

DEV = T.DEV

# F, Hs, Ws, H, d, channels per axis, halves, norm, layout, weights.  Odd token
# counts: the tokens that go side by side in a block of two warps a token end unevenly.
MORE = {
    "two_warps": (3, 5, 7, 3, 128, (44, 42, 42), False, 2, "packed", torch.float32),
    "two_warps_full": (3, 3, 5, 4, 128, (32, 48, 48), True, 2, "split", torch.bfloat16),
    "two_warps_d64": (1, 1, 7, 7, 64, (16, 16, 16), True, 2, "heads", torch.float32),
    "four_warps": (3, 5, 7, 8, 128, (44, 42, 42), False, 2, "split", torch.float32),
    "six_warps": (2, 5, 7, 12, 128, (32, 48, 48), True, 2, "packed", torch.bfloat16),
    "eight_warps": (2, 3, 7, 14, 128, (44, 42, 42), False, 2, "heads", torch.float32),
    "sixteen_heads": (2, 3, 5, 16, 128, (32, 48, 48), True, 2, "packed", torch.float32),
    "two_pieces": (2, 3, 7, 20, 128, (44, 42, 42), False, 2, "packed", torch.bfloat16),
    "two_pieces_halves": (2, 3, 7, 31, 64, (16, 24, 24), True, 2, "split", "none"),
}
T.CASES.update(MORE)  # Case looks them up by name; the tests there keep their own list


@pytest.mark.gpu
@pytest.mark.parametrize("name", MORE)
def test_forward(bss, name):
    T.test_forward(bss, name)


@pytest.mark.gpu
@pytest.mark.parametrize("name", MORE)
def test_backward(bss, name):
    T.test_backward(bss, name)


@pytest.mark.gpu
@pytest.mark.parametrize("name", ["token_norm", "head_norm_halves", "two_warps"])
def test_zero_tokens_have_no_part_in_the_gradients(bss, name):
    """Tokens of zeros (padding) add nothing to the weights' gradients, and their own are finite."""
    c = T.Case(bss, name)
    g = torch.Generator().manual_seed(5)
    dy = torch.randn(c.H, c.N, c.d, generator=g).to(torch.bfloat16)
    for rows in (torch.arange(c.N), torch.arange(0, c.N, 3)):
        x = c.tokens[0].clone()
        x[rows] = 0.0
        dx = torch.full((c.N, c.H, c.d), -7.0, dtype=torch.bfloat16, device=DEV)
        dw = torch.full((c.weights[0].numel(),), -7.0, device=DEV)
        bss.heads_from_tokens_backward(dy.to(DEV), None, None, dx, None, None, c.p, c.fl, **c.kw, q=x.to(DEV), dq_weight=dw)
        ref, mag, rw, rwmag = R.heads_grad(dy.double(), x.double(), c.weights[0], c.norm, c.eps, c.ang, c.halves,
                                           c.flags, c.F, c.S)
        R.check(dx, ref, mag, T.K_GRAD, "dx")
        R.check(dw, rw, rwmag, 300, "dw")
        if len(rows) == c.N:
            assert torch.all(dw == 0)


@pytest.mark.gpu
def test_gradient_of_a_shared_head_comes_a_head_each(bss):
    """One K head read by every head (stride 0): dK is written head by head, the caller sums them."""
    c = T.Case(bss, "head_norm_halves")
    shared = c.dev[1][:, :1].expand(c.N, c.H, c.d)
    g = torch.Generator().manual_seed(6)
    dy = torch.randn(c.H, c.N, c.d, generator=g).to(torch.bfloat16)
    dk = torch.full((c.N, c.H, c.d), -7.0, dtype=torch.bfloat16, device=DEV)
    dw = torch.full((c.d,), -7.0, device=DEV)
    bss.heads_from_tokens_backward(None, dy.to(DEV), None, None, dk, None, c.p, c.fl, **c.kw, k=shared, dk_weight=dw)
    ref, mag, rw, rwmag = R.heads_grad(dy.double(), shared.cpu().double(), c.weights[1], c.norm, c.eps, c.ang, c.halves,
                                       c.flags, c.F, c.S)
    R.check(dk, ref, mag, T.K_GRAD, "dk")
    R.check(dw, rw, rwmag, 300, "dw")

"""The gradient formulas of the layers' 64-bit references against differences."""
import pytest
import torch

import _layers_ref as L

H = 1e-6


def difference(f, t):
    """df/dt of a scalar function, element by element."""
    out = torch.zeros_like(t)
    flat, o = t.view(-1), out.view(-1)
    for i in range(flat.numel()):
        keep = flat[i].item()
        flat[i] = keep + H
        up = f()
        flat[i] = keep - H
        down = f()
        flat[i] = keep
        o[i] = (up - down) / (2 * H)
    return out


@pytest.mark.parametrize("kind", [0, 1, 2, 3])
@pytest.mark.parametrize("gated", [False, True])
def test_linear_gradients(kind, gated):
    g = torch.Generator().manual_seed(kind)
    r = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    x, w, b, d = r(5, 3), r(4, 3), r(4), r(5, 4)
    gate = r(3, 4) if gated else None
    f = lambda: (L.linear(x, w, b, kind, gate, None, 2)["out"][0] * d).sum()  # noqa: E731
    got = L.linear_grad(d, x, w, L.linear(x, w, b)["pre"][0], kind, gate, 2)
    for name, t in (("dx", x), ("dweight", w), ("dbias", b)) + ((("dgate", gate),) if gated else ()):
        assert torch.allclose(got[name][0], difference(f, t), atol=1e-7), name


@pytest.mark.parametrize("H,Hk,lengths", [(2, 2, [3, 0]), (4, 2, [2, 3]), (3, 1, [1, 3])])
def test_cross_gradients(H, Hk, lengths):
    g = torch.Generator().manual_seed(H)
    r = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    q, k, v, do = r(5, H, 4), r(2, 3, Hk, 4), r(2, 3, Hk, 4), r(5, H, 4)
    f = lambda: (L.cross(q, k, v, lengths, 3)["O"][0] * do).sum()  # noqa: E731
    o = L.cross(q, k, v, lengths, 3)
    got = L.cross_grad(do, q, k, v, o["O"][0], o["lse"][0], lengths, 3)
    for name, t in (("dq", q), ("dk", k), ("dv", v)):
        assert torch.allclose(got[name][0], difference(f, t), atol=1e-7), name

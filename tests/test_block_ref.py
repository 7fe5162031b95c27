"""The 64-bit references of the operators around the attention step: their
gradient formulas against differences of their forward forms, on the CPU."""
import pytest
import torch

import _block_ref as R


def differences(f, x, g, eps=1e-6):
    """Gradient of sum(f(x) g) by central differences."""
    out = torch.zeros_like(x)
    flat, o = x.view(-1), out.view(-1)
    for i in range(flat.numel()):
        keep = flat[i].item()
        flat[i] = keep + eps
        hi = (f(x) * g).sum()
        flat[i] = keep - eps
        lo = (f(x) * g).sum()
        flat[i] = keep
        o[i] = (hi - lo) / (2 * eps)
    return out


def near(a, b):
    assert (a - b).abs().max() <= 1e-7 * (1 + b.abs().max()), (a - b).abs().max()


@pytest.mark.parametrize("norm", [0, 1, 2])
@pytest.mark.parametrize("halves", [False, True])
def test_heads_gradient_formula(norm, halves):
    F, Hs, Ws, H, d = 2, 1, 3, 2, 32
    N = F * Hs * Ws
    g = torch.Generator().manual_seed(norm)
    x, dy = (torch.randn(s, generator=g, dtype=torch.float64) for s in ((N, H, d), (H, N, d)))
    w = None if norm == 0 else torch.randn(d if norm == 1 else H * d, generator=g, dtype=torch.float64)
    tabs = [R.table(6, p) for p in (4, 2, 2)]
    ang = R.angles(tabs, (1, 2, 0), F, Hs, Ws)

    def f(x, w):
        return R.heads(x, w, norm, 1e-3, ang, halves, [0, 1], F, Hs * Ws)[0]
    dx, _, dw, _ = R.heads_grad(dy, x, w, norm, 1e-3, ang, halves, [0, 1], F, Hs * Ws)
    near(dx, differences(lambda t: f(t, w), x, dy))
    if norm:
        near(dw, differences(lambda t: f(x, t), w, dy))


@pytest.mark.parametrize("norm,y_norm", [(1, 0), (1, 1), (2, 2), (0, 1), (2, 0)])
def test_residual_norm_gradient_formula(norm, y_norm):
    rows, C, group, a = 5, 8, 2, 0.7
    g = torch.Generator().manual_seed(10 * norm + y_norm)
    rnd = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    v = dict(x=rnd(rows, C), y=rnd(rows, C), gate=rnd(3, C), scale=rnd(3, C), shift=rnd(3, C), weight=rnd(C),
             bias=rnd(C), y_weight=rnd(C))
    dr, dh = rnd(rows, C), rnd(rows, C)
    kw = dict(norm=norm, y_norm=y_norm, group=group, a=a)
    o = R.residual_norm(eps=1e-3, **v, **kw)
    got = R.residual_norm_grad(o["r"], v["y"], dr, dh, torch.cat((o["mean"], o["rstd"]), 1),
                               torch.cat((o["ymean"], o["yrstd"]), 1), v["gate"], v["scale"], v["weight"], v["bias"],
                               v["y_weight"], **kw)
    names = {"x": "dx", "y": "dy", "gate": "dgate", "scale": "dscale", "shift": "dshift", "weight": "dweight",
             "bias": "dbias", "y_weight": "dy_weight"}
    for k, name in names.items():
        def f(t, k=k):
            o = R.residual_norm(eps=1e-3, **{**v, k: t}, **kw)
            return torch.cat((o["r"], o["h"]), 1)
        near(got[name][0], differences(f, v[k], torch.cat((dr, dh), 1)))

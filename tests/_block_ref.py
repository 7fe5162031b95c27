"""Plain 64-bit references of the operators around the attention step, with the
magnitude of each result's terms (what 32-bit roundings are relative to).

A stored value may be off by one rounding to its type, torch.finfo(t).eps / 2
relative, plus K roundings of 2^-24 of its terms' magnitude; K counts the longest
chain of 32-bit operations behind a value (sums of n terms add log2 n in a tree,
n in a row)."""
import torch

HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
U32 = 2.0 ** -24



def check(got, ref, mag, K, what=""):
    """got (as stored) against ref: one rounding to its type and K 32-bit ones of mag."""
    half = HALF[got.dtype]
    got, ref, mag = got.double().cpu(), ref.double().cpu(), mag.double().cpu()
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    slack = K * U32 * mag
    over = (got - ref).abs() - (half * (ref.abs() + slack) + slack)
    worst = over.max().item() if over.numel() else 0.0
    assert torch.isfinite(got).all(), f"{what}: not finite"
    assert worst <= 0.0, f"{what}: {int((over > 0).sum())} of {over.numel()} values off, worst by {worst:.3g}"


# ---------------------------------------------------------------- heads

def table(length, pairs, base=10000.0):
    i = torch.arange(pairs, dtype=torch.float64)
    a = torch.arange(length, dtype=torch.float64)[:, None] * base ** (-i / max(pairs, 1))
    return torch.stack((a.cos(), a.sin()), -1).float()


def pair_channels(R, halves):
    p = torch.arange(R // 2)
    return (p, p + R // 2) if halves else (2 * p, 2 * p + 1)


def angles(tables, offset, F, Hs, Ws):
    """(cos, sin) [N][pairs] in 64 bits."""
    n = torch.arange(F * Hs * Ws)
    pos = (n // (Hs * Ws), n // Ws % Hs, n % Ws)
    t = torch.cat([tab.double().cpu()[p + o] for tab, p, o in zip(tables, pos, offset)], 1)
    return t[..., 0], t[..., 1]


def rows_of(F, S, temporal):
    """Output row of every token."""
    n = torch.arange(F * S)
    return n % S * F + n // S if temporal else n


def rms(x, norm, eps):
    """1 / deviation of [N][H][d] (norm 1: a head, 2: a token)."""
    dims = (2,) if norm == 1 else (1, 2)
    return (x.square().mean(dims, keepdim=True) + eps).rsqrt()


def heads(x, w, norm, eps, ang, halves, flags, F, S):
    """[N][H][d] float64 -> ([H][N][d], magnitude); ang None: no rotation."""
    N, H, d = x.shape
    y = x
    if norm:
        y = x * rms(x, norm, eps)
        if w is not None:
            y = y * w.double().view(-1, d)
    mag = y.abs()
    if ang is not None:
        cos, sin = (t[:, None] for t in ang)
        a, b = pair_channels(2 * cos.shape[-1], halves)
        out, mag = y.clone(), mag.clone()
        out[..., a] = y[..., a] * cos - y[..., b] * sin
        out[..., b] = y[..., a] * sin + y[..., b] * cos
        both = y[..., a].abs() + y[..., b].abs()
        mag[..., a] = both
        mag[..., b] = both
        y = out
    res, rmag = torch.empty(H, N, d, dtype=torch.float64), torch.empty(H, N, d, dtype=torch.float64)
    for h in range(H):
        row = rows_of(F, S, bool(flags[h]))
        res[h, row] = y[:, h]
        rmag[h, row] = mag[:, h]
    return res, rmag


def heads_grad(dy, x, w, norm, eps, ang, halves, flags, F, S):
    """Gradient of ``heads``: (dx, its magnitude, dw, its magnitude); dw None without a norm."""
    H, N, d = dy.shape
    g = torch.empty(N, H, d, dtype=torch.float64)
    for h in range(H):
        g[:, h] = dy[h, rows_of(F, S, bool(flags[h]))]
    gm = g.abs()
    if ang is not None:
        cos, sin = (t[:, None] for t in ang)
        a, b = pair_channels(2 * cos.shape[-1], halves)
        out, gm = g.clone(), gm.clone()
        out[..., a] = g[..., a] * cos + g[..., b] * sin
        out[..., b] = g[..., b] * cos - g[..., a] * sin
        both = g[..., a].abs() + g[..., b].abs()
        gm[..., a] = both
        gm[..., b] = both
        g = out
    if not norm:
        return g, gm, None, None
    r = rms(x, norm, eps)
    W = torch.ones(1, d, dtype=torch.float64) if w is None else w.double().view(-1, d)
    dims = (2,) if norm == 1 else (1, 2)
    dx = r * (g * W - x * r * r * (g * W * x).mean(dims, keepdim=True))
    mag = r * (gm * W.abs() + x.abs() * r * r * (gm * W.abs() * x.abs()).mean(dims, keepdim=True))
    over = (0, 1) if norm == 1 else (0,)
    return dx, mag, (g * x * r).sum(over).reshape(-1), (gm * x.abs() * r).sum(over).reshape(-1)


# ---------------------------------------------------------------- norm, gate and residual

def statistics(x, kind, eps):
    """(mean, 1 / deviation), [rows][1] each; kind 0: (0, 1)."""
    zero = torch.zeros(x.shape[0], 1, dtype=torch.float64)
    if kind == 0:
        return zero, zero + 1.0
    mean = x.mean(1, keepdim=True) if kind == 1 else zero
    return mean, ((x - mean).square().mean(1, keepdim=True) + eps).rsqrt()


def per_row(m, rows, group):
    return m.double()[torch.arange(rows) // group]


def residual_norm(x, y=None, gate=None, scale=None, shift=None, weight=None, bias=None, y_weight=None, norm=1, y_norm=0,
                  group=None, a=1.0, eps=1e-6):
    """Everything in float64.  Returns r, h, their magnitudes and the statistics."""
    rows = x.shape[0]
    group = rows if group is None else group
    r, rmag = x.double(), x.double().abs()
    ymean, yrstd = (None, None)
    if y is not None:
        y = y.double()
        ymean, yrstd = statistics(y, y_norm, eps)
        f = torch.ones(1, 1, dtype=torch.float64)
        if y_weight is not None:
            f = f * y_weight.double()
        if gate is not None:
            f = f * per_row(gate, rows, group)
        r = a * r + (y - ymean) * yrstd * f
        rmag = abs(a) * rmag + (y.abs() + ymean.abs()) * yrstd * f.abs()
    mean, rstd = statistics(r, norm, eps)
    # the mean of the magnitudes stands for what the mean and the deviation inherit
    h, hmag = (r - mean) * rstd, (rmag + rmag.mean(1, keepdim=True)) * rstd
    if norm:
        hmag = hmag + h.abs() * hmag.mean(1, keepdim=True)
    if weight is not None:
        h, hmag = h * weight.double(), hmag * weight.double().abs()
    if bias is not None:
        h, hmag = h + bias.double(), hmag + bias.double().abs()
    if scale is not None:
        s = per_row(scale, rows, group)
        h, hmag = h * (1 + s), hmag * (1 + s.abs())
    if shift is not None:
        s = per_row(shift, rows, group)
        h, hmag = h + s, hmag + s.abs()
    return {"r": r, "rmag": rmag, "h": h, "hmag": hmag, "mean": mean, "rstd": rstd, "ymean": ymean, "yrstd": yrstd}


def group_sums(t, group):
    rows = t.shape[0]
    G = -(-rows // group)
    out = torch.zeros(G, t.shape[1], dtype=torch.float64)
    return out.index_add_(0, torch.arange(rows) // group, t)


def residual_norm_grad(r, y=None, dr=None, dh=None, stats=None, y_stats=None, gate=None, scale=None, weight=None,
                       bias=None, y_weight=None, norm=1, y_norm=0, group=None, a=1.0):
    """Formula of the gradients in float64, from the statistics given:
    {name: (value, magnitude)}."""
    some = r if r is not None else dr
    rows, C = some.shape
    group = rows if group is None else group
    one, zero = torch.ones(rows, C, dtype=torch.float64), torch.zeros(rows, C, dtype=torch.float64)
    out = {}
    u, um = (zero, zero) if dr is None else (dr.double(), dr.double().abs())
    if dh is not None:
        dh, r = dh.double(), r.double()
        mean, rstd = (zero[:, :1], one[:, :1]) if norm == 0 else (stats.double()[:, :1], stats.double()[:, 1:])
        xh, xm = (r - mean) * rstd, (r.abs() + mean.abs()) * rstd
        w = one if weight is None else one * weight.double()
        b = zero if bias is None else zero + bias.double()
        m = one if scale is None else 1 + per_row(scale, rows, group)
        mm = one if scale is None else 1 + per_row(scale, rows, group).abs()
        out["dscale"] = group_sums(dh * (xh * w + b), group), group_sums(dh.abs() * (xm * w.abs() + b.abs()), group)
        out["dshift"] = group_sums(dh, group), group_sums(dh.abs(), group)
        out["dweight"] = (dh * m * xh).sum(0), (dh.abs() * mm * xm).sum(0)
        out["dbias"] = (dh * m).sum(0), (dh.abs() * mm).sum(0)
        t, tm = dh * m * w, dh.abs() * mm * w.abs()
        m1 = t.mean(1, keepdim=True) if norm == 1 else zero[:, :1]
        m2 = (t * xh).mean(1, keepdim=True) if norm else zero[:, :1]
        u = u + rstd * (t - m1 - xh * m2)
        um = um + rstd * (tm + (tm.mean(1, keepdim=True) if norm == 1 else 0)
                          + (xm * (tm * xm).mean(1, keepdim=True) if norm else 0))
    out["dx"] = a * u, abs(a) * um
    if y is None:
        return out
    y = y.double()
    ymean, yrstd = (zero[:, :1], one[:, :1]) if y_norm == 0 else (y_stats.double()[:, :1], y_stats.double()[:, 1:])
    yh, ym = (y - ymean) * yrstd, (y.abs() + ymean.abs()) * yrstd
    wy = one if y_weight is None else one * y_weight.double()
    gt = one if gate is None else per_row(gate, rows, group)
    out["dgate"] = group_sums(u * yh * wy, group), group_sums(um * ym * wy.abs(), group)
    out["dy_weight"] = (u * yh * gt).sum(0), (um * ym * gt.abs()).sum(0)
    z, zm = u * gt * wy, um * gt.abs() * wy.abs()
    if y_norm:
        m1 = z.mean(1, keepdim=True) if y_norm == 1 else zero[:, :1]
        m2 = (z * yh).mean(1, keepdim=True)
        out["dy"] = (yrstd * (z - m1 - yh * m2),
                     yrstd * (zm + (zm.mean(1, keepdim=True) if y_norm == 1 else 0) + ym * (zm * ym).mean(1, keepdim=True)))
    else:
        out["dy"] = z, zm
    return out

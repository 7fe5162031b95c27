"""Plain 64-bit references of the matrix products and the cross attention, with the
magnitude of each result's terms, for ``_block_ref.check``.

Roundings counted (in units of 2^-24 of the terms' magnitude):
  a tensor core's sum of k products: every 16 of k the running sum is cut to 24
  bits (one unit of its last place, 2 of 2^-24): 2 * k / 16, and 4 for the ends;
  a tensor rounded to bf16 on the way (half a step, 2^-8): BF16 = 2^16;
  an activation: exp of u (fast form: 2 + 1.2 |u| units in the last place, |u| its
  own rounding) and a fast quotient: |u| < 90 where the value is not 0 to 1e-38,
  so ACT = 512 covers value and slope."""
import math

import torch

BF16 = 2 ** 16
ACT = 512


def chain(k):
    return 2 * (k / 16 + 4)


def act(z, kind):
    """Value and slope of ACT_* in 64 bits (z float64)."""
    if kind == 1:
        # (1 + tanh u) / 2 = sigmoid(2 u): where the left side cancels (z < -6) it keeps
        # no more than 1e-16 absolute in 64 bits, above a 32-bit rounding of values of 1e-10
        c = 2 * math.sqrt(2 / math.pi)
        s = torch.sigmoid(c * (z + 0.044715 * z ** 3))
        return z * s, s + z * s * (1 - s) * c * (1 + 3 * 0.044715 * z * z)
    if kind == 2:
        half = 0.5 * torch.erfc(-z / math.sqrt(2))
        return z * half, half + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    if kind == 3:
        s = torch.sigmoid(z)
        return z * s, s * (1 + z * (1 - s))
    return z, torch.ones_like(z)


def per_row(m, rows, group):
    return m.double()[torch.arange(rows) // group]


def linear(x, w, bias=None, kind=0, gate=None, residual=None, group=None, a=1.0):
    """{name: (value, magnitude)} of out and pre; magnitudes hold CHAIN units of the product."""
    x, w = x.double(), w.double()
    rows = x.shape[0]
    z, zm = x @ w.t(), x.abs() @ w.abs().t()
    if bias is not None:
        z, zm = z + bias.double(), zm + bias.double().abs()
    v, _ = act(z, kind)
    # slopes are at most 1.13
    k = chain(x.shape[1]) + 4
    vm = 1.13 * k * zm + (ACT if kind else 1) * v.abs()
    if gate is not None:
        g = per_row(gate, rows, group)
        v, vm = v * g, (vm + v.abs()) * g.abs()
    if residual is not None:
        v, vm = v + a * residual.double(), vm + 4 * (v.abs() + abs(a) * residual.double().abs())
    return {"out": (v, vm), "pre": (z, k * zm)}


def group_sums(t, group):
    rows = t.shape[0]
    return torch.stack([t[i:i + group].sum(0) for i in range(0, rows, group)])


def linear_grad(dout, x, w, pre=None, kind=0, gate=None, group=None):
    """{name: (value, slack in units of 2^-24)}."""
    d = dout.double()
    rows = d.shape[0]
    z = torch.zeros_like(d) if pre is None else pre.double()
    v, s = act(z, kind)
    out = {}
    g = torch.ones_like(d)
    if gate is not None:
        g = per_row(gate, rows, group)
        chain_g = ACT + 2 * group + 32
        out["dgate"] = group_sums(d * v, group), chain_g * group_sums((d * v).abs(), group)
    dz = d * g * s
    # a slope is a difference of terms of at most 1.2
    dzm = (d * g).abs() * (s.abs() if kind == 0 else torch.full_like(s, 1.2))
    cut = 0 if kind == 0 and gate is None and dout.dtype == torch.bfloat16 else BF16
    out["dbias"] = dz.sum(0), (ACT + rows + 32) * dzm.sum(0)
    if w is not None:
        out["dx"] = dz @ w.double(), (cut + ACT + chain(d.shape[1])) * (dzm @ w.double().abs())
    if x is not None:
        out["dweight"] = dz.t() @ x.double(), (cut + ACT + chain(rows)) * (dzm.t() @ x.double().abs())
    return out


# ---------------------------------------------------------------- cross attention

def cross(q, k, v, lengths, group, scale=None):
    """O and lse with their slacks, q [rows][H][d], k, v [groups][keys][Hk][d], in units of 2^-24.

    A score is off by chain(d) units of its terms and 8 of itself (the scale, the
    reference and the exponential's argument), its weight by as many relative ones, 4
    of the exponential and a rounding to bf16 on the way to the product."""
    q, k, v = q.double(), k.double(), v.double()
    rows, H, d = q.shape
    Hk = k.shape[2]
    scale = d ** -0.5 if scale is None else scale
    O, Om = torch.zeros_like(q), torch.zeros_like(q)
    lse = torch.full((H, rows), -math.inf, dtype=torch.float64)
    lm = torch.zeros_like(lse)
    for i, n in enumerate(lengths):
        at = slice(i * group, min((i + 1) * group, rows))
        n = min(max(n, 0), k.shape[1])
        if n == 0:
            continue
        for h in range(H):
            kk, vv = k[i, :n, h * Hk // H], v[i, :n, h * Hk // H]
            s = q[at, h] @ kk.t() * scale
            off = (chain(d) * (q[at, h].abs() @ kk.abs().t()) * scale + 8 * s.abs()).amax(1, keepdim=True)
            top = s.amax(1, keepdim=True)
            p = (s - top).exp()
            l = p.sum(1, keepdim=True)
            O[at, h] = p @ vv / l
            Om[at, h] = (BF16 + 2 * off + 16 + chain(n) + n / 2) * (p @ vv.abs()) / l
            lse[h, at] = (top + l.log())[:, 0]
            lm[h, at] = (off + 8 * (top.abs() + l.log()) + 16 + n / 2)[:, 0]
    return {"O": (O, Om), "lse": (lse, lm)}


def cross_grad(do, q, k, v, O, lse, lengths, group, scale=None):
    """{name: (value, slack in units of 2^-24)} of dq, dk, dv; O and lse as a forward pass kept them.

    P is off as in ``cross``, with lse's own rounding; dS by P's, by its terms' chains
    and by a rounding to bf16 on the way to the products."""
    do, q, k, v, O, lse = (t.double() for t in (do, q, k, v, O, lse))
    rows, H, d = q.shape
    Hk = k.shape[2]
    scale = d ** -0.5 if scale is None else scale
    out = {n: (torch.zeros_like(t), torch.zeros_like(t)) for n, t in (("dq", q), ("dk", k), ("dv", v))}
    for i, n in enumerate(lengths):
        at = slice(i * group, min((i + 1) * group, rows))
        m = at.stop - at.start
        n = min(max(n, 0), k.shape[1])
        if n == 0:
            continue
        for h in range(H):
            j = h * Hk // H
            qq, kk, vv, g = q[at, h], k[i, :n, j], v[i, :n, j], do[at, h]
            s = qq @ kk.t() * scale
            off = chain(d) * (qq.abs() @ kk.abs().t()) * scale + 8 * (s.abs() + lse[h, at, None].abs()) + 16
            p = (s - lse[h, at, None]).exp()
            D = (g * O[at, h]).sum(1, keepdim=True)
            dp = g @ vv.t()
            ds = p * (dp - D)
            dse = p * ((BF16 + off) * (dp - D).abs() + chain(d) * (g.abs() @ vv.abs().t())
                       + d * (g * O[at, h]).abs().sum(1, keepdim=True))
            pe = p * (BF16 + off)
            for name, to, value, slack in (
                    ("dq", (at, h), scale * ds @ kk, scale * ((dse + chain(n) * ds.abs()) @ kk.abs())),
                    ("dk", (i, slice(0, n), j), scale * ds.t() @ qq, scale * ((dse + (chain(m) + H) * ds.abs()).t() @ qq.abs())),
                    ("dv", (i, slice(0, n), j), p.t() @ g, (pe + (chain(m) + H) * p).t() @ g.abs())):
                out[name][0][to] += value
                out[name][1][to] += slack
    return out

"""The operators around the attention step of a video transformer's block, as
measured cases: the norm, gate and residual update of the token stream
(``residual_norm``), and the turn from the projections' token-major Q, K, V to
the attention step's heads (``heads_from_tokens``: Q/K norm, rotary positions
of the (time, height, width) axes, head-major layout with the temporal heads in
(H,W,F) order), each with its backward pass.

``own`` False computes them in plain torch operations in 32 bits; True calls
the library.
"""
import math

import torch

own = False

EPS = 1e-6
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------- the cases

def _heads(name, op, F, Hs, Ws, H, d, axes, pairing, norm, temporal, layout="packed", at=(0, 0, 0), params="f32"):
    return {"name": name, "op": op, "F": F, "Hs": Hs, "Ws": Ws, "H": H, "d": d, "at": axes[0], "ah": axes[1],
            "aw": axes[2], "pairing": pairing, "norm": norm, "temporal": temporal, "layout": layout, "t0": at[0],
            "h0": at[1], "w0": at[2], "params": params}


def _norm(name, op, rows, channels, group, stream, branch, params, norm, y_norm, residual=True, modulated=True,
          affine=False, residual_scale=1.0):
    return {"name": name, "op": op, "rows": rows, "channels": channels, "group": group, "stream": stream,
            "branch": branch, "params": params, "norm": norm, "y_norm": y_norm, "residual": residual,
            "modulated": modulated, "affine": affine, "residual_scale": residual_scale}


def listed():
    return [
        # one token's heads at a position of its own: the call's latency
        _heads("heads_one_token", "heads", 1, 1, 1, 10, 128, (44, 42, 42), "interleaved", "token", 0, "split",
               (20, 44, 79)),
        # a short odd clip, 64 channels a head, part of them rotated
        _heads("heads_odd_clip", "heads", 5, 9, 13, 5, 64, (16, 16, 16), "halves", "head", 2, "split", (0, 0, 0), "bf16"),
        # the attention benchmark's mixed workload, from one packed projection
        _heads("heads_75k", "heads", 21, 45, 80, 10, 128, (44, 42, 42), "interleaved", "token", 5),
        # its 1440p form
        _heads("heads_1440p", "heads", 21, 90, 160, 10, 128, (32, 48, 48), "halves", "head", 5, "split"),
        # training: the gradients of the mixed workload, and of a small odd clip
        _heads("heads_bwd_75k", "heads_backward", 21, 45, 80, 10, 128, (44, 42, 42), "interleaved", "token", 5),
        _heads("heads_bwd_odd", "heads_backward", 7, 11, 13, 3, 64, (24, 20, 20), "interleaved", "head", 1, "split"),
        # one token through the norm in front of a block: the call's latency
        _norm("norm_one_token", "norm", 1, 1280, 1, "bf16", "bf16", "bf16", "layer", "none", residual=False),
        # between two blocks: gate, residual and the next block's modulated norm, modulations a frame
        _norm("norm_75k", "norm", 75600, 1280, 3600, "bf16", "bf16", "f32", "layer", "none"),
        # a block normed on both sides on a 32-bit stream, learned weights
        _norm("norm_sandwich_75k", "norm", 75600, 1280, 75600, "f32", "bf16", "f32", "rms", "rms", modulated=False,
              affine=True, residual_scale=0.5),
        # training: modulations a frame; odd sizes with every part; one set of modulations for a long clip
        _norm("norm_bwd_75k", "norm_backward", 75600, 1280, 3600, "bf16", "bf16", "f32", "layer", "none"),
        _norm("norm_bwd_odd", "norm_backward", 1001, 1000, 77, "f32", "bf16", "bf16", "rms", "layer", affine=True),
        _norm("norm_bwd_1440p", "norm_backward", 302400, 1280, 302400, "bf16", "bf16", "f32", "rms", "rms", affine=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    most = 302400 * 1280
    if rng.random() < 0.5:
        d, H = rng.choice((64, 128)), rng.randint(1, 16)
        F, Hs, Ws = rng.randint(1, 21), _log(rng, 1, 90), _log(rng, 1, 160)
        while F * Hs * Ws * H * d > most * 3 // 4:
            H -= 1
        pairing = rng.choice(("interleaved", "halves"))
        rotated = rng.choice((d, d, d - 16))
        a = 2 * rng.randint(d // 8, rotated // 5)
        c = _heads("", rng.choice(("heads", "heads_backward")), F, Hs, Ws, H, d, (rotated - 2 * a, a, a), pairing,
                   rng.choice(("none", "head", "token")), rng.randint(0, H), rng.choice(("packed", "split", "heads")),
                   (rng.randint(0, 40), rng.randint(0, 3), rng.randint(0, 3)), rng.choice(("f32", "bf16")))
    else:
        channels, rows = 8 * _log(rng, 8, 320), _log(rng, 1, 302400)
        rows = min(rows, most // channels)
        residual = rng.random() < 0.75
        stream, branch = rng.choice((("bf16", "bf16"), ("f32", "bf16"), ("f32", "f32")))
        if stream == "f32":
            rows = (rows + 1) // 2
        c = _norm("", rng.choice(("norm", "norm_backward")), rows, channels, max(1, rows // rng.choice((1, 1, 3, 21))),
                  stream, branch, rng.choice(("f32", "bf16")), rng.choice(("layer", "rms")),
                  rng.choice(("none", "layer", "rms")) if residual else "none", residual, rng.random() < 0.7,
                  rng.random() < 0.5, rng.choice((1.0, 0.5)) if residual else 1.0)
    del c["name"]
    return c


# ---------------------------------------------------------------- inputs

def _randn(g, *shape, dtype=torch.float32, scale=1.0, mean=0.0):
    x = torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)
    return x.mul_(scale).add_(mean).to(dtype)


def _table(length, pairs):
    """(cos, sin) of positions 0 .. length - 1, float32 from 64 bits."""
    i = torch.arange(pairs, dtype=torch.float64, device="cuda")
    a = torch.arange(length, dtype=torch.float64, device="cuda")[:, None] * 10000.0 ** (-i / max(pairs, 1))
    return torch.stack((a.cos(), a.sin()), -1).float().contiguous()


def _token_major(g, c, fill=True):
    """q, k, v as [N][H][d] views of the case's layout: one packed projection
    output, three outputs, or heads already apart."""
    N, H, d = c["F"] * c["Hs"] * c["Ws"], c["H"], c["d"]
    make = (lambda *s: _randn(g, *s, dtype=torch.bfloat16, scale=1.5)) if fill else \
        (lambda *s: torch.empty(*s, device="cuda", dtype=torch.bfloat16))
    if c["layout"] == "packed":
        return list(make(N, 3, H, d).unbind(1))
    if c["layout"] == "split":
        return [make(N, H, d) for _ in range(3)]
    return [make(H, N, d).transpose(0, 1) for _ in range(3)]


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": c}
    pd = DTYPES[c["params"]]
    if c["op"].startswith("heads"):
        H, d = c["H"], c["d"]
        N = c["F"] * c["Hs"] * c["Ws"]
        s["q"], s["k"], s["v"] = _token_major(g, c)
        width = {"none": 0, "head": d, "token": H * d}[c["norm"]]
        s["q_weight"], s["k_weight"] = (_randn(g, width, dtype=pd, scale=0.2, mean=1.0) if width else None
                                        for _ in range(2))
        order = torch.randperm(H, generator=torch.Generator().manual_seed(seed)).tolist()
        flags = torch.zeros(H, dtype=torch.uint8)
        flags[order[:c["temporal"]]] = 1
        s["flags"] = flags.cuda()
        s["tables"] = [_table(off + n, a // 2) for off, n, a in
                       ((c["t0"], c["F"], c["at"]), (c["h0"], c["Hs"], c["ah"]), (c["w0"], c["Ws"], c["aw"]))]
        if c["op"] == "heads":
            s["out"] = [torch.empty(H, N, d, device="cuda", dtype=torch.bfloat16) for _ in range(3)]
        else:
            s["grad"] = [_randn(g, H, N, d, dtype=torch.bfloat16) for _ in range(3)]
            s["out"] = _token_major(g, c, fill=False)
            s["dweight"] = [torch.empty(width, device="cuda") if width else None for _ in range(2)]
        return s
    rows, C, sd, bd = c["rows"], c["channels"], DTYPES[c["stream"]], DTYPES[c["branch"]]
    G = -(-rows // c["group"])
    # a stream whose channels have means and sizes of their own
    size, mean = _randn(g, C, scale=0.3).exp_(), _randn(g, C, scale=0.5)
    stream = _randn(g, rows, C).mul_(size).add_(mean)
    s["y"] = _randn(g, rows, C, dtype=bd, scale=1.5) if c["residual"] else None
    mod = _randn(g, G, 3, C, dtype=pd, scale=0.3)
    s["gate"] = mod[:, 0] if c["residual"] and c["modulated"] else None
    s["scale"], s["shift"] = (mod[:, 1], mod[:, 2]) if c["modulated"] else (None, None)
    s["weight"] = _randn(g, C, dtype=pd, scale=0.2, mean=1.0) if c["affine"] else None
    s["bias"] = _randn(g, C, dtype=pd, scale=0.2) if c["affine"] and c["norm"] == "layer" else None
    s["y_weight"] = _randn(g, C, dtype=pd, scale=0.2, mean=1.0) if c["affine"] and c["y_norm"] != "none" else None
    x = s["x"] = stream.to(sd)
    del stream
    if c["op"] == "norm":
        s["r"] = torch.empty(rows, C, device="cuda", dtype=sd) if c["residual"] else None
        s["h"] = torch.empty(rows, C, device="cuda", dtype=bd)
        return s
    # backward: x stands for the updated stream that the forward pass wrote, with the statistics it kept
    s["dh"] = _randn(g, rows, C, dtype=bd)
    s["dr"] = _randn(g, rows, C, dtype=sd) if c["residual"] else None
    s["stats"] = _statistics(x, c["norm"])
    s["y_stats"] = _statistics(s["y"], c["y_norm"]) if c["y_norm"] != "none" else None
    s["dx"] = torch.empty(rows, C, device="cuda", dtype=sd)
    s["dy"] = torch.empty(rows, C, device="cuda", dtype=bd) if c["residual"] else None
    for k in ("gate", "scale", "shift"):
        s["d" + k] = torch.empty(G, C, device="cuda") if s[k] is not None else None
    for k in ("weight", "bias", "y_weight"):
        s["d" + k] = torch.empty(C, device="cuda") if s[k] is not None else None
    return s


def _statistics(x, norm):
    """(mean, 1 / deviation) of each row, as a forward pass keeps them."""
    mean = x.double().mean(1) if norm == "layer" else torch.zeros(x.shape[0], dtype=torch.float64, device=x.device)
    var = (x.double() - mean[:, None]).square_().mean(1)
    return torch.stack((mean, (var + EPS).rsqrt()), 1).float()


# ---------------------------------------------------------------- plain forms

def _angles(s):
    """(cos, sin) of every token, [N][1][pairs]."""
    c = s["case"]
    n = torch.arange(c["F"] * c["Hs"] * c["Ws"], device="cuda")
    pos = (n // (c["Hs"] * c["Ws"]) + c["t0"], n // c["Ws"] % c["Hs"] + c["h0"], n % c["Ws"] + c["w0"])
    t = torch.cat([tab[p] for tab, p in zip(s["tables"], pos)], 1)
    return t[:, None, :, 0], t[:, None, :, 1]


def _pairs(x, c):
    rotated = c["at"] + c["ah"] + c["aw"]
    if c["pairing"] == "halves":
        return x[..., :rotated // 2], x[..., rotated // 2:rotated]
    return x[..., 0:rotated:2], x[..., 1:rotated:2]


def _rotated(x, cos, sin, c):
    out = x.clone()
    (a, b), (oa, ob) = _pairs(x, c), _pairs(out, c)
    oa.copy_(a * cos - b * sin)
    ob.copy_(a * sin + b * cos)
    return out


def _layout(x, s, inverse=False):
    """[N][H][d] -> [H][N][d], flagged heads in (H,W,F) order; inverse: back."""
    c = s["case"]
    F, S = c["F"], c["Hs"] * c["Ws"]
    n = torch.arange(F * S, device="cuda")
    flagged = s["flags"].bool()[:, None, None]
    if not inverse:
        x = x.transpose(0, 1)
        return torch.where(flagged, x[:, n % F * S + n // F], x)
    return torch.where(flagged, x[:, n % S * F + n // S], x).transpose(0, 1)


def _rms(x, c):
    dims = (1, 2) if c["norm"] == "token" else (2,)
    return (x.square().mean(dims, keepdim=True) + EPS).rsqrt()


def _weight(w, c):
    return w.float().view(-1, c["d"])


def _heads_plain(s):
    c = s["case"]
    cos, sin = _angles(s)
    out = []
    for x, w in ((s["q"], s["q_weight"]), (s["k"], s["k_weight"])):
        x = x.float()
        if w is not None:
            x = x * _rms(x, c) * _weight(w, c)
        out.append(_layout(_rotated(x, cos, sin, c), s).to(torch.bfloat16))
    return out + [_layout(s["v"], s)]


def _heads_backward_plain(s):
    c = s["case"]
    cos, sin = _angles(s)
    out, dws = [], []
    for x, w, dy in ((s["q"], s["q_weight"], s["grad"][0]), (s["k"], s["k_weight"], s["grad"][1])):
        g = _rotated(_layout(dy.float(), s, True), cos, -sin, c)
        if w is not None:
            x = x.float()
            r = _rms(x, c)
            n = g * x * r
            dws.append(n.sum(0).view(-1) if c["norm"] == "token" else n.sum((0, 1)))
            g = g * _weight(w, c)
            dims = (1, 2) if c["norm"] == "token" else (2,)
            g = r * (g - x * r * r * (g * x).mean(dims, keepdim=True))
        out.append(g.to(torch.bfloat16))
    return out + [_layout(s["grad"][2], s, True)] + dws


def _rows_of(m, c):
    """A group's values for each of its rows."""
    return m.float().repeat_interleave(c["group"], 0)[:c["rows"]]


def _normed(x, norm):
    if norm == "layer":
        x = x - x.mean(1, keepdim=True)
    return x * (x.square().mean(1, keepdim=True) + EPS).rsqrt()


def _norm_plain(s):
    c = s["case"]
    r = s["x"].float()
    if s["y"] is not None:
        y = s["y"].float()
        if c["y_norm"] != "none":
            y = _normed(y, c["y_norm"])
        if s["y_weight"] is not None:
            y = y * s["y_weight"].float()
        if s["gate"] is not None:
            y = y * _rows_of(s["gate"], c)
        r = c["residual_scale"] * r + y
    h = _normed(r, c["norm"])
    if s["weight"] is not None:
        h = h * s["weight"].float()
    if s["bias"] is not None:
        h = h + s["bias"].float()
    if s["scale"] is not None:
        h = h * (1 + _rows_of(s["scale"], c)) + _rows_of(s["shift"], c)
    out = [h.to(DTYPES[c["branch"]])]
    return out + [r.to(DTYPES[c["stream"]])] if s["y"] is not None else out


def _group_sum(x, c):
    G = -(-c["rows"] // c["group"])
    if G * c["group"] != c["rows"]:
        x = torch.cat((x, x.new_zeros(G * c["group"] - c["rows"], x.shape[1])))
    return x.view(G, c["group"], -1).sum(1)


def _through_norm(t, xh, rstd, norm):
    u = t - xh * (t * xh).mean(1, keepdim=True)
    return rstd * (u - t.mean(1, keepdim=True) if norm == "layer" else u)


def _norm_backward_plain(s):
    c, out = s["case"], {}
    dh, stats = s["dh"].float(), s["stats"]
    xh = (s["x"].float() - stats[:, :1]) * stats[:, 1:]
    n = xh if s["weight"] is None else xh * s["weight"].float()
    n = n if s["bias"] is None else n + s["bias"].float()
    t = dh
    if s["scale"] is not None:
        out["dscale"], out["dshift"] = _group_sum(dh * n, c), _group_sum(dh, c)
        t = dh * (1 + _rows_of(s["scale"], c))
    if s["weight"] is not None:
        out["dweight"] = (t * xh).sum(0)
    if s["bias"] is not None:
        out["dbias"] = t.sum(0)
    if s["weight"] is not None:
        t = t * s["weight"].float()
    u = _through_norm(t, xh, stats[:, 1:], c["norm"])
    if s["y"] is None:
        out["dx"] = u.to(DTYPES[c["stream"]])
        return out
    u = u + s["dr"].float()
    out["dx"] = (c["residual_scale"] * u).to(DTYPES[c["stream"]])
    yh = s["y"].float()
    if c["y_norm"] != "none":
        yh = (yh - s["y_stats"][:, :1]) * s["y_stats"][:, 1:]
    z = u
    if s["gate"] is not None:
        out["dgate"] = _group_sum(u * (yh if s["y_weight"] is None else yh * s["y_weight"].float()), c)
        z = u * _rows_of(s["gate"], c)
    if s["y_weight"] is not None:
        out["dy_weight"] = (z * yh).sum(0)
        z = z * s["y_weight"].float()
    if c["y_norm"] != "none":
        z = _through_norm(z, yh, s["y_stats"][:, 1:], c["y_norm"])
    out["dy"] = z.to(DTYPES[c["branch"]])
    return out


# ---------------------------------------------------------------- the library's calls

def _own(s):
    import block_sparse_spatio_gb300 as bss
    c = s["case"]
    if c["op"].startswith("heads"):
        p = bss.MaskParams(c["F"], c["Hs"], c["Ws"], c["d"], 0, 0)
        rot = bss.Rotary(*s["tables"], offset=(c["t0"], c["h0"], c["w0"]),
                         pairing=bss.PAIR_HALVES if c["pairing"] == "halves" else bss.PAIR_INTERLEAVED)
        norm = {"none": bss.HEAD_NORM_NONE, "head": bss.HEAD_NORM_HEAD, "token": bss.HEAD_NORM_TOKEN}[c["norm"]]
        if c["op"] == "heads":
            bss.heads_from_tokens(s["q"], s["k"], s["v"], *s["out"], p, s["flags"], rotary=rot,
                                  q_weight=s["q_weight"], k_weight=s["k_weight"], norm=norm, eps=EPS)
            return s["out"]
        bss.heads_from_tokens_backward(*s["grad"], *s["out"], p, s["flags"], rotary=rot, q=s["q"], k=s["k"],
                                       q_weight=s["q_weight"], k_weight=s["k_weight"], dq_weight=s["dweight"][0],
                                       dk_weight=s["dweight"][1], norm=norm, eps=EPS)
        return s["out"] + [w for w in s["dweight"] if w is not None]
    kind = {"none": bss.NORM_NONE, "layer": bss.NORM_LAYER, "rms": bss.NORM_RMS}
    if c["op"] == "norm":
        bss.residual_norm(s["x"], s["y"], r=s["r"], h=s["h"], gate=s["gate"], scale=s["scale"], shift=s["shift"],
                          weight=s["weight"], bias=s["bias"], y_weight=s["y_weight"], norm=kind[c["norm"]],
                          y_norm=kind[c["y_norm"]], rows_per_group=c["group"], residual_scale=c["residual_scale"],
                          eps=EPS)
        return [s["h"]] + ([s["r"]] if s["r"] is not None else [])
    grads = {k: s[k] for k in ("dx", "dy", "dgate", "dscale", "dshift", "dweight", "dbias", "dy_weight")}
    bss.residual_norm_backward(s["x"], s["y"], dr=s["dr"], dh=s["dh"], stats=s["stats"], y_stats=s["y_stats"],
                               gate=s["gate"], scale=s["scale"], weight=s["weight"], bias=s["bias"],
                               y_weight=s["y_weight"], norm=kind[c["norm"]], y_norm=kind[c["y_norm"]],
                               rows_per_group=c["group"], residual_scale=c["residual_scale"], **grads)
    return {k: t for k, t in grads.items() if t is not None}


def run(state):
    if own:
        return _own(state)
    return {"heads": _heads_plain, "heads_backward": _heads_backward_plain, "norm": _norm_plain,
            "norm_backward": _norm_backward_plain}[state["case"]["op"]](state)


def work(case):
    """Each input read once, each output written once."""
    c = case
    width = {"bf16": 2, "f32": 4}
    if c["op"].startswith("heads"):
        n = c["F"] * c["Hs"] * c["Ws"] * c["H"] * c["d"]
        tensors = 6 if c["op"] == "heads" else 6 + (2 if c["norm"] != "none" else 0)
        return {"bytes": 2 * tensors * n, "flops": (20 if c["op"] == "heads" else 40) * n}
    n = c["rows"] * c["channels"]
    small = 3 * -(-c["rows"] // c["group"]) * c["channels"] * width[c["params"]] if c["modulated"] else 0
    per = (width[c["stream"]] + width[c["branch"]]) * (2 if c["residual"] else 1)
    if c["op"] == "norm_backward":  # reads the stream, y, dr and dh; writes dx and dy
        per = (3 * width[c["stream"]] + 3 * width[c["branch"]]) if c["residual"] else \
            2 * width[c["stream"]] + width[c["branch"]]
        small *= 2
    return {"bytes": per * n + small, "flops": (12 if c["op"] == "norm" else 30) * n}


# ---------------------------------------------------------------- the definition, in 64 bits

def _exact_heads(s, x, w, rotate=True):
    """One tensor's heads by complex products, token by token of each head's own order."""
    c = s["case"]
    F, Hs, Ws, H, d = (c[k] for k in ("F", "Hs", "Ws", "H", "d"))
    if w is not None and c["norm"] == "head":
        x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / d + EPS) * w
    elif w is not None:
        flat = x.flatten(1)
        x = (flat / torch.sqrt((flat * flat).sum(-1, keepdim=True) / (H * d) + EPS) * w).view_as(x)
    grid = x.reshape(F, Hs, Ws, H, d)
    if rotate:
        t, h, w_ = (torch.view_as_complex(tab.double()) for tab in s["tables"])
        turn = torch.cat((t[c["t0"]:c["t0"] + F, None, None].expand(F, Hs, Ws, -1),
                          h[None, c["h0"]:c["h0"] + Hs, None].expand(F, Hs, Ws, -1),
                          w_[None, None, c["w0"]:c["w0"] + Ws].expand(F, Hs, Ws, -1)), -1)[..., None, :]
        R = 2 * turn.shape[-1]
        if c["pairing"] == "halves":
            z = torch.complex(grid[..., :R // 2], grid[..., R // 2:R]) * turn
            grid = torch.cat((z.real, z.imag, grid[..., R:]), -1)
        else:
            z = torch.complex(grid[..., 0:R:2], grid[..., 1:R:2]) * turn
            grid = torch.cat((torch.view_as_real(z).flatten(-2), grid[..., R:]), -1)
    spatial = grid.permute(3, 0, 1, 2, 4).reshape(H, -1, d)
    temporal = grid.permute(3, 1, 2, 0, 4).reshape(H, -1, d)
    pick = s["flags"].double()[:, None, None]
    return temporal * pick + spatial * (1 - pick)


def _exact_normed(x, kind):
    if kind == "none":
        return x
    var, mean = torch.var_mean(x, 1, correction=0, keepdim=True)
    return (x - mean) / torch.sqrt(var + EPS) if kind == "layer" else x / torch.sqrt(var + mean * mean + EPS)


def _exact_rows(m, c):
    return m[torch.arange(c["rows"], device="cuda") // c["group"]]


def _exact_parts(s, r, v):
    """The branch's part of the update, and the normed output of a stream r."""
    c = s["case"]
    part = None
    if v.get("y") is not None:
        part = _exact_normed(v["y"], c["y_norm"])
        part = part if v.get("y_weight") is None else part * v["y_weight"]
        part = part if v.get("gate") is None else part * _exact_rows(v["gate"], c)
    stream = r(part)
    h = _exact_normed(stream, c["norm"])
    h = h if v.get("weight") is None else h * v["weight"]
    h = h if v.get("bias") is None else h + v["bias"]
    if v.get("scale") is not None:
        h = h + h * _exact_rows(v["scale"], c) + _exact_rows(v["shift"], c)
    return stream, h


def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    if c["op"].startswith("heads"):
        names = ("q", "k", "v")
        leaf = [s[k].double().requires_grad_() for k in names]
        ws = [None if s[k + "_weight"] is None else s[k + "_weight"].double().requires_grad_() for k in ("q", "k")]
        if c["op"] == "heads":
            with torch.no_grad():
                return [_exact_heads(s, x, w, rot) for x, w, rot in zip(leaf, ws + [None], (True, True, False))]
        grads, dws = [], []
        for i in range(3):
            w = ws[i] if i < 2 else None
            out = _exact_heads(s, leaf[i], w, i < 2)
            got = torch.autograd.grad(out, [leaf[i]] + ([w] if w is not None else []), s["grad"][i].double())
            grads.append(got[0])
            dws += list(got[1:])
        return grads + dws
    keys = ("y", "gate", "scale", "shift", "weight", "bias", "y_weight")
    v = {k: s[k].double().requires_grad_() for k in keys if s[k] is not None}
    x = s["x"].double().requires_grad_()
    if c["op"] == "norm":
        with torch.no_grad():
            r, h = _exact_parts(s, lambda part: x if part is None else c["residual_scale"] * x + part, v)
        return [h, r] if s["y"] is not None else [h]
    # the gradient at the stream x that the update gave: x + what changes of it
    move = torch.zeros_like(x).requires_grad_()
    r, h = _exact_parts(s, lambda part: x.detach() + c["residual_scale"] * move + (0 if part is None else part - part.detach()), v)
    outs, gs = [h], [s["dh"].double()]
    if s["dr"] is not None:
        outs, gs = outs + [r], gs + [s["dr"].double()]
    got = torch.autograd.grad(outs, [move] + list(v.values()), gs)
    return dict(zip(["dx"] + ["d" + k for k in v], got))

"""The matrix products and the cross attention of a video transformer's block, as
measured cases: a linear layer with bias, activation, gate and residual in its
epilogue (``linear``), and attention of the video's tokens over an encoder's
states of another length (``cross_attention``), each with its backward pass.

``own`` False computes them in plain torch operations in 32 bits; True calls
the library.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------- the cases

def _linear(name, op, rows, inner, outer, activation="none", bias=True, gate=False, residual=False, group=0, out="bf16",
            params="f32", keep=False):
    return {"name": name, "op": op, "rows": rows, "inner": inner, "outer": outer, "activation": activation, "bias": bias,
            "gate": gate, "residual": residual, "group": group or rows, "out": out, "params": params, "keep": keep}


def _cross(name, op, rows, heads, d, keys, group=0, kv_heads=0, lengths="full", layout="packed", keep=False):
    return {"name": name, "op": op, "rows": rows, "heads": heads, "kv_heads": kv_heads or heads, "d": d, "keys": keys,
            "group": group or rows, "lengths": lengths, "layout": layout, "keep": keep}


def listed():
    return [
        # a time step's six modulations of one sample, in 32 bits: the call's latency
        _linear("linear_one_row", "linear", 1, 1280, 7680, out="f32"),
        # an encoder's 512 states brought to the block's width
        _linear("linear_context", "linear", 512, 4096, 1280, "gelu_tanh"),
        # odd sizes with every part, the pre-activation kept for a backward pass
        _linear("linear_odd", "linear", 1001, 1000, 1288, "silu", gate=True, residual=True, group=77, params="bf16", keep=True),
        # the feed-forward layers of the attention benchmark's 75,600 tokens: up with the activation,
        # down with a gate a frame and the residual
        _linear("linear_up_75k", "linear", 75600, 1280, 5120, "gelu_tanh"),
        _linear("linear_down_75k", "linear", 75600, 5120, 1280, gate=True, residual=True, group=3600),
        # training: the gradients of the layer up, and of an odd gated one
        _linear("linear_bwd_75k", "linear_backward", 75600, 1280, 5120, "gelu_tanh"),
        _linear("linear_bwd_odd", "linear_backward", 1001, 1000, 1288, "none", gate=True, group=77, params="bf16"),
        # one token over a prompt: the call's latency
        _cross("cross_one_token", "cross", 1, 10, 128, 512),
        # 75,600 tokens over a padded prompt of 512 states
        _cross("cross_75k", "cross", 75600, 10, 128, 512, keep=True),
        # a prompt a piece of the clip: short ragged prompts (none and one state among them), shared key heads
        _cross("cross_pieces_odd", "cross", 16001, 12, 64, 77, group=3001, kv_heads=4, lengths="ragged", layout="split"),
        # training: the gradients of both
        _cross("cross_bwd_75k", "cross_backward", 75600, 10, 128, 512),
        _cross("cross_bwd_odd", "cross_backward", 5003, 6, 64, 333, group=1250, kv_heads=2, lengths="ragged", layout="split"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    if rng.random() < 0.5:
        rows, inner, outer = _log(rng, 1, 75600), 8 * _log(rng, 8, 640), 8 * _log(rng, 8, 640)
        rows = min(rows, 75600 * 1280 * 5120 // (inner * outer))
        op = rng.choice(("linear", "linear_backward"))
        gate = rng.random() < 0.4
        c = _linear("", op, rows, inner, outer, rng.choice(("none", "gelu_tanh", "gelu", "silu")), rng.random() < 0.8, gate,
                    op == "linear" and rng.random() < 0.4, max(1, rows // rng.choice((1, 1, 3, 21))),
                    "f32" if op == "linear" and rows <= 16 else "bf16", rng.choice(("f32", "bf16")), rng.random() < 0.3)
    else:
        d, kv_heads, rows, keys = rng.choice((64, 128)), rng.randint(1, 10), _log(rng, 1, 75600), _log(rng, 1, 2048)
        heads = kv_heads * rng.choice((1, 1, 2, 4))
        rows = max(1, min(rows, 75600 * 10 * 512 // (heads * keys), 75600 * 10 // heads))
        c = _cross("", rng.choice(("cross", "cross_backward")), rows, heads, d, keys, max(1, rows // rng.choice((1, 1, 2, 7))),
                   kv_heads, rng.choice(("full", "ragged")), rng.choice(("packed", "split")), rng.random() < 0.5)
    del c["name"]
    return c


def _groups(c):
    return -(-c["rows"] // c["group"])


def _lengths(c):
    """The valid keys of each group."""
    n = c["keys"]
    if c["lengths"] == "full":
        return [n] * _groups(c)
    return [((n + 1) // 2, n, 1, 0, max(n - 3, 0))[i % 5] for i in range(_groups(c))]


# ---------------------------------------------------------------- inputs

def _randn(g, *shape, dtype=torch.float32, scale=1.0):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32).mul_(scale).to(dtype)


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda").manual_seed(seed)
    bf = torch.bfloat16
    s = {"case": c}
    rows = c["rows"]
    if c["op"].startswith("linear"):
        K, N, pd, G = c["inner"], c["outer"], DTYPES[c["params"]], _groups(c)
        s["x"] = _randn(g, rows, K, dtype=bf)
        s["weight"] = _randn(g, N, K, dtype=bf, scale=1.5 * K ** -0.5)
        s["bias"] = _randn(g, N, dtype=pd, scale=0.3) if c["bias"] else None
        s["gate"] = _randn(g, G, N, dtype=pd, scale=0.5) if c["gate"] else None
        od = DTYPES[c["out"]]
        if c["op"] == "linear":
            s["residual"] = _randn(g, rows, N, dtype=od) if c["residual"] else None
            s["out"] = torch.empty(rows, N, device="cuda", dtype=od)
            s["pre"] = torch.empty(rows, N, device="cuda", dtype=bf) if c["keep"] else None
            return s
        s["dout"] = _randn(g, rows, N, dtype=bf)
        s["pre"] = _product(s).to(bf) if c["activation"] != "none" or c["gate"] else None
        s["dx"], s["dweight"] = torch.empty_like(s["x"]), torch.empty_like(s["weight"])
        s["dbias"] = torch.empty(N, device="cuda") if c["bias"] else None
        s["dgate"] = torch.empty(G, N, device="cuda") if c["gate"] else None
        return s
    H, Hk, d, L, G = c["heads"], c["kv_heads"], c["d"], c["keys"], _groups(c)
    s["q"] = _randn(g, rows, H, d, dtype=bf, scale=1.5)
    if c["layout"] == "packed":  # one projection of the states gives both
        s["k"], s["v"] = _randn(g, G, L, 2, Hk, d, dtype=bf).unbind(2)
    else:
        s["k"], s["v"] = (_randn(g, G, L, Hk, d, dtype=bf) for _ in range(2))
    s["lengths"] = torch.tensor(_lengths(c), dtype=torch.int32, device="cuda") if c["lengths"] != "full" else None
    s["O"] = torch.empty(rows, H, d, device="cuda", dtype=bf)
    s["lse"] = torch.empty(H, rows, device="cuda") if c["keep"] else None
    if c["op"] == "cross":
        return s
    # what a forward pass kept
    s["O"], s["lse"] = _cross_plain(s, True)
    s["dO"] = _randn(g, rows, H, d, dtype=bf)
    s["dq"] = torch.empty(rows, H, d, device="cuda", dtype=bf)
    s["dk"], s["dv"] = torch.empty(G, L, 2, Hk, d, device="cuda", dtype=bf).unbind(2) if c["layout"] == "packed" else \
        (torch.empty(G, L, Hk, d, device="cuda", dtype=bf) for _ in range(2))
    return s


# ---------------------------------------------------------------- plain forms

def _product(s):
    z = s["x"].float() @ s["weight"].float().t()
    return z if s["bias"] is None else z + s["bias"].float()


def _inner_tanh(z):
    return math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)


def _act(z, kind):
    if kind == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(_inner_tanh(z)))
    if kind == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    return z / (1 + torch.exp(-z)) if kind == "silu" else z


def _act_slope(z, kind):
    if kind == "gelu_tanh":
        t = torch.tanh(_inner_tanh(z))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * z * z)
    if kind == "gelu":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    if kind == "silu":
        y = 1 / (1 + torch.exp(-z))
        return y * (1 + z * (1 - y))
    return torch.ones_like(z)


def _rows_of(m, c):
    """A group's values for each of its rows."""
    return m.float().repeat_interleave(c["group"], 0)[:c["rows"]]


def _padded(x, c):
    """[rows]... -> [groups][rows of a group]..., zeros behind the last row."""
    G = _groups(c)
    if G * c["group"] != c["rows"]:
        x = torch.cat((x, x.new_zeros(G * c["group"] - c["rows"], *x.shape[1:])))
    return x.view(G, c["group"], *x.shape[1:])


def _linear_plain(s):
    c = s["case"]
    z = _product(s)
    out = _act(z, c["activation"])
    if s["gate"] is not None:
        out = out * _rows_of(s["gate"], c)
    if s["residual"] is not None:
        out = out + s["residual"].float()
    out = out.to(DTYPES[c["out"]])
    return [out] if s["pre"] is None else [out, z.to(torch.bfloat16)]


def _linear_backward_plain(s):
    c, out = s["case"], {}
    da = s["dout"].float()
    z = s["pre"].float() if s["pre"] is not None else None
    if s["gate"] is not None:
        out["dgate"] = _padded(da * _act(z, c["activation"]), c).sum(1)
        da = da * _rows_of(s["gate"], c)
    if c["activation"] != "none":
        da = da * _act_slope(z, c["activation"])
    if s["dbias"] is not None:
        out["dbias"] = da.sum(0)
    out["dx"] = (da @ s["weight"].float()).to(torch.bfloat16)
    out["dweight"] = (da.t() @ s["x"].float()).to(torch.bfloat16)
    return out


def _scores(s):
    """softmax(q k) [groups][heads][rows][keys] of padded rows, its log-sum-exp, and q, k, v by heads."""
    c = s["case"]
    share = c["heads"] // c["kv_heads"]
    q = _padded(s["q"].float(), c).transpose(1, 2)
    k, v = (t.float().repeat_interleave(share, 2).transpose(1, 2) for t in (s["k"], s["v"]))
    x = q @ k.transpose(2, 3)
    x *= c["d"] ** -0.5
    if s["lengths"] is not None:
        x.masked_fill_((torch.arange(c["keys"], device="cuda") >= s["lengths"][:, None])[:, None, None], -math.inf)
    top = x.amax(3, keepdim=True)
    x -= torch.where(top == -math.inf, 0.0, top)
    x.exp_()
    total = x.sum(3, keepdim=True)
    x /= torch.where(total == 0, 1.0, total)
    return x, top + total.log(), q, k, v


def _tokens(x, c):
    """[groups][heads][rows][d] of padded rows -> [rows][heads][d]."""
    return x.transpose(1, 2).flatten(0, 1)[:c["rows"]]


def _cross_plain(s, keep):
    c = s["case"]
    p, lse, _, _, v = _scores(s)
    O = _tokens(p @ v, c).to(torch.bfloat16).contiguous()
    return [O, _tokens(lse, c)[..., 0].t().contiguous()] if keep else [O]


def _cross_backward_plain(s):
    c = s["case"]
    p, _, q, k, v = _scores(s)
    do = _padded(s["dO"].float(), c).transpose(1, 2)
    o = _padded(s["O"].float(), c).transpose(1, 2)
    shared = (_groups(c), c["kv_heads"], -1, c["keys"], c["d"])

    def states(x):  # a key head's gradient is the sum over the heads that share it
        return x.view(shared).sum(2).transpose(1, 2).to(torch.bfloat16)

    dv = states(p.transpose(2, 3) @ do)
    ds = do @ v.transpose(2, 3)
    ds -= (do * o).sum(3, keepdim=True)
    ds *= p
    ds *= c["d"] ** -0.5
    return [_tokens(ds @ k, c).to(torch.bfloat16), states(ds.transpose(2, 3) @ q), dv]


# ---------------------------------------------------------------- the library's calls

def _own(s):
    import block_sparse_spatio_gb300 as bss
    c = s["case"]
    if c["op"].startswith("linear"):
        kind = {"none": bss.ACT_NONE, "gelu_tanh": bss.ACT_GELU_TANH, "gelu": bss.ACT_GELU, "silu": bss.ACT_SILU}[c["activation"]]
        if c["op"] == "linear":
            bss.linear(s["x"], s["weight"], s["out"], bias=s["bias"], activation=kind, gate=s["gate"], residual=s["residual"],
                       rows_per_group=c["group"], pre=s["pre"])
            return [s["out"]] if s["pre"] is None else [s["out"], s["pre"]]
        grads = {k: s[k] for k in ("dx", "dweight", "dbias", "dgate")}
        bss.linear_backward(s["dout"], s["x"], s["weight"], activation=kind, pre=s["pre"], gate=s["gate"],
                            rows_per_group=c["group"], **grads)
        return {k: t for k, t in grads.items() if t is not None}
    if c["op"] == "cross":
        bss.cross_attention(s["q"], s["k"], s["v"], s["O"], lengths=s["lengths"], lse=s["lse"], rows_per_group=c["group"])
        return [s["O"]] if s["lse"] is None else [s["O"], s["lse"]]
    bss.cross_attention_backward(s["dO"], s["q"], s["k"], s["v"], s["O"], s["lse"], s["dq"], s["dk"], s["dv"],
                                 lengths=s["lengths"], rows_per_group=c["group"])
    return [s["dq"], s["dk"], s["dv"]]


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    if op == "cross":
        return _cross_plain(state, state["case"]["keep"])
    return {"linear": _linear_plain, "linear_backward": _linear_backward_plain, "cross_backward": _cross_backward_plain}[op](state)


def work(case):
    """Each input read once, each output written once."""
    c = case
    width = {"bf16": 2, "f32": 4}
    rows = c["rows"]
    if c["op"].startswith("linear"):
        K, N = c["inner"], c["outer"]
        small = width[c["params"]] * N * (int(c["bias"]) + (_groups(c) if c["gate"] else 0))
        if c["op"] == "linear":
            moved = 2 * (rows * K + N * K) + rows * N * (width[c["out"]] * (2 if c["residual"] else 1) + (2 if c["keep"] else 0))
            return {"bytes": moved + small, "flops": 2 * rows * K * N}
        reads_pre = c["activation"] != "none" or c["gate"]
        moved = 4 * (rows * K + N * K) + 2 * rows * N * (2 if reads_pre else 1)
        return {"bytes": moved + 2 * small, "flops": 4 * rows * K * N}
    H, Hk, d, G = c["heads"], c["kv_heads"], c["d"], _groups(c)
    valid = _lengths(c)
    pairs = H * sum(n * min(c["group"], rows - i * c["group"]) for i, n in enumerate(valid))
    states = 4 * Hk * d * sum(valid)  # K and V, as far as they are valid
    if c["op"] == "cross":
        return {"bytes": 4 * rows * H * d + states + (4 * rows * H if c["keep"] else 0), "flops": 4 * d * pairs}
    return {"bytes": 8 * rows * H * d + 4 * rows * H + states + 4 * Hk * d * G * c["keys"], "flops": 10 * d * pairs}


# ---------------------------------------------------------------- the definition, in 64 bits

def _exact_act(z, kind):
    if kind == "silu":
        return z * torch.sigmoid(z)
    return z if kind == "none" else torch.nn.functional.gelu(z, approximate="tanh" if kind == "gelu_tanh" else "none")


def _exact_gate(s, c):
    return s["gate"].double()[torch.arange(c["rows"], device="cuda") // c["group"]]


def _exact_linear(s):
    c = s["case"]
    z = torch.einsum("rk,nk->rn", s["x"].double(), s["weight"].double())
    if s["bias"] is not None:
        z += s["bias"].double()
    out = _exact_act(z, c["activation"])
    if s["gate"] is not None:
        out = out * _exact_gate(s, c)
    if s["residual"] is not None:
        out = out + s["residual"].double()
    return [out] if s["pre"] is None else [out, z]


def _exact_linear_backward(s):
    """The gradient at the pre-activation that a forward pass kept."""
    c, out = s["case"], {}
    d = s["dout"].double()
    leaf = torch.zeros_like(d) if s["pre"] is None else s["pre"].double()
    leaf.requires_grad_()
    ends = _exact_act(leaf, c["activation"])
    if s["gate"] is not None:
        at = torch.arange(c["rows"], device="cuda") // c["group"]
        out["dgate"] = torch.zeros(_groups(c), c["outer"], device="cuda", dtype=torch.float64).index_add_(0, at, (d * ends).detach())
        ends = ends * _exact_gate(s, c)
    dz, = torch.autograd.grad(ends, leaf, d)
    if s["dbias"] is not None:
        out["dbias"] = torch.einsum("rn->n", dz)
    out["dx"] = torch.einsum("rn,nk->rk", dz, s["weight"].double())
    out["dweight"] = torch.einsum("rn,rk->nk", dz, s["x"].double())
    return out


def _exact_cross(s, grads):
    """Group by group and head by head; the gradients by differentiation."""
    c = s["case"]
    share = c["heads"] // c["kv_heads"]
    O = torch.zeros(c["rows"], c["heads"], c["d"], device="cuda", dtype=torch.float64)
    lse = torch.full((c["heads"], c["rows"]), -math.inf, device="cuda", dtype=torch.float64)
    dq = torch.zeros_like(O)
    dk, dv = (torch.zeros(*s["k"].shape, device="cuda", dtype=torch.float64) for _ in range(2))
    for i, n in enumerate(_lengths(c)):
        at = slice(i * c["group"], min((i + 1) * c["group"], c["rows"]))
        for h in range(c["heads"] if n else 0):
            leaf = [t.double().requires_grad_() for t in (s["q"][at, h], s["k"][i, :n, h // share], s["v"][i, :n, h // share])]
            x = torch.einsum("rc,kc->rk", leaf[0], leaf[1]) / math.sqrt(c["d"])
            o = torch.einsum("rk,kc->rc", torch.softmax(x, 1), leaf[2])
            if grads:
                got = torch.autograd.grad(o, leaf, s["dO"][at, h].double())
                dq[at, h] = got[0]
                dk[i, :n, h // share] += got[1]
                dv[i, :n, h // share] += got[2]
            else:
                O[at, h], lse[h, at] = o.detach(), torch.logsumexp(x, 1).detach()
    return [dq, dk, dv] if grads else [O, lse] if c["keep"] else [O]


def exact(case, seed):
    s = prepare(case, seed)
    op = s["case"]["op"]
    if op.startswith("linear"):
        return _exact_linear(s) if op == "linear" else _exact_linear_backward(s)
    return _exact_cross(s, op == "cross_backward")

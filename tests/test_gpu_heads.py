"""heads_from_tokens and its gradient against 64-bit references, and the step
from token-major tensors against the calls it joins."""
import numpy as np
import pytest
import torch

import _block_ref as R
import oracle
import workloads as W

DEV = "cuda"
# Longest 32-bit chain behind a value: 8 squares in a row, 4 steps over a head's
# lanes, up to 34 steps over 128 heads, halved by the root, then the quotient,
# the root, two products and the rotation: below 48 roundings.
K_HEADS = 48
# A gradient has two such sums.
K_GRAD = 96

# F, Hs, Ws, H, d, channels per axis, halves, norm, layout, weights
CASES = {
    "token_norm": (3, 5, 7, 10, 128, (44, 42, 42), False, 2, "packed", torch.float32),
    "head_norm_halves": (3, 5, 7, 5, 64, (16, 16, 16), True, 1, "split", torch.bfloat16),
    "one_token": (1, 1, 1, 10, 128, (44, 42, 42), False, 2, "split", torch.float32),
    "one_head_d64": (4, 3, 11, 1, 64, (24, 20, 20), False, 1, "heads", torch.float32),
    "one_head_token_norm": (4, 3, 11, 1, 64, (16, 16, 32), True, 2, "split", torch.bfloat16),
    "rotation_only": (2, 7, 9, 3, 128, (44, 42, 42), False, 0, "packed", None),
    "rotation_only_halves": (2, 7, 9, 3, 128, (32, 48, 48), True, 0, "heads", None),
    "no_rotation": (5, 4, 4, 4, 64, None, False, 2, "split", torch.float32),
    "layout_only": (5, 4, 4, 4, 64, None, False, 0, "heads", None),
    "no_weights": (2, 3, 5, 2, 128, (8, 0, 6), False, 1, "split", "none"),
    "two_head_slices": (2, 3, 5, 17, 128, (64, 32, 32), True, 1, "packed", torch.float32),
    "many_heads_d64": (2, 3, 5, 33, 64, (0, 32, 32), False, 1, "split", torch.bfloat16),
    "widest_token": (2, 2, 3, 128, 64, (24, 20, 20), False, 2, "packed", torch.float32),
    "wide_token_halves": (2, 2, 3, 37, 128, (32, 32, 48), True, 2, "split", torch.bfloat16),
    "one_frame": (1, 9, 31, 10, 64, (24, 20, 20), False, 2, "split", torch.float32),
    "one_position": (19, 1, 1, 6, 128, (44, 42, 42), False, 1, "split", torch.float32),
}


def token_major(layout, N, H, d, g):
    if layout == "packed":
        return list((torch.randn(N, 3, H, d, generator=g) * 2).to(torch.bfloat16).unbind(1))
    if layout == "split":
        return [(torch.randn(N, H, d, generator=g) * 2).to(torch.bfloat16) for _ in range(3)]
    return [(torch.randn(H, N, d, generator=g) * 2).to(torch.bfloat16).transpose(0, 1) for _ in range(3)]


def to_device(t):
    """The same strides on the device."""
    base = torch.empty_strided(t.shape, t.stride(), dtype=t.dtype, device=DEV)
    return base.copy_(t)


class Case:
    def __init__(self, bss, name, seed=0):
        F, Hs, Ws, H, d, axes, halves, norm, layout, wt = CASES[name]
        g = torch.Generator().manual_seed(seed + 7)
        self.N, self.H, self.d, self.F, self.S = F * Hs * Ws, H, d, F, Hs * Ws
        self.norm, self.halves, self.layout, self.eps = norm, halves, layout, 1e-6
        self.p = bss.MaskParams(F, Hs, Ws, d, 1, 1)
        self.tokens = token_major(layout, self.N, H, d, g)
        self.flags = torch.randint(0, 2, (H,), generator=g, dtype=torch.uint8)
        width = {0: 0, 1: d, 2: H * d}[norm]
        self.weights = [None, None]
        if norm and wt != "none":
            self.weights = [(1 + 0.3 * torch.randn(width, generator=g)).to(wt) for _ in range(2)]
        self.rotary = self.ang = None
        if axes is not None:
            off = (2, 1, 3)
            tabs = [R.table(o + n, a // 2) for o, n, a in zip(off, (F, Hs, Ws), axes)]
            self.ang = R.angles(tabs, off, F, Hs, Ws)
            dev = [t.to(DEV) if t.numel() else None for t in tabs]
            self.rotary = bss.Rotary(*dev, offset=off, pairing=bss.PAIR_HALVES if halves else bss.PAIR_INTERLEAVED)
        self.dev = [to_device(t) for t in self.tokens]
        self.dw = [None if w is None else w.to(DEV) for w in self.weights]
        self.fl = self.flags.to(DEV)
        self.kw = dict(rotary=self.rotary, q_weight=self.dw[0], k_weight=self.dw[1], norm=norm, eps=self.eps)

    def outputs(self):
        return [torch.full((self.H, self.N, self.d), -7.0, device=DEV, dtype=torch.bfloat16) for _ in range(3)]

    def reference(self, i, flags=None):
        x = self.tokens[i].double()
        flags = self.flags if flags is None else flags
        if i == 2:
            return R.heads(x, None, 0, self.eps, None, False, flags, self.F, self.S)
        return R.heads(x, self.weights[i], self.norm, self.eps, self.ang, self.halves, flags, self.F, self.S)


@pytest.mark.gpu
@pytest.mark.parametrize("name", CASES)
def test_forward(bss, name):
    c = Case(bss, name)
    out = c.outputs()
    bss.heads_from_tokens(*c.dev, *out, c.p, c.fl, **c.kw)
    torch.cuda.synchronize()
    for i in range(2):
        R.check(out[i], *c.reference(i), K_HEADS, f"{name} {'QK'[i]}")
    assert torch.equal(out[2].cpu().double(), c.reference(2)[0])
    plain = c.outputs()
    bss.heads_from_tokens(*c.dev, *plain, c.p, None, **c.kw)  # no flags: the same rows, not permuted
    for a, b in zip(out, plain):
        moved = torch.full_like(b, -7.0)
        bss.permute(b, moved, c.fl, c.p)
        assert torch.equal(a, moved)


@pytest.mark.gpu
@pytest.mark.parametrize("name", CASES)
def test_backward(bss, name):
    c = Case(bss, name)
    g = torch.Generator().manual_seed(3)
    grads = [torch.randn(c.H, c.N, c.d, generator=g).to(torch.bfloat16) for _ in range(3)]
    outs = [to_device(t).fill_(-7.0) for t in token_major(c.layout, c.N, c.H, c.d, g)]
    if c.layout == "packed":  # one packed gradient, as the projection's backward wants it
        outs = list(torch.full((c.N, 3, c.H, c.d), -7.0, dtype=torch.bfloat16, device=DEV).unbind(1))
    width = {0: 0, 1: c.d, 2: c.H * c.d}[c.norm]
    dws = [torch.full((width,), -7.0, device=DEV) if c.norm else None for _ in range(2)]
    x = dict(q=c.dev[0], k=c.dev[1]) if c.norm else {}
    bss.heads_from_tokens_backward(*(t.to(DEV) for t in grads), *outs, c.p, c.fl, **c.kw, **x, dq_weight=dws[0],
                                   dk_weight=dws[1])
    torch.cuda.synchronize()
    for i in range(2):
        dx, mag, dw, dwmag = R.heads_grad(grads[i].double(), c.tokens[i].double(), c.weights[i], c.norm, c.eps, c.ang,
                                          c.halves, c.flags, c.F, c.S)
        R.check(outs[i], dx, mag, K_GRAD, f"{name} d{'qk'[i]}")
        if c.norm:  # a sum over tokens (and heads) of up to 2048 terms in a row at worst
            R.check(dws[i], dw, dwmag, 300, f"{name} d{'qk'[i]}_weight")
    dv = R.heads_grad(grads[2].double(), c.tokens[2].double(), None, 0, c.eps, None, False, c.flags, c.F, c.S)[0]
    assert torch.equal(outs[2].cpu().double(), dv)
    # the same call again: bit for bit
    again = [torch.empty_like(t) for t in dws if t is not None]
    if c.norm:
        bss.heads_from_tokens_backward(*(t.to(DEV) for t in grads), *outs, c.p, c.fl, **c.kw, **x, dq_weight=again[0],
                                       dk_weight=again[1])
        assert all(torch.equal(a, b) for a, b in zip(dws, again))


@pytest.mark.gpu
def test_each_tensor_alone_equals_all_three(bss):
    c = Case(bss, "token_norm")
    whole = c.outputs()
    bss.heads_from_tokens(*c.dev, *whole, c.p, c.fl, **c.kw)
    for i in range(3):
        ins, outs = [None] * 3, [None] * 3
        ins[i], outs[i] = c.dev[i], c.outputs()[0]
        bss.heads_from_tokens(*ins, *outs, c.p, c.fl, **c.kw)
        assert torch.equal(outs[i], whole[i])
        grads, dx = [None] * 3, [None] * 3
        grads[i], dx[i] = whole[i], torch.full((c.N, c.H, c.d), -7.0, dtype=torch.bfloat16, device=DEV)
        bss.heads_from_tokens_backward(*grads, *dx, c.p, c.fl, q=c.dev[0], k=c.dev[1], **c.kw)
        full = [torch.empty_like(dx[i]) for _ in range(3)]
        bss.heads_from_tokens_backward(*whole, *full, c.p, c.fl, q=c.dev[0], k=c.dev[1], **c.kw)
        assert torch.equal(dx[i], full[i])


@pytest.mark.gpu
def test_broadcast_heads(bss):
    """One K head read by every head (stride 0): each gets it; the gradient comes a head each."""
    c = Case(bss, "no_weights")
    one = c.dev[1][:, :1]
    shared = one.expand(c.N, c.H, c.d)
    a, b = c.outputs()[0], c.outputs()[0]
    bss.heads_from_tokens(None, shared, None, None, a, None, c.p, c.fl, **c.kw)
    bss.heads_from_tokens(None, shared.contiguous(), None, None, b, None, c.p, c.fl, **c.kw)
    assert torch.equal(a, b)


@pytest.mark.gpu
def test_writes_only_its_outputs(bss):
    c = Case(bss, "two_head_slices")
    G = 4096
    n = c.H * c.N * c.d
    bufs = [torch.full((n + 2 * G,), -7.0, dtype=torch.bfloat16, device=DEV) for _ in range(3)]
    outs = [b[G:G + n].view(c.H, c.N, c.d) for b in bufs]
    keep = [t.clone() for t in c.dev]
    bss.heads_from_tokens(*c.dev, *outs, c.p, c.fl, **c.kw)
    packed = torch.full((c.N + 2, 4, c.H, c.d), -7.0, dtype=torch.bfloat16, device=DEV)
    dx = [packed[1:-1, i] for i in range(3)]  # the fourth slot and the rows around stay as they are
    dw = torch.full((c.d + 16,), -7.0, device=DEV)
    ws = torch.full((1 << 20,), 171, dtype=torch.uint8, device=DEV)
    bss.heads_from_tokens_backward(*(o.contiguous() for o in outs), *dx, c.p, c.fl, q=c.dev[0], k=c.dev[1],
                                   dq_weight=dw[8:8 + c.d], workspace=ws[:1 << 19], **c.kw)
    torch.cuda.synchronize()
    for b in bufs:
        assert torch.all(b[:G] == -7.0) and torch.all(b[-G:] == -7.0)
    assert all(torch.equal(a, b) for a, b in zip(keep, c.dev))
    assert torch.all(packed[0] == -7.0) and torch.all(packed[-1] == -7.0) and torch.all(packed[:, 3] == -7.0)
    assert torch.all(dw[:8] == -7.0) and torch.all(dw[-8:] == -7.0) and torch.all(dw[8:-8] != -7.0)
    assert torch.all(ws[1 << 19:] == 171)


@pytest.mark.gpu
def test_nonfinite_values_stay_in_their_token(bss):
    for name in ("token_norm", "head_norm_halves", "rotation_only"):
        c = Case(bss, name)
        want = c.outputs()
        bss.heads_from_tokens(*c.dev, *want, c.p, None, **c.kw)
        q = c.dev[0].clone()
        q[4, 1, 5] = float("inf")
        q[9, 0, 3] = float("nan")
        got = c.outputs()
        bss.heads_from_tokens(q, c.dev[1], c.dev[2], *got, c.p, None, **c.kw)
        rows = [n for n in range(c.N) if n not in (4, 9)]
        assert torch.equal(got[0][:, rows], want[0][:, rows])
        assert torch.equal(got[1], want[1]) and torch.equal(got[2], want[2])
        assert torch.isnan(got[0][0, 9]).any()


@pytest.mark.gpu
@pytest.mark.parametrize("name,rotated", [("no_weights", 14), ("head_norm_halves", 48)])
def test_channels_that_pass_keep_their_bits(bss, name, rotated):
    """Unrotated channels next to infinities and of zeros of both signs."""
    c = Case(bss, name)
    q = c.dev[0].clone()
    q[1, :, rotated] = float("inf")
    q[2, :, -1] = float("-inf")
    q[3, :, rotated:] = -0.0
    out = c.outputs()[0]
    bss.heads_from_tokens(q, None, None, out, None, None, c.p, None, rotary=c.rotary)
    bits = lambda t: t.contiguous().view(torch.int16)  # noqa: E731
    assert torch.equal(bits(out[:, :, rotated:]), bits(q.transpose(0, 1)[:, :, rotated:]))
    back = torch.empty_like(q)
    bss.heads_from_tokens_backward(out, None, None, back, None, None, c.p, None, rotary=c.rotary)
    assert torch.equal(bits(back[:, :, rotated:]), bits(q[:, :, rotated:]))


@pytest.mark.gpu
def test_zero_tokens_stay_zero(bss):
    """A token of zeros (padding): finite, zero heads, and no part in the gradients."""
    c = Case(bss, "token_norm")
    c.kw["eps"] = 1e-6
    q = torch.zeros(c.N, c.H, c.d, dtype=torch.bfloat16, device=DEV)
    out = c.outputs()[0]
    bss.heads_from_tokens(q, None, None, out, None, None, c.p, c.fl, **c.kw)
    assert torch.all(out == 0)


@pytest.mark.gpu
def test_other_stream_and_two_captured_graphs(bss):
    c = Case(bss, "token_norm")
    want = c.outputs()
    bss.heads_from_tokens(*c.dev, *want, c.p, c.fl, **c.kw)
    grads = [torch.randn(c.H, c.N, c.d, device=DEV).to(torch.bfloat16) for _ in range(3)]

    def backward(dx, dw, **kw):
        bss.heads_from_tokens_backward(*grads, *dx, c.p, c.fl, q=c.dev[0], k=c.dev[1], dq_weight=dw[0], dk_weight=dw[1],
                                       **c.kw, **kw)

    def buffers():
        return ([torch.zeros(c.N, c.H, c.d, dtype=torch.bfloat16, device=DEV) for _ in range(3)],
                [torch.zeros(c.H * c.d, device=DEV) for _ in range(2)])
    dx0, dw0 = buffers()
    backward(dx0, dw0)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got, (dx, dw) = c.outputs(), buffers()
    torch.cuda.synchronize()
    bss.heads_from_tokens(*c.dev, *got, c.p, c.fl, stream=s, **c.kw)
    backward(dx, dw, stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got + dx + dw, want + dx0 + dw0))
    # two graphs, replayed in turn and back to back, each with its own workspace
    sets = []
    for _ in range(2):
        got, (dx, dw) = c.outputs(), buffers()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            bss.heads_from_tokens(*c.dev, *got, c.p, c.fl, **c.kw)
            backward(dx, dw)
        sets.append((graph, got + dx + dw))
    for _ in range(3):
        for graph, _ in sets:
            graph.replay()
    torch.cuda.synchronize()
    for _, got in sets:
        assert all(torch.equal(a, b) for a, b in zip(got, want + dx0 + dw0))
    new = torch.randn_like(c.dev[0].float()).to(torch.bfloat16)
    c.dev[0].copy_(new)  # new inputs reach a replay
    bss.heads_from_tokens(*c.dev, *want, c.p, c.fl, **c.kw)
    sets[0][0].replay()
    torch.cuda.synchronize()
    assert torch.equal(sets[0][1][0], want[0])


@pytest.mark.gpu
def test_rotary_table(bss):
    got = bss.rotary_table(50, 21, base=10000.0, dim=42)
    i = torch.arange(21, dtype=torch.float64)
    a = torch.arange(50, dtype=torch.float64)[:, None] * 10000.0 ** (-2 * i / 42)
    # one rounding to float, and the 64-bit angle's error (2 ulp of at most 50)
    assert ((got[..., 0].cpu().double() - a.cos()).abs() <= 2.0 ** -25 + 2.0 ** -24 * a.cos().abs() * 0.5 + 1e-13).all()
    assert ((got[..., 1].cpu().double() - a.sin()).abs() <= 2.0 ** -25 + 2.0 ** -24 * a.sin().abs() * 0.5 + 1e-13).all()
    pos = torch.tensor([0.5, 1e6, -3.25], dtype=torch.float64)  # far and fractional positions
    got = bss.rotary_table(3, 4, base=500.0, positions=pos.to(DEV))
    a = pos[:, None] * 500.0 ** (-torch.arange(4, dtype=torch.float64) / 4)
    assert ((got[..., 0].cpu().double() - a.cos()).abs() <= 2.0 ** -24 + 1e-9).all()
    assert ((got[..., 1].cpu().double() - a.sin()).abs() <= 2.0 ** -24 + 1e-9).all()


@pytest.mark.gpu
@pytest.mark.parametrize("permuted", [1, 0])
@pytest.mark.parametrize("flagged", [True, False])
def test_step_equals_the_calls_it_joins(bss, permuted, flagged):
    F, Hs, Ws, H, d = 5, 7, 9, 3, 64
    p = bss.MaskParams(F, Hs, Ws, d, 1, 9, temporal_permuted=permuted)
    N = p.N
    g = torch.Generator().manual_seed(5)
    qkv = torch.randn(N, 3, H, d, generator=g).to(torch.bfloat16).to(DEV)
    q, k, v = qkv.unbind(1)
    rot = bss.Rotary(bss.rotary_table(F, 12), bss.rotary_table(Hs, 10), bss.rotary_table(Ws, 10))
    w = torch.rand(H * d, device=DEV) + 0.5
    kw = dict(rotary=rot, q_weight=w, k_weight=w, norm=bss.HEAD_NORM_TOKEN)
    fl = torch.tensor([1, 0, 1], dtype=torch.uint8, device=DEV) if flagged else None
    make = lambda: torch.full((H, N, d), -7.0, dtype=torch.bfloat16, device=DEV)  # noqa: E731
    O1, O2, L1, L2 = make(), make(), torch.zeros(H, N, device=DEV), torch.zeros(H, N, device=DEV)
    with bss.build_tile_map(p) as tm:
        Q, K, V = make(), make(), make()
        bss.heads_from_tokens(q, k, v, Q, K, V, p, None, **kw)
        bss.attention_step(Q, K, V, O1, tm, fl, make(), make(), make(), lse=L1)
        ws = make(), make(), make()
        bss.attention_step_tokens(q, k, v, O2, tm, fl, *ws, lse=L2, **kw)
        torch.cuda.synchronize()
    assert bss.get_device_status() == 0
    assert torch.equal(O1, O2) and torch.equal(L1, L2)
    # and the whole path against the oracle, from the rounded Q and K
    geo = oracle.Geometry(F, Hs, Ws, wf=1, ws=9, bkv=128)
    for h in range(H):
        kind = oracle.TEMPORAL_FHW if flagged and fl[h] else oracle.SPATIAL
        ref, _ = oracle.attention(W.bf16_bits(Q[h].cpu()), W.bf16_bits(K[h].cpu()), W.bf16_bits(V[h].cpu()), kind, geo)
        assert np.abs(O2[h].float().cpu().numpy() - ref).max() <= 1e-2


@pytest.mark.gpu
def test_offsets_past_32_bits(bss):
    """More than 2^32 bytes in one tensor: the last tokens of the last heads."""
    F, Hs, Ws, H, d = 21, 90, 160, 57, 128
    p = bss.MaskParams(F, Hs, Ws, d, 1, 1)
    N = p.N
    assert N * H * d * 2 > 1 << 32
    q = torch.empty(N, H, d, dtype=torch.bfloat16, device=DEV)
    q.view(-1).copy_(torch.arange(1 << 16, device=DEV, dtype=torch.int32).remainder(251).to(torch.bfloat16)
                     .repeat(-(-q.numel() // (1 << 16)))[:q.numel()])
    out = torch.empty(H, N, d, dtype=torch.bfloat16, device=DEV)
    fl = torch.zeros(H, dtype=torch.uint8, device=DEV)
    fl[H - 1] = 1
    bss.heads_from_tokens(None, None, q, None, None, out, p, fl)
    assert torch.equal(out[H - 2], q[:, H - 2])
    assert torch.equal(out[H - 1].view(Hs * Ws, F, d), q[:, H - 1].view(F, Hs * Ws, d).transpose(0, 1))
    back = torch.empty_like(q)
    bss.heads_from_tokens_backward(None, None, out, None, None, back, p, fl)
    assert torch.equal(back, q)
    del back
    w = torch.rand(d, device=DEV) + 0.5
    bss.heads_from_tokens(q, None, None, out, None, None, p, fl, q_weight=w, norm=bss.HEAD_NORM_HEAD)
    rows = torch.tensor([0, 1, N // 2, N - 2, N - 1])
    x = q[rows].cpu().double()
    ref, mag = R.heads(x, w.cpu(), 1, 1e-6, None, False, [0] * H, 5, 1)
    R.check(out[:H - 1, rows], ref[:H - 1], mag[:H - 1], K_HEADS)


@pytest.mark.gpu
def test_step_refusals_launch_nothing(bss):
    """What the attention call would refuse is refused before Q, K and V are touched."""
    p = bss.MaskParams(2, 3, 5, 64, 1, 2)
    H, N, d = 2, p.N, 64
    q = torch.randn(N, H, d, device=DEV).to(torch.bfloat16)
    make = lambda: torch.full((H, N, d), -7.0, dtype=torch.bfloat16, device=DEV)  # noqa: E731
    ws, O = [make() for _ in range(3)], make()
    with bss.build_tile_map(p, BQ=64, BKV=64) as tm:  # a tile the attention kernel does not run
        with pytest.raises(bss.BssError) as e:
            bss.attention_step_tokens(q, q, q, O, tm, None, *ws)
        assert e.value.status == 2
    with bss.build_tile_map(p) as tm:
        for bad in (ws[0], ws[2]):
            with pytest.raises(bss.BssError):
                bss.attention_step_tokens(q, q, q, bad, tm, None, *ws)
        with pytest.raises(bss.BssError):
            bss.attention_step_tokens(q, None, q, O, tm, None, *ws)
        with pytest.raises(ValueError):
            bss.attention_step_tokens(q, q, q, O[:, :-1], tm, None, *ws)
        with pytest.raises(ValueError):
            bss.attention_step_tokens(q, q, q, O, tm, torch.ones(H + 1, dtype=torch.uint8, device=DEV), *ws)
    torch.cuda.synchronize()
    assert all(torch.all(t == -7.0) for t in ws + [O])

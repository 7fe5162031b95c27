"""The matrix products and the cross attention as a transformer block uses them:
together with the norms and the attention step, captured into graphs, on other
streams, and writing nothing beside their outputs."""
import ctypes

import pytest
import torch

import _block_ref as R
import _layers_ref as L
from test_gpu_canary import guarded, intact

pytestmark = pytest.mark.gpu
DEV, BF, F32 = "cuda", torch.bfloat16, torch.float32
F, Hs, Ws, H, d = 4, 6, 7, 3, 64
S, N, C = Hs * Ws, F * Hs * Ws, H * d
STATES, WIDTH = 50, 136  # of the encoder


class Block:
    """Self attention, cross attention and a feed-forward layer of a small clip."""

    def __init__(self, bss):
        g = torch.Generator().manual_seed(5)
        rnd = lambda *s, scale=1.0: (torch.randn(*s, generator=g) * scale)  # noqa: E731
        w = lambda o, i: rnd(o, i, scale=i ** -0.5).to(BF).to(DEV)  # noqa: E731
        b = lambda o: rnd(o, scale=0.1).to(DEV)  # noqa: E731
        self.p = bss.MaskParams(F, Hs, Ws, d, 1, 9)
        self.x, self.context = rnd(N, C).to(BF).to(DEV), rnd(2 * STATES, WIDTH).to(BF).to(DEV)
        self.mod = rnd(F, 6, C, scale=0.3).to(DEV)
        self.w = {n: (w(o, i), b(o)) for n, o, i in (("qkv", 3 * C, C), ("out", C, C), ("q", C, C), ("kv", 2 * C, WIDTH),
                                                      ("cross", C, C), ("up", 4 * C, C), ("down", C, 4 * C))}
        self.fl = torch.tensor([1, 0, 1], dtype=torch.uint8, device=DEV)
        self.lengths = torch.tensor([STATES, 11], dtype=torch.int32, device=DEV)  # a prompt for each half of the clip
        e = lambda *s: torch.zeros(*s, dtype=BF, device=DEV)  # noqa: E731
        self.t = {n: e(N, C) for n in ("h", "a", "r1", "h2", "q", "c", "r2", "h3", "r3")}
        self.t.update(qkv=e(N, 3 * C), kv=e(2 * STATES, 2 * C), up=e(N, 4 * C), pre=e(N, 4 * C))
        self.heads, self.O = [e(H, N, d) for _ in range(3)], e(H, N, d)
        self.lse = torch.zeros(H, N, device=DEV)

    def states(self):
        return self.t["kv"].view(2, STATES, 2, H, d).unbind(2)

    def forward(self, bss, tm):
        t, m, w = self.t, self.mod, self.w
        bss.residual_norm(self.x, h=t["h"], shift=m[:, 0], scale=m[:, 1], rows_per_group=S)
        bss.linear(t["h"], w["qkv"][0], t["qkv"], bias=w["qkv"][1])
        bss.attention_step_tokens(*t["qkv"].view(N, 3, H, d).unbind(1), self.O, tm, self.fl, *self.heads)
        t["a"].view(N, H, d).copy_(self.O.transpose(0, 1))
        bss.linear(t["a"], w["out"][0], t["r1"], bias=w["out"][1], gate=m[:, 2], residual=self.x, rows_per_group=S)
        bss.residual_norm(t["r1"], h=t["h2"])
        bss.linear(t["h2"], w["q"][0], t["q"], bias=w["q"][1])
        bss.linear(self.context, w["kv"][0], t["kv"], bias=w["kv"][1])
        k, v = self.states()
        bss.cross_attention(t["q"].view(N, H, d), k, v, t["c"].view(N, H, d), lengths=self.lengths, lse=self.lse,
                            rows_per_group=N // 2)
        bss.linear(t["c"], w["cross"][0], t["r2"], bias=w["cross"][1], residual=t["r1"])
        bss.residual_norm(t["r2"], h=t["h3"], shift=m[:, 3], scale=m[:, 4], rows_per_group=S)
        bss.linear(t["h3"], w["up"][0], t["up"], bias=w["up"][1], activation=bss.ACT_GELU_TANH, pre=t["pre"])
        bss.linear(t["up"], w["down"][0], t["r3"], bias=w["down"][1], gate=m[:, 5], residual=t["r2"], rows_per_group=S)

    def kept(self):
        return [t.clone() for t in (*self.t.values(), self.O, self.lse)]


def test_block(bss):
    b = Block(bss)
    with bss.build_tile_map(b.p) as tm:
        b.forward(bss, tm)
        torch.cuda.synchronize()
        assert bss.get_device_status() == 0
        once = b.kept()
        # captured on a stream of its own, replayed twice on cleared buffers
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            b.forward(bss, tm)
        for _ in range(2):
            for t in (*b.t.values(), b.O, b.lse):
                t.zero_()
            graph.replay()
            torch.cuda.synchronize()
            for x, y in zip(b.kept(), once):
                assert torch.equal(x, y)
    t, m, w = {n: x.cpu() for n, x in b.t.items()}, b.mod.cpu(), {n: (x.cpu(), y.cpu()) for n, (x, y) in b.w.items()}
    for out, x, name, kw in (("qkv", "h", "qkv", {}), ("r1", "a", "out", dict(gate=m[:, 2], residual=b.x.cpu(), group=S)),
                             ("q", "h2", "q", {}), ("r2", "c", "cross", dict(residual=t["r1"])),
                             ("up", "h3", "up", dict(kind=1)), ("r3", "up", "down", dict(gate=m[:, 5], residual=t["r2"], group=S))):
        ref = L.linear(t[x], *w[name], **{"group": N, **kw})
        R.check(t[out], *ref["out"], 1, out)
        if out == "up":
            R.check(t["pre"], *ref["pre"], 1, "pre")
    R.check(t["kv"], *L.linear(b.context.cpu(), *w["kv"])["out"], 1, "kv")
    k, v = (x.cpu() for x in b.states())
    ref = L.cross(t["q"].view(N, H, d), k, v, [STATES, 11], N // 2)
    R.check(t["c"].view(N, H, d), *ref["O"], 1, "cross attention")
    R.check(b.lse.cpu(), *ref["lse"], 1, "lse")


def backward(bss, b, dr3):
    """Gradients of the block behind its self attention."""
    t, m, w, o = b.t, b.mod, b.w, {}
    e = lambda *s, dtype=BF: torch.full(s, float("nan"), dtype=dtype, device=DEV)  # noqa: E731
    dup, do, dq, dh3, dkv = e(N, 4 * C), e(N, C), e(N, C), e(N, C), e(2 * STATES, 2 * C)
    o["w_down"], o["b_down"], o["gate"] = e(C, 4 * C), e(C, dtype=F32), e(F, C, dtype=F32)
    down = e(N, C)
    bss.linear(t["up"], w["down"][0], down, bias=w["down"][1])  # what the gate multiplied, for its gradient
    bss.linear_backward(dr3, t["up"], w["down"][0], dup, o["w_down"], o["b_down"], o["gate"], pre=down, gate=m[:, 5], rows_per_group=S)
    o["w_up"], o["b_up"] = e(4 * C, C, dtype=F32), e(4 * C, dtype=F32)
    bss.linear_backward(dup, t["h3"], w["up"][0], dh3, o["w_up"], o["b_up"], activation=bss.ACT_GELU_TANH, pre=t["pre"])
    o["w_cross"] = e(C, C)
    bss.linear_backward(dr3, t["c"], w["cross"][0], do, o["w_cross"])
    k, v = b.states()
    dk, dv = dkv.view(2, STATES, 2, H, d).unbind(2)
    bss.cross_attention_backward(do.view(N, H, d), t["q"].view(N, H, d), k, v, t["c"].view(N, H, d), b.lse, dq.view(N, H, d),
                                 dk, dv, lengths=b.lengths, rows_per_group=N // 2)
    o["context"], o["w_kv"] = e(2 * STATES, WIDTH), e(2 * C, WIDTH)
    bss.linear_backward(dkv, b.context, w["kv"][0], o["context"], o["w_kv"])
    o.update(dup=dup, dh3=dh3, do=do, dq=dq, dkv=dkv, down=down)
    return o


def test_block_backward(bss):
    b = Block(bss)
    with bss.build_tile_map(b.p) as tm:
        b.forward(bss, tm)
    dr3 = torch.randn(N, C, generator=torch.Generator().manual_seed(8)).to(BF).to(DEV)
    got = backward(bss, b, dr3)
    # two graphs of it at once, on streams of their own: each has workspaces of its own
    graphs, outs = [], []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(backward(bss, b, dr3))
        graphs.append(graph)
    streams = [torch.cuda.Stream() for _ in graphs]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        for graph, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    assert bss.get_device_status() == 0
    for o in outs:
        for n, t in o.items():
            assert torch.equal(t, got[n]), n
    cpu = {n: t.cpu() for n, t in got.items()}
    t, m, w = {n: x.cpu() for n, x in b.t.items()}, b.mod.cpu(), {n: x.cpu() for n, (x, _) in b.w.items()}
    ref = L.linear_grad(dr3.cpu(), t["up"], w["down"], cpu["down"], 0, m[:, 5], S)
    for n, x in (("dup", "dx"), ("w_down", "dweight"), ("b_down", "dbias"), ("gate", "dgate")):
        R.check(cpu[n], *ref[x], 1, n)
    ref = L.linear_grad(cpu["dup"], t["h3"], w["up"], t["pre"], 1)
    for n, x in (("dh3", "dx"), ("w_up", "dweight"), ("b_up", "dbias")):
        R.check(cpu[n], *ref[x], 1, n)
    k, v = (x.cpu() for x in b.states())
    ref = L.cross_grad(cpu["do"].view(N, H, d), t["q"].view(N, H, d), k, v, t["c"].view(N, H, d), b.lse.cpu(), [STATES, 11], N // 2)
    R.check(cpu["dq"].view(N, H, d), *ref["dq"], 1, "dq")
    for i, n in enumerate(("dk", "dv")):
        R.check(cpu["dkv"].view(2, STATES, 2, H, d)[:, :, i], *ref[n], 1, n)
    ref = L.linear_grad(cpu["dkv"], b.context.cpu(), w["kv"])
    R.check(cpu["context"], *ref["dx"], 1, "context")
    R.check(cpu["w_kv"], *ref["dweight"], 1, "w_kv")


# rows, in, out: few rows, single tiles, a split contraction, pairs of CTAs
@pytest.mark.parametrize("rows,inner,outer", [(3, 64, 40), (130, 72, 136), (50, 4096, 72), (20100, 64, 72)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_linear_writes_only_its_outputs(bss, rows, inner, outer, dtype):
    x, w = torch.randn(rows, inner, device=DEV).to(BF), torch.randn(outer, inner, device=DEV).to(BF)
    sent = -7.0
    bufs = {"out": guarded((rows, outer), dtype, sent, DEV), "pre": guarded((rows, outer), BF, sent, DEV),
            "dx": guarded((rows, inner), BF, sent, DEV), "dweight": guarded((outer, inner), dtype, sent, DEV),
            "dbias": guarded((outer,), F32, sent, DEV), "dgate": guarded((-(-rows // 7), outer), F32, sent, DEV)}
    gate = torch.randn(-(-rows // 7), outer, device=DEV)
    bss.linear(x, w, bufs["out"][1], activation=bss.ACT_SILU, gate=gate, rows_per_group=7, pre=bufs["pre"][1])
    dout = torch.randn(rows, outer, device=DEV).to(dtype)
    a = bss._LinearGrads(rows, 7, inner, outer, 0 if dtype == BF else 1, 1, 0 if dtype == BF else 1, 3,
                         *(t.data_ptr() for t in (dout, x, w, bufs["pre"][1], gate, bufs["dx"][1], bufs["dweight"][1],
                                                  bufs["dbias"][1], bufs["dgate"][1])),
                         outer, inner, inner, outer, outer, inner, inner)
    need = ctypes.c_int64()
    bss._check(bss.load().bss_linear_backward_workspace(ctypes.byref(a), ctypes.byref(need)))
    wbuf, ws = guarded((need.value,), torch.uint8, 77, DEV)
    bss.linear_backward(dout, x, w, activation=bss.ACT_SILU, pre=bufs["pre"][1], gate=gate, rows_per_group=7, workspace=ws,
                        **{n: bufs[n][1] for n in ("dx", "dweight", "dbias", "dgate")})
    torch.cuda.synchronize()
    assert bss.get_device_status() == 0
    for n, (buf, view) in bufs.items():
        assert intact(buf, sent), n
        assert torch.isfinite(view).all(), n
    assert intact(wbuf, 77)


@pytest.mark.parametrize("rows,group,keys,d_", [(1, 1, 3, 64), (300, 130, 70, 128), (257, 257, 200, 64), (2000, 600, 129, 128)])
def test_cross_writes_only_its_outputs(bss, rows, group, keys, d_):
    groups, heads, kv = -(-rows // group), 4, 2
    sent = -7.0
    r = lambda *s: torch.randn(*s, device=DEV).to(BF)  # noqa: E731
    q, k, v, do = r(rows, heads, d_), r(groups, keys, kv, d_), r(groups, keys, kv, d_), r(rows, heads, d_)
    shapes = {"O": (rows, heads, d_), "dq": (rows, heads, d_), "dk": k.shape, "dv": k.shape}
    bufs = {n: guarded(s, BF, sent, DEV) for n, s in shapes.items()}
    lbuf, lse = guarded((heads, rows), F32, sent, DEV)
    lengths = torch.tensor([keys - 1, 0, keys][:groups] + [1] * (groups - 3), dtype=torch.int32, device=DEV)
    bss.cross_attention(q, k, v, bufs["O"][1], lengths=lengths, lse=lse, rows_per_group=group)
    bss.cross_attention_backward(do, q, k, v, bufs["O"][1], lse, *(bufs[n][1] for n in ("dq", "dk", "dv")), lengths=lengths,
                                 rows_per_group=group)
    torch.cuda.synchronize()
    assert bss.get_device_status() == 0
    for n, (buf, view) in bufs.items():
        assert intact(buf, sent), n
        assert torch.isfinite(view).all(), n
    assert intact(lbuf, sent)


def test_other_streams(bss):
    """Calls of several streams at once, each with workspaces of its own stream."""
    rows = 400
    x, w = torch.randn(rows, 4096, device=DEV).to(BF), torch.randn(264, 4096, device=DEV).to(BF)
    q, k = torch.randn(rows, 3, 64, device=DEV).to(BF), torch.randn(1, 90, 3, 64, device=DEV).to(BF)

    def calls(stream):
        o, dw, O = torch.empty(rows, 264, device=DEV, dtype=BF), torch.empty(264, 4096, device=DEV), torch.empty_like(q)
        lse, dq, dk, dv = torch.empty(3, rows, device=DEV), torch.empty_like(q), torch.empty_like(k), torch.empty_like(k)
        if stream is not None:
            stream.wait_stream(torch.cuda.current_stream())
        bss.linear(x, w, o, stream=stream)
        bss.linear_backward(o, x=x, dweight=dw, stream=stream)
        bss.cross_attention(q, k, k, O, lse=lse, stream=stream)
        bss.cross_attention_backward(O, q, k, k, O, lse, dq, dk, dv, stream=stream)
        return o, dw, O, dq, dk, dv

    want = calls(None)
    got = [calls(s) for s in (torch.cuda.Stream(), torch.cuda.Stream(), torch.cuda.Stream())]
    torch.cuda.synchronize()
    for one in got:
        for a, b in zip(one, want):
            assert torch.equal(a, b)


def test_refused_by_the_binding(bss):
    x, w, o = (torch.zeros(*s, device=DEV, dtype=BF) for s in ((4, 16), (8, 16), (4, 8)))
    for bad in (dict(x=x.float()), dict(x=x.cpu()), dict(weight=w[:, :8]), dict(out=o.half()), dict(out=o[:2]),
                dict(bias=torch.zeros(8, device=DEV, dtype=torch.float16)), dict(bias=torch.zeros(4, device=DEV)),
                dict(gate=torch.zeros(3, 8, device=DEV)), dict(gate=torch.zeros(1, 8, device=DEV), bias=torch.zeros(8, device=DEV, dtype=BF)),
                dict(residual=o.float()), dict(pre=torch.zeros(4, 8, device=DEV)), dict(x=x.t()), dict(rows_per_group=0)):
        with pytest.raises((ValueError, bss.BssError)):
            bss.linear(**{**dict(x=x, weight=w, out=o), **bad})
    with pytest.raises((ValueError, bss.BssError)):
        bss.linear_backward(o, weight=w)
    q, k, O = torch.zeros(4, 2, 64, device=DEV, dtype=BF), torch.zeros(1, 5, 2, 64, device=DEV, dtype=BF), torch.zeros(4, 2, 64, device=DEV, dtype=BF)
    for bad in (dict(q=q.float()), dict(k=k.float()), dict(k=k[:, :, :, :32]), dict(v=k[:, :4]), dict(k=k.expand(2, -1, -1, -1)),
                dict(O=O[:3]), dict(lengths=torch.zeros(1, device=DEV)), dict(lengths=torch.zeros(2, device=DEV, dtype=torch.int32)),
                dict(lse=torch.zeros(4, 2, device=DEV)), dict(rows_per_group=2), dict(q=q[:, 0]), dict(q=q.cpu()),
                dict(softmax_scale=float("nan"))):
        with pytest.raises((ValueError, bss.BssError)):
            bss.cross_attention(**{**dict(q=q, k=k, v=k, O=O), **bad})
    with pytest.raises((ValueError, bss.BssError)):
        bss.cross_attention_backward(O, q, k, k, O, None, q, k, k)

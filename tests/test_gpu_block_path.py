"""The operators around the attention step run together, as a transformer block
uses them, forward and backward: every stage against its 64-bit reference on the
stage before it, the whole in place and captured into one graph."""
import numpy as np
import pytest
import torch

import _block_ref as R
import oracle
import workloads as W
from test_gpu_heads import K_GRAD, K_HEADS
from test_gpu_residual_norm import K_DX, K_H, K_R, K_SUM

DEV = "cuda"
F, Hs, Ws, H, d = 4, 6, 7, 3, 64
S, N, C = Hs * Ws, F * Hs * Ws, H * d


class Block:
    """Weights, inputs and buffers of one block of a small clip; modulations a frame."""

    def __init__(self, bss):
        g = torch.Generator().manual_seed(3)
        rnd = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
        bf = torch.bfloat16
        self.p = bss.MaskParams(F, Hs, Ws, d, 1, 9)
        self.x = rnd(N, C).to(bf).to(DEV)
        self.mod = (rnd(F, 5, C) * 0.3).to(DEV)  # shift, scale | gate, shift, scale of the next norm
        self.w_qkv = (rnd(C, 3 * C) / C ** 0.5).to(bf).to(DEV)
        self.w_out = (rnd(C, C) / C ** 0.5).to(bf).to(DEV)
        self.wq, self.wk = ((1 + 0.2 * rnd(C)).to(DEV) for _ in range(2))
        self.tabs = [R.table(n, p_) for n, p_ in ((F, 12), (Hs, 10), (Ws, 10))]
        self.rot = bss.Rotary(*(t.to(DEV) for t in self.tabs))
        self.flags = torch.tensor([1, 0, 1], dtype=torch.uint8)
        self.fl = self.flags.to(DEV)
        e = lambda *s: torch.zeros(*s, dtype=bf, device=DEV)  # noqa: E731
        self.h, self.qkv, self.y, self.r, self.h2 = e(N, C), e(N, 3 * C), e(N, C), e(N, C), e(N, C)
        self.heads, self.O = [e(H, N, d) for _ in range(3)], e(H, N, d)
        self.st, self.st2 = torch.zeros(N, 2, device=DEV), torch.zeros(N, 2, device=DEV)
        self.kw = dict(rotary=self.rot, q_weight=self.wq, k_weight=self.wk, norm=bss.HEAD_NORM_TOKEN)

    def forward(self, bss, tm):
        m = self.mod
        bss.residual_norm(self.x, h=self.h, shift=m[:, 0], scale=m[:, 1], rows_per_group=S, stats=self.st)
        torch.mm(self.h, self.w_qkv, out=self.qkv)
        q, k, v = self.qkv.view(N, 3, H, d).unbind(1)
        bss.attention_step_tokens(q, k, v, self.O, tm, self.fl, *self.heads, **self.kw)
        torch.mm(self.O.transpose(0, 1).reshape(N, C), self.w_out, out=self.y)
        bss.residual_norm(self.x, self.y, self.r, self.h2, gate=m[:, 2], shift=m[:, 3], scale=m[:, 4], rows_per_group=S,
                          stats=self.st2)


@pytest.mark.gpu
def test_block_forward_stage_by_stage(bss):
    b = Block(bss)
    with bss.build_tile_map(b.p) as tm:
        b.forward(bss, tm)
        torch.cuda.synchronize()
        assert bss.get_device_status() == 0
        kept = [t.clone() for t in (b.h, b.qkv, *b.heads, b.O, b.y, b.r, b.h2, b.st2)]
        # captured into one graph and replayed on new inputs
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            b.forward(bss, tm)  # the matrix products' own first calls
        torch.cuda.current_stream().wait_stream(s)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            b.forward(bss, tm)
        for t in (b.h, b.qkv, *b.heads, b.O, b.y, b.r, b.h2, b.st2):
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for t, want in zip((b.h, b.qkv, *b.heads, b.O, b.y, b.r, b.h2, b.st2), kept):
            assert torch.equal(t, want)
    m = b.mod.cpu()
    o = R.residual_norm(b.x.cpu(), shift=m[:, 0], scale=m[:, 1], group=S)
    R.check(b.h, o["h"], o["hmag"], K_H, "h")
    ang = R.angles(b.tabs, (0, 0, 0), F, Hs, Ws)
    q, k, v = (t.double().cpu() for t in b.qkv.view(N, 3, H, d).unbind(1))
    for got, x, w in ((b.heads[0], q, b.wq), (b.heads[1], k, b.wk)):
        ref, mag = R.heads(x, w.cpu(), 2, 1e-6, ang, False, b.flags, F, S)
        R.check(got, ref, mag, K_HEADS, "heads")
    assert torch.equal(b.heads[2].cpu().double(), R.heads(v, None, 0, 0.0, None, False, b.flags, F, S)[0])
    geo = oracle.Geometry(F, Hs, Ws, wf=1, ws=9, bkv=128)
    for i in range(H):  # the oracle takes and gives every head in (F,H,W) order
        kind = oracle.TEMPORAL_PERMUTED if b.flags[i] else oracle.SPATIAL
        rows = R.rows_of(F, S, bool(b.flags[i]))
        ref, _ = oracle.attention(*(W.bf16_bits(t[i].cpu()[rows]) for t in b.heads), kind, geo)
        assert np.abs(b.O[i].float().cpu().numpy() - ref).max() <= 1e-2
    o = R.residual_norm(b.x.cpu(), b.y.cpu(), m[:, 2], m[:, 4], m[:, 3], group=S)
    R.check(b.r, o["r"], o["rmag"], K_R, "r")
    R.check(b.h2, o["h"], o["hmag"], K_H, "h2")


@pytest.mark.gpu
def test_block_backward_stage_by_stage(bss):
    """The backward calls on what the forward calls kept (their own statistics and
    rounded stream), the first norm's gradient added to the stream's in place."""
    b = Block(bss)
    with bss.build_tile_map(b.p) as tm:
        b.forward(bss, tm)
    g = torch.Generator().manual_seed(4)
    bf = torch.bfloat16
    dh2, dr2 = (torch.randn(N, C, generator=g).to(bf).to(DEV) for _ in range(2))
    dheads = [torch.randn(H, N, d, generator=g).to(bf).to(DEV) for _ in range(3)]
    m = b.mod
    dx, dy = torch.empty_like(b.x), torch.empty_like(b.x)
    dm = [torch.empty(F, C, device=DEV) for _ in range(5)]
    bss.residual_norm_backward(b.r, b.y, dr=dr2, dh=dh2, dx=dx, dy=dy, stats=b.st2, gate=m[:, 2], scale=m[:, 4],
                               dgate=dm[2], dshift=dm[3], dscale=dm[4], rows_per_group=S)
    dqkv = torch.zeros(N, 3, H, d, dtype=bf, device=DEV)
    dw = [torch.empty(C, device=DEV) for _ in range(2)]
    q, k, v = b.qkv.view(N, 3, H, d).unbind(1)
    bss.heads_from_tokens_backward(*dheads, *dqkv.unbind(1), b.p, b.fl, q=q, k=k, dq_weight=dw[0], dk_weight=dw[1], **b.kw)
    dh = dqkv.view(N, 3 * C) @ b.w_qkv.t()
    before = dx.clone()
    # the norm in front of the block: its gradient on top of the residual's, in place
    bss.residual_norm_backward(b.x, dr=dx, dh=dh, dx=dx, stats=b.st, scale=m[:, 1], dshift=dm[0], dscale=dm[1],
                               rows_per_group=S)
    torch.cuda.synchronize()
    cpu = lambda *t: [x.cpu() for x in t]  # noqa: E731
    r, y, dr_, dh_, st2 = cpu(b.r, b.y, dr2, dh2, b.st2)
    ref = R.residual_norm_grad(r, y, dr_, dh_, st2, gate=m[:, 2].cpu(), scale=m[:, 4].cpu(), group=S)
    R.check(before, *ref["dx"], K_DX, "dx")
    R.check(dy, *ref["dy"], K_DX, "dy")
    for i, name in ((2, "dgate"), (3, "dshift"), (4, "dscale")):
        R.check(dm[i], *ref[name], K_SUM, name)
    ang = R.angles(b.tabs, (0, 0, 0), F, Hs, Ws)
    for i, (x, w) in enumerate(((q, b.wq), (k, b.wk))):
        ref_, mag, rw, rwmag = R.heads_grad(dheads[i].double().cpu(), x.double().cpu(), w.cpu(), 2, 1e-6, ang, False,
                                            b.flags, F, S)
        R.check(dqkv[:, i], ref_, mag, K_GRAD, "dqk")
        R.check(dw[i], rw, rwmag, 300, "dw")
    x, dr_, dh_, st = cpu(b.x, before, dh, b.st)
    ref = R.residual_norm_grad(x, None, dr_, dh_, st, scale=m[:, 1].cpu(), group=S)
    R.check(dx, *ref["dx"], K_DX, "dx of the first norm")
    R.check(dm[0], *ref["dshift"], K_SUM, "dshift")
    R.check(dm[1], *ref["dscale"], K_SUM, "dscale")

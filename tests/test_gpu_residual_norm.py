"""residual_norm and its gradient against 64-bit references."""
import subprocess
import sys
from pathlib import Path

import pytest
import torch

import _block_ref as R

DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32
# Longest 32-bit chains: a row's sum adds up to 40 values a lane in a row, 5 steps
# over the lanes and 8 over the warps; r inherits the branch norm's two sums, h
# those and its own two.
K_R, K_H = 128, 256
# dx has two sums behind it, dy two more; a column's sum over the rows adds at most
# a few hundred rows one after the other.
K_DX, K_DY, K_SUM = 192, 384, 512

# rows, channels, rows per group, stream, branch, params, norm, y_norm, parts given
CASES = {
    "one_row": (1, 64, 1, BF, BF, F32, 1, 0, "y gate scale shift"),
    "norm_only": (37, 256, 37, BF, BF, BF, 1, 0, "scale shift"),
    "rms_weight": (19, 1280, 19, BF, BF, F32, 2, 0, "weight"),
    "frames": (103, 1280, 25, BF, BF, F32, 1, 0, "y gate scale shift"),
    "sandwich": (65, 1000, 13, F32, BF, BF, 2, 1, "y gate scale shift weight y_weight"),
    "all_float": (50, 520, 50, F32, F32, F32, 1, 2, "y gate scale shift weight bias y_weight"),
    "per_row_groups": (23, 136, 1, BF, BF, BF, 1, 1, "y gate scale shift weight bias"),
    "layer_scale_only": (33, 640, 33, F32, BF, F32, 2, 0, "y y_weight"),
    "plain_residual": (33, 72, 11, BF, BF, F32, 1, 0, "y"),
    "no_norm": (21, 320, 7, F32, F32, BF, 0, 0, "y gate scale shift"),
    "five_warps": (40, 1288, 40, BF, BF, F32, 1, 2, "y gate weight bias"),
    "long_row": (9, 5000, 4, F32, F32, F32, 1, 1, "y gate scale shift weight bias y_weight"),
    "longest_row": (5, 8192, 2, BF, BF, BF, 1, 2, "y gate scale shift weight bias y_weight"),
    "smallest_row": (300, 8, 100, BF, BF, F32, 2, 0, "y gate scale shift"),
    # the shapes whose slots fill shared memory furthest
    "wide_stream": (11, 4096, 4, F32, BF, F32, 1, 0, "y gate scale shift"),
    "widest_stream": (5, 8192, 2, F32, BF, F32, 1, 0, "y gate scale shift weight bias"),
    "widest_float": (9, 8192, 9, F32, F32, F32, 1, 1, "y gate scale shift weight bias y_weight"),
    "many_rows": (2011, 512, 301, BF, BF, F32, 1, 0, "y gate scale shift weight bias"),
}


class Case:
    def __init__(self, name, seed=0):
        rows, C, group, sd, bd, pd, norm, y_norm, parts = CASES[name]
        g = torch.Generator().manual_seed(seed + 1)
        G = -(-rows // group)
        self.rows, self.C, self.G, self.sd, self.bd = rows, C, G, sd, bd
        self.kw = dict(norm=norm, y_norm=y_norm)
        self.group, self.a = group, (0.5 if "y" in parts.split() else 1.0)
        v = {"x": (torch.randn(rows, C, generator=g) * 2 + 0.7).to(sd)}
        for k in parts.split():
            if k == "y":
                v[k] = (torch.randn(rows, C, generator=g) - 0.3).to(bd)
            elif k in ("gate", "scale", "shift"):
                v[k] = (torch.randn(G, C, generator=g) * 0.5).to(pd)
            else:
                v[k] = (torch.randn(C, generator=g) * 0.3 + 1).to(pd)
        self.v = v
        self.dev = {k: t.to(DEV) for k, t in v.items()}
        self.ref = R.residual_norm(**v, **self.kw, group=group, a=self.a, eps=1e-6)
        self.call = dict(rows_per_group=group, residual_scale=self.a, **self.kw)

    def forward(self, bss, **kw):
        out = {"r": torch.full((self.rows, self.C), -7.0, dtype=self.sd, device=DEV) if "y" in self.v else None,
               "h": torch.full((self.rows, self.C), -7.0, dtype=self.bd, device=DEV),
               "stats": torch.full((self.rows, 2), -7.0, device=DEV) if self.kw["norm"] else None,
               "y_stats": torch.full((self.rows, 2), -7.0, device=DEV) if self.kw["y_norm"] else None}
        bss.residual_norm(**self.dev, **out, **self.call, eps=1e-6, **kw)
        return out

    def grads(self):
        """Upstream gradients and the reference of every gradient, from the statistics as stored."""
        g = torch.Generator().manual_seed(11)
        dh = torch.randn(self.rows, self.C, generator=g).to(self.bd)
        dr = torch.randn(self.rows, self.C, generator=g).to(self.sd) if "y" in self.v else None
        r = (self.ref["r"] if "y" in self.v else self.v["x"]).to(self.sd)
        stats = torch.cat((self.ref["mean"], self.ref["rstd"]), 1).float() if self.kw["norm"] else None
        ys = torch.cat((self.ref["ymean"], self.ref["yrstd"]), 1).float() if self.kw["y_norm"] else None
        p = {k: t for k, t in self.v.items() if k not in ("x", "shift")}
        ref = R.residual_norm_grad(r, dr=dr, dh=dh, stats=stats, y_stats=ys, group=self.group, a=self.a, **self.kw, **p)
        ins = {"r": r, "dr": dr, "dh": dh, "stats": stats, "y_stats": ys, **p}
        return {k: t.to(DEV) for k, t in ins.items() if t is not None}, ref

    def grad_outputs(self):
        out = {"dx": torch.full((self.rows, self.C), -7.0, dtype=self.sd, device=DEV)}
        if "y" in self.v:
            out["dy"] = torch.full((self.rows, self.C), -7.0, dtype=self.bd, device=DEV)
            out["dgate"] = torch.full((self.G, self.C), -7.0, device=DEV)
            out["dy_weight"] = torch.full((self.C,), -7.0, device=DEV)
        for k in ("dscale", "dshift"):
            out[k] = torch.full((self.G, self.C), -7.0, device=DEV)
        for k in ("dweight", "dbias"):
            out[k] = torch.full((self.C,), -7.0, device=DEV)
        return out


@pytest.mark.gpu
@pytest.mark.parametrize("name", CASES)
def test_forward(bss, name):
    c = Case(name)
    out = c.forward(bss)
    torch.cuda.synchronize()
    if out["r"] is not None:
        R.check(out["r"], c.ref["r"], c.ref["rmag"], K_R, f"{name} r")
    R.check(out["h"], c.ref["h"], c.ref["hmag"], K_H, f"{name} h")
    if out["stats"] is not None:
        R.check(out["stats"][:, :1], c.ref["mean"], c.ref["rmag"].mean(1, keepdim=True), K_H, f"{name} mean")
        # the deviation inherits the errors of the values under it
        spread = c.ref["rstd"] * (1 + (c.ref["rmag"] * c.ref["rstd"]).mean(1, keepdim=True))
        R.check(out["stats"][:, 1:], c.ref["rstd"], spread, K_H, f"{name} rstd")
    if out["y_stats"] is not None:
        y = c.v["y"].double()
        R.check(out["y_stats"][:, :1], c.ref["ymean"], y.abs().mean(1, keepdim=True), K_R, f"{name} ymean")
        R.check(out["y_stats"][:, 1:], c.ref["yrstd"], c.ref["yrstd"] * 2, K_R, f"{name} yrstd")


@pytest.mark.gpu
@pytest.mark.parametrize("name", CASES)
def test_backward(bss, name):
    c = Case(name)
    ins, ref = c.grads()
    out = c.grad_outputs()
    bss.residual_norm_backward(**ins, **out, **c.call)
    torch.cuda.synchronize()
    for k, t in out.items():
        value, mag = ref[k]
        K = K_DX if k == "dx" else K_DY if k == "dy" else K_SUM
        R.check(t, value, mag, K, f"{name} {k}")
    again = c.grad_outputs()
    bss.residual_norm_backward(**ins, **again, **c.call)
    assert all(torch.equal(out[k], again[k]) for k in out)
    # each gradient alone, and none: the same values
    for k in list(out)[1:]:
        if k == "dy":
            continue
        some = {n: t for n, t in c.grad_outputs().items() if n in ("dx", "dy", k)}
        bss.residual_norm_backward(**ins, **some, **c.call)
        R.check(some[k], *ref[k], K_SUM, f"{name} {k} alone")
        assert torch.equal(some["dx"], out["dx"])


@pytest.mark.gpu
@pytest.mark.parametrize("name", ["frames", "sandwich", "all_float"])
def test_backward_of_one_side(bss, name):
    """Only dr (nothing uses h), and only dh (the last block)."""
    c = Case(name)
    for drop in ("dh", "dr"):
        ins, _ = c.grads()
        del ins[drop]
        cpu = {k: t.cpu() for k, t in ins.items()}
        ref = R.residual_norm_grad(**cpu, group=c.group, a=c.a, **c.kw)
        out = c.grad_outputs()
        if drop == "dh":
            for k in ("dscale", "dshift", "dweight", "dbias"):
                del out[k]
        bss.residual_norm_backward(**ins, **out, **c.call)
        for k, t in out.items():
            R.check(t, *ref[k], K_DX if k == "dx" else K_DY if k == "dy" else K_SUM, f"{name} without {drop}: {k}")


@pytest.mark.gpu
@pytest.mark.parametrize("name", ["frames", "sandwich", "long_row"])
def test_strided_and_in_place(bss, name):
    c = Case(name)
    want = c.forward(bss)
    C = c.C

    def strided(t):  # rows inside a wider tensor
        buf = torch.full((t.shape[0], C + 24), -7.0, dtype=t.dtype, device=DEV)
        buf[:, 8:8 + C] = t
        return buf, buf[:, 8:8 + C]
    xb, x = strided(c.dev["x"])
    yb, y = strided(c.dev["y"])
    mods = {}
    packed = [c.dev[k] for k in ("gate", "scale", "shift") if k in c.dev]
    if packed:
        m = torch.stack(packed, 1)  # [groups][3][channels], as a modulation layer makes them
        mods = {k: m[:, i] for i, k in enumerate(k for k in ("gate", "scale", "shift") if k in c.dev)}
    rest = {k: t for k, t in c.dev.items() if k not in ("x", "y", "gate", "scale", "shift")}
    rb, r = strided(torch.full_like(c.dev["x"], 3.0))
    hb, h = strided(torch.full_like(c.dev["y"], 3.0))
    bss.residual_norm(x, y, r, h, **mods, **rest, **c.call)
    assert torch.equal(r, want["r"]) and torch.equal(h, want["h"])
    bss.residual_norm(x, y, x, y, **mods, **rest, **c.call)  # r over x, h over y
    torch.cuda.synchronize()
    assert torch.equal(x, want["r"]) and torch.equal(y, want["h"])
    for b in (xb, yb, rb, hb):
        assert torch.all(b[:, :8] == -7.0) and torch.all(b[:, 8 + C:] == -7.0)
    # two views of one tensor that share no byte
    both = torch.full((c.rows, 2 * C), -7.0, dtype=c.sd, device=DEV)
    both[:, :C] = c.dev["x"]
    bss.residual_norm(both[:, :C], c.dev["y"], both[:, C:], None, **{k: t for k, t in mods.items() if k == "gate"},
                      **{k: t for k, t in rest.items() if k == "y_weight"}, rows_per_group=c.group,
                      residual_scale=c.a, norm=bss.NORM_NONE, y_norm=c.kw["y_norm"])
    assert torch.equal(both[:, C:], want["r"])
    # backward: dx over dr, dy over dh
    ins, _ = c.grads()
    out = c.grad_outputs()
    bss.residual_norm_backward(**ins, **out, **c.call)
    over = {**c.grad_outputs(), "dx": ins["dr"], "dy": ins["dh"]}
    bss.residual_norm_backward(**ins, **over, **c.call)
    assert all(torch.equal(out[k], over[k]) for k in out)


@pytest.mark.gpu
def test_writes_only_its_outputs(bss):
    c = Case("frames")
    G = 4096

    def guarded(shape, dtype):
        n = shape[0] * (shape[1] if len(shape) > 1 else 1)
        buf = torch.full((n + 2 * G,), -7.0, dtype=dtype, device=DEV)
        return buf, buf[G:G + n].view(*shape)
    ins, _ = c.grads()
    outs = {k: guarded(tuple(t.shape), t.dtype) for k, t in c.grad_outputs().items()}
    ws = torch.full((1 << 22,), 171, dtype=torch.uint8, device=DEV)
    keep = {k: t.clone() for k, t in {**ins, **c.dev}.items()}
    bss.residual_norm_backward(**ins, **{k: t for k, (_, t) in outs.items()}, **c.call, workspace=ws[:1 << 21])
    r = guarded((c.rows, c.C), c.sd)
    h = guarded((c.rows, c.C), c.bd)
    st = guarded((c.rows, 2), F32)
    bss.residual_norm(**c.dev, r=r[1], h=h[1], stats=st[1], **c.call)
    torch.cuda.synchronize()
    for b, t in list(outs.values()) + [r, h, st]:
        assert torch.all(b[:G] == -7.0) and torch.all(b[-G:] == -7.0)
    assert torch.all(ws[1 << 21:] == 171)
    assert all(torch.equal(keep[k], t) for k, t in {**c.dev, **ins}.items())


@pytest.mark.gpu
def test_nonfinite_rows_and_constant_rows(bss):
    c = Case("norm_only")
    want = c.forward(bss)["h"]
    x = c.dev["x"].clone()
    x[3, 7] = float("inf")
    x[8] = float("nan")
    x[5] = 1.5   # no spread: the norm is 0
    x[6] = 0.0
    h = torch.empty_like(x)
    bss.residual_norm(x, h=h, scale=c.dev["scale"], shift=c.dev["shift"], **c.call)
    rows = [i for i in range(c.rows) if i not in (3, 8, 5, 6)]
    assert torch.equal(h[rows], want[rows])
    assert torch.isnan(h[8]).all() and not torch.isfinite(h[3]).all()
    for row in (5, 6):
        assert torch.equal(h[row], c.dev["shift"][0])


@pytest.mark.gpu
@pytest.mark.parametrize("stream", [BF, F32])
@pytest.mark.parametrize("y_norm", [0, 2])
def test_infinite_stream_without_a_norm(bss, stream, y_norm):
    """Without a norm dx and dy do not depend on r: they stay what they are next to its infinities."""
    rows, C = 9, 264
    g = torch.Generator().manual_seed(5)
    v = {k: torch.randn(rows, C, generator=g).to(BF).to(DEV) for k in ("y", "dh")}
    r, dr = (torch.randn(rows, C, generator=g).to(stream).to(DEV) for _ in range(2))
    ys = torch.stack((torch.zeros(rows), torch.rand(rows, generator=g) + 0.5), 1).to(DEV) if y_norm else None
    got = []
    for value in (1.0, float("inf"), float("-inf"), float("nan")):
        r[2, 5], r[7, 263] = value, value
        dx, dy = torch.empty_like(r), torch.empty_like(v["y"])
        bss.residual_norm_backward(r, dr=dr, dx=dx, dy=dy, y_stats=ys, norm=0, y_norm=y_norm, **v)
        got.append((dx.clone(), dy.clone()))
    torch.cuda.synchronize()
    assert torch.isfinite(got[0][0]).all() and torch.isfinite(got[0][1]).all()
    for dx, dy in got[1:]:
        assert torch.equal(dx, got[0][0]) and torch.equal(dy, got[0][1])


FIRST_CALL = """
import torch
import block_sparse_spatio_gb300 as bss
x = torch.randn(16, {channels}, device="cuda").to(torch.{stream})
mods = dict(zip(("scale", "shift", "gate"), torch.zeros(3, 1, {channels}, device="cuda")[:{folds}]))
y = torch.zeros({channels}, device="cuda").to(torch.{branch}).expand(16, -1) if {folds} > 2 else None
h = torch.empty(16, {channels}, device="cuda", dtype=torch.{branch})
bss.residual_norm(x, y=y, h=h, **mods)
ref = torch.nn.functional.layer_norm(x.double(), ({channels},), eps=1e-6)
assert (h.double() - ref).abs().max() <= 2.0 ** -8 * ref.abs().max() + 1e-4
print("ran")
"""
# Calls whose dynamic shared memory alone just fits 48 KiB, with static memory no
# longer.  Each is its process's first: a larger call before it would have raised
# the kernel's limit.  channels, stream, branch, vectors folded
FIRST_CALLS = [(2048, "float32", "float32", 0), (1536, "float32", "bfloat16", 2), (2048, "bfloat16", "bfloat16", 3),
               (1024, "bfloat16", "bfloat16", 2)]


@pytest.mark.gpu
@pytest.mark.parametrize("channels,stream,branch,folds", FIRST_CALLS)
def test_first_call_of_a_process(channels, stream, branch, folds):
    code = FIRST_CALL.format(channels=channels, stream=stream, branch=branch, folds=folds)
    out = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True,
                         timeout=300, cwd=Path(__file__).resolve().parents[1])
    assert out.returncode == 0 and "ran" in out.stdout, out.stderr[-600:]


@pytest.mark.gpu
def test_large_means_keep_the_deviation(bss):
    """A row far from zero: the variance is about the mean, not a difference of squares."""
    g = torch.Generator().manual_seed(2)
    x = 3000.0 + torch.randn(16, 1280, generator=g)
    h = torch.empty(16, 1280, device=DEV)
    bss.residual_norm(x.to(DEV), h=h)
    ref = R.residual_norm(x)["h"]
    # x - mean is exact to half an ulp of 3000 (2^-13) plus the mean's own rounding
    assert (h.cpu().double() - ref).abs().max() <= 4 * 2.0 ** -13


@pytest.mark.gpu
def test_other_stream_and_two_captured_graphs(bss):
    c = Case("frames")
    want = c.forward(bss)
    ins, _ = c.grads()
    ref = c.grad_outputs()
    bss.residual_norm_backward(**ins, **ref, **c.call)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    out = c.grad_outputs()
    torch.cuda.synchronize()
    got = None
    with torch.cuda.stream(s):
        got = c.forward(bss)
    bss.residual_norm_backward(**ins, **out, **c.call, stream=s)
    s.synchronize()
    assert torch.equal(got["h"], want["h"]) and all(torch.equal(out[k], ref[k]) for k in ref)
    sets = []
    for _ in range(2):
        out = c.grad_outputs()
        h, r = torch.zeros_like(want["h"]), torch.zeros_like(want["r"])
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            bss.residual_norm(**c.dev, r=r, h=h, **c.call)
            bss.residual_norm_backward(**ins, **out, **c.call)
        sets.append((graph, out, h, r))
    for _ in range(3):
        for x in sets:
            x[0].replay()
    torch.cuda.synchronize()
    for _, out, h, r in sets:
        assert torch.equal(h, want["h"]) and torch.equal(r, want["r"])
        assert all(torch.equal(out[k], ref[k]) for k in ref)


@pytest.mark.gpu
def test_offsets_past_32_bits(bss):
    """More than 2^32 bytes in one tensor: the first and the last rows."""
    rows, C = 302400, 7200
    x = torch.empty(rows, C, dtype=BF, device=DEV)
    assert x.numel() * 2 > 1 << 32
    for i in range(0, rows, 30240):
        x[i:i + 30240] = torch.randn(30240, C, device=DEV).to(BF)
    h, st = torch.empty_like(x), torch.empty(rows, 2, device=DEV)
    mod = torch.randn(21, 2, C, device=DEV) * 0.3
    bss.residual_norm(x, h=h, scale=mod[:, 0], shift=mod[:, 1], rows_per_group=rows // 21, stats=st)
    at = torch.tensor([0, 1, rows // 2, rows - 2, rows - 1])
    G = (at // (rows // 21)).tolist()
    cpu = x[at].cpu()
    o = R.residual_norm(cpu, scale=mod[G, 0].cpu(), shift=mod[G, 1].cpu(), group=1)
    R.check(h[at], o["h"], o["hmag"], K_H)
    dx, dscale = torch.empty_like(x), torch.empty(21, C, device=DEV)
    bss.residual_norm_backward(x, dh=h, dx=dx, stats=st, scale=mod[:, 0], rows_per_group=rows // 21, dscale=dscale)
    ref = R.residual_norm_grad(cpu, dh=h[at].cpu(), stats=st[at].cpu(), scale=mod[G, 0].cpu(), group=1)
    R.check(dx[at], *ref["dx"], K_DX)
    last = slice(rows - rows // 21, rows)
    xh = (x[last].double() - st[last, :1].double()) * st[last, 1:].double()
    t = h[last].double() * xh
    # a group's 14400 rows: chunks of a few hundred added in a row
    R.check(dscale[-1], t.sum(0), t.abs().sum(0), K_SUM)

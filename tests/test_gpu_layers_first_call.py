"""The matrix products and the cross attention captured into a graph by their very first
calls, in a process of their own, in each of their forms."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

SCRIPT = r"""
import torch
import block_sparse_spatio_gb300 as bss
BF = torch.bfloat16
torch.manual_seed(0)
r = lambda *s: torch.randn(*s, device="cuda").to(BF)
calls = []
# few rows, tiles, joined by a cluster, summed from memory, pairs of CTAs
for rows, inner, outer in ((3, 64, 72), (130, 72, 136), (130, 3000, 264), (50, 4096, 72), (20003, 72, 1032), (12001, 1288, 1288)):
    x, w, d = r(rows, inner), r(outer, inner), r(rows, outer)
    def linear(x=x, w=w, d=d, rows=rows, inner=inner, outer=outer):
        out, pre = (torch.zeros(rows, outer, device="cuda", dtype=BF) for _ in range(2))
        dx, dw, db = torch.zeros_like(x), torch.zeros_like(w), torch.zeros(outer, device="cuda")
        bss.linear(x, w, out, activation=bss.ACT_SILU, residual=d, pre=pre)
        bss.linear_backward(d, x, w, dx, dw, db, activation=bss.ACT_SILU, pre=pre)
        return out, pre, dx, dw, db
    calls.append(linear)
for rows, group, H, keys, dim in ((1, 1, 4, 300, 64), (700, 300, 10, 300, 128), (3000, 77, 8, 150, 64)):
    G = -(-rows // group)
    q, k, v, d = r(rows, H, dim), r(G, keys, H, dim), r(G, keys, H, dim), r(rows, H, dim)
    lengths = torch.tensor([keys - i % 5 for i in range(G)], device="cuda", dtype=torch.int32)
    def cross(q=q, k=k, v=v, d=d, lengths=lengths, group=group):
        O, lse = torch.zeros_like(q), torch.zeros(q.shape[1], q.shape[0], device="cuda")
        dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
        bss.cross_attention(q, k, v, O, lengths=lengths, lse=lse, rows_per_group=group)
        bss.cross_attention_backward(d, q, k, v, O, lse, dq, dk, dv, lengths=lengths, rows_per_group=group)
        return O, lse, dq, dk, dv
    calls.append(cross)
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    kept = [f() for f in calls]
for _ in range(2):
    graph.replay()
torch.cuda.synchronize()
for f, outs in zip(calls, kept):
    for a, b in zip(f(), outs):
        assert torch.equal(a, b)
assert bss.get_device_status() == 0
print("same bits")
"""


def test_first_calls_captured():
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    env = dict(os.environ, PYTHONPATH=root)
    p = subprocess.run([sys.executable, "-c", SCRIPT], cwd=root, env=env, capture_output=True, text=True, timeout=300)
    assert p.returncode == 0 and "same bits" in p.stdout, p.stdout + p.stderr

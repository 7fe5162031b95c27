"""The matrix products and the cross attention on the GPU with inputs that are repeated
(strides of 0, as torch's expand gives them) or given twice, and called by threads at once."""
import threading

import pytest
import torch

import _layers_ref as L
from _block_ref import check
from test_gpu_linear import BF, DEV, F32, rnd

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows,inner,outer", [(5, 96, 136), (130, 96, 136), (130, 3000, 264), (50, 4096, 72), (20003, 72, 1032)])
@pytest.mark.parametrize("out", [BF, F32])
def test_linear(bss, rows, inner, outer, out):
    g = torch.Generator().manual_seed(1)
    group = max(1, rows // 3)
    G = -(-rows // group)
    x, w = rnd(g, 1, inner, dtype=BF).expand(rows, inner), rnd(g, outer, inner, dtype=BF, scale=inner ** -0.5)
    gate, r, d = (rnd(g, 1, outer, dtype=t) for t in (F32, out, BF))
    pre = rnd(g, 1, outer, dtype=BF)
    o = torch.empty(rows, outer, dtype=out, device=DEV)
    far = lambda t, n: t.to(DEV).expand(n, -1)  # noqa: E731
    xd = far(x[:1], rows)
    bss.linear(xd, w.to(DEV), o, gate=far(gate, G), residual=far(r, rows), rows_per_group=group, activation=2)
    check(o, *L.linear(x, w, None, 2, gate.expand(G, -1), r.expand(rows, -1), group)["out"], 1, "out")
    dx, dw = torch.empty(rows, inner, dtype=BF, device=DEV), torch.empty(outer, inner, device=DEV)
    db, dg = torch.empty(outer, device=DEV), torch.empty(G, outer, device=DEV)
    bss.linear_backward(far(d, rows), xd, w.to(DEV), dx, dw, db, dg, activation=2, pre=far(pre, rows), gate=far(gate, G),
                        rows_per_group=group)
    ref = L.linear_grad(d.expand(rows, -1), x, w, pre.expand(rows, -1), 2, gate.expand(G, -1), group)
    for name, t in (("dx", dx), ("dweight", dw), ("dbias", db), ("dgate", dg)):
        check(t, *ref[name], 1, name)
    # without activation and gate dout is an operand of the products itself
    bss.linear_backward(far(d, rows), xd, w.to(DEV), dx, dw, db)
    ref = L.linear_grad(d.expand(rows, -1), x, w)
    for name, t in (("dx", dx), ("dweight", dw), ("dbias", db)):
        check(t, *ref[name], 1, name)
    assert bss.get_device_status() == 0


def test_one_tensor_given_twice(bss):
    g = torch.Generator().manual_seed(2)
    for rows in (16, 264):
        x = rnd(g, rows, rows, dtype=BF)
        xd, o = x.to(DEV), torch.empty(rows, rows, dtype=BF, device=DEV)
        bss.linear(xd, xd, o, residual=xd, activation=1)
        check(o, *L.linear(x, x, None, 1, None, x, rows)["out"], 1)
        dx, dw = torch.empty_like(o), torch.empty_like(o)
        bss.linear_backward(xd, xd, xd, dx, dw, activation=1, pre=xd)
        ref = L.linear_grad(x, x, x, x, 1)
        check(dx, *ref["dx"], 1)
        check(dw, *ref["dweight"], 1)
    for rows in (6, 300):  # self attention without a mask
        q = rnd(g, rows, 2, 64, dtype=BF)
        qd = q.to(DEV)
        O, lse = torch.empty_like(qd), torch.empty(2, rows, device=DEV)
        bss.cross_attention(qd, qd, qd, O, lse=lse)
        check(O, *L.cross(q, q[None], q[None], [rows], rows)["O"], 1)
        outs = [torch.empty_like(qd) for _ in range(3)]
        bss.cross_attention_backward(qd, qd, qd, qd, O, lse, *outs)
        ref = L.cross_grad(q, q, q[None], q[None], O.cpu(), lse.cpu(), [rows], rows)
        check(outs[0], *ref["dq"], 1)
        check(outs[1], ref["dk"][0][0], ref["dk"][1][0], 1)
        check(outs[2], ref["dv"][0][0], ref["dv"][1][0], 1)
    assert bss.get_device_status() == 0


def test_threads_at_once(bss):
    """Calls of several threads, each on a stream of its own, with the bits of one alone."""
    g = torch.Generator().manual_seed(3)
    x, w, d = (t.to(DEV) for t in (rnd(g, 700, 2048, dtype=BF), rnd(g, 264, 2048, dtype=BF, scale=0.02), rnd(g, 700, 264, dtype=BF)))
    q, k, v = (t.to(DEV) for t in (rnd(g, 900, 6, 64, dtype=BF), rnd(g, 3, 150, 2, 64, dtype=BF), rnd(g, 3, 150, 2, 64, dtype=BF)))

    def calls():
        o, pre = (torch.empty(700, 264, dtype=BF, device=DEV) for _ in range(2))
        dx, dw, db = torch.empty_like(x), torch.empty_like(w), torch.empty(264, device=DEV)
        bss.linear(x, w, o, activation=3, pre=pre)
        bss.linear_backward(d, x, w, dx, dw, db, activation=3, pre=pre)
        O, lse, dq, dk, dv = torch.empty_like(q), torch.empty(6, 900, device=DEV), torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
        bss.cross_attention(q, k, v, O, lse=lse, rows_per_group=300)
        bss.cross_attention_backward(O, q, k, v, O, lse, dq, dk, dv, rows_per_group=300)
        return o, pre, dx, dw, db, O, lse, dq, dk, dv

    want = calls()
    torch.cuda.synchronize()
    wrong = []

    def work():
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(20):
                got = calls()
                torch.cuda.current_stream().synchronize()
                if not all(torch.equal(a, b) for a, b in zip(got, want)):
                    wrong.append(1)

    threads = [threading.Thread(target=work) for _ in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not wrong and bss.get_device_status() == 0

"""residual_norm and its gradient in place where further row inputs are that same
tensor, against the same call on copies."""
import pytest
import torch

DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32


# one warp a row, several, and rows of the widest form
@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows,C,group", [(37, 520, 9), (23, 2056, 1), (5, 8192, 5)])
def test_same_tensor_in_place(bss, dtype, rows, C, group):
    g = torch.Generator().manual_seed(C)
    t = torch.randn(rows, C, generator=g).to(dtype).to(DEV)
    mod = (torch.randn(-(-rows // group), 3, C, generator=g) * 0.3).to(DEV)
    kw = dict(gate=mod[:, 0], scale=mod[:, 1], shift=mod[:, 2], rows_per_group=group, y_norm=bss.NORM_LAYER)
    r, h, st, ys = torch.empty_like(t), torch.empty_like(t), torch.empty(rows, 2, device=DEV), torch.empty(rows, 2, device=DEV)
    bss.residual_norm(t.clone(), t.clone(), r, h, stats=st, y_stats=ys, **kw)
    for over in ("r", "h"):
        x = t.clone()
        out = {"r": torch.empty_like(t), "h": torch.empty_like(t), over: x}
        bss.residual_norm(x, x, **out, **kw)
        assert torch.equal(out["r"], r) and torch.equal(out["h"], h)
    del kw["shift"]
    dh = torch.randn(rows, C, generator=g).to(dtype).to(DEV)
    kw.update(stats=st, y_stats=ys)

    def backward(r, y, dr, dh, dx, dy):
        bss.residual_norm_backward(r, y, dr=dr, dh=dh, dx=dx, dy=dy, **kw)
        return dx, dy
    new = lambda: torch.empty_like(t)  # noqa: E731
    want = backward(r.clone(), t.clone(), r.clone(), dh.clone(), new(), new())
    a = r.clone()
    got = backward(a, t.clone(), a, dh.clone(), a, new())          # dx over dr, which is r too
    assert all(torch.equal(x, y) for x, y in zip(got, want))
    want = backward(r.clone(), dh.clone(), r.clone(), dh.clone(), new(), new())
    b = dh.clone()
    got = backward(r.clone(), b, r.clone(), b, new(), b)           # dy over dh, which is y too
    assert all(torch.equal(x, y) for x, y in zip(got, want))
    want = backward(r.clone(), t.clone(), dh.clone(), dh.clone(), new(), new())
    c = dh.clone()
    got = backward(r.clone(), t.clone(), c, c, c, new())           # dx over dr, which is dh too
    assert all(torch.equal(x, y) for x, y in zip(got, want))

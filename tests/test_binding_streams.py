"""Memory that the binding takes itself belongs to the stream its kernels run on:
from another stream's it could still be in use there."""
import contextlib

import pytest
import torch

import block_sparse_spatio_gb300 as bss


class FakeStream:
    cuda_stream = 0x5000


class FakeLibrary:
    """Takes every call."""

    def __getattr__(self, name):
        return lambda *a: 0


def test_rotary_table_is_allocated_on_its_stream(monkeypatch):
    entered, at_empty = [], []
    given = FakeStream()

    @contextlib.contextmanager
    def stream(s):
        entered.append(s)
        yield
        entered.pop()
    empty = torch.empty
    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: -1)  # where CPU tensors are
    monkeypatch.setattr(torch, "empty", lambda *a, device=None, **kw: (at_empty.append(list(entered)), empty(*a, **kw))[1])
    monkeypatch.setattr(bss, "load", FakeLibrary)
    bss.rotary_table(4, 3, stream=given)
    assert at_empty == [[given]]
    own = empty(4, 3, 2)
    assert bss.rotary_table(4, 3, out=own, stream=given) is own and len(at_empty) == 1


@pytest.mark.gpu
@pytest.mark.parametrize("as_address", [False, True])
def test_rotary_table_takes_no_memory_of_the_current_stream(bss, as_address):
    s = torch.cuda.Stream()
    want = bss.rotary_table(4099, 21)
    torch.cuda.synchronize()
    freed = torch.empty_like(want)
    address = freed.data_ptr()
    del freed  # the current stream's again: kernels there may still use it
    got = bss.rotary_table(4099, 21, stream=s.cuda_stream if as_address else s)
    assert got.data_ptr() != address
    s.synchronize()
    assert torch.equal(got, want)

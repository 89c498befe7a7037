"""What the binding takes for an address, without a GPU."""
import enum

import numpy as np
import pytest
import torch

import token_indexed_sparse_staple_b200 as stp


ORIGINAL = stp._current_stream      # before any call has chosen


class Address(enum.IntEnum):
    A = 0x10000


def test_addresses():
    a = np.zeros(4, dtype=np.int32)
    t = torch.zeros(4)
    assert stp._p(None) is None
    assert stp._p(a) == a.ctypes.data and stp._p(t) == t.data_ptr()
    for v in (0x10000, np.int64(0x10000), Address.A):
        assert stp._p(v) == 0x10000


@pytest.mark.parametrize("v", [1.0, 65536.0, np.float32(2), "65536", b"65536", [65536], 0.1])
def test_what_is_no_address_is_refused(v):
    """A probability or a weight given in a tensor's place must not become an address."""
    with pytest.raises(TypeError):
        stp._p(v)
    with pytest.raises(TypeError):
        stp.make_drop(0.1, v)


class FakeStream:
    cuda_stream = 4242


@pytest.mark.parametrize("missing", [(), ("_cuda_getCurrentRawStream",), ("_cuda_getDevice",)])
def test_the_current_stream_with_and_without_private_lookups(monkeypatch, missing):
    monkeypatch.setattr(stp, "_current_stream", ORIGINAL)
    monkeypatch.setattr(torch.cuda, "init", lambda: None)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: FakeStream)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 3, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: 1000 + d, raising=False)
    for name in missing:
        monkeypatch.delattr(torch._C, name)
    for _ in range(2):      # the first call chooses, later ones use its choice
        assert stp._stream(None) == (4242 if missing else 1003)
    assert stp._stream(7) == 7 and stp._stream(FakeStream) == 4242

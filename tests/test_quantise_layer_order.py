"""quantise_layer on a stream of its own, without a GPU: its kernels come after what the
current stream holds (the weights, and earlier uses of the memory that the copy gets) and
before what the current stream does next."""
import pytest
import torch

import token_indexed_sparse_staple_b200 as stp
from token_indexed_sparse_staple_b200 import stack


class FakeStream:
    def __init__(self, name, log):
        self.name, self.log = name, log

    def wait_stream(self, other):
        self.log.append((self.name, "waits for", other.name))


@pytest.fixture
def log(monkeypatch):
    log = []
    current = FakeStream("current", log)
    empty = torch.empty

    def on_the_host(*a, device=None, **kw):
        log.append(("current", "allocates", None))
        return empty(*a, **kw)

    monkeypatch.setattr(torch, "empty", on_the_host)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: current)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda h: FakeStream(f"handle {h}", log))
    monkeypatch.setattr(stp, "staple_quant_rows",
                        lambda *a, stream=None: log.append((getattr(stream, "name", "current"),
                                                            "quantises", a[2:4])))
    return log


def weights():
    z = torch.zeros
    return stack.LayerWeights(z(32, 16), z(32, 16), z(16, 32))


@pytest.mark.parametrize("raw", [False, True])
def test_a_side_stream_waits_and_is_waited_for(log, raw):
    side = 77 if raw else FakeStream("handle 77", log)
    out = stack.quantise_layer(None, weights(), stream=side)
    assert out.w_gate_up.shape == (64, 16) and out.w_down.shape == (16, 32)
    work = [i for i, e in enumerate(log) if e[1] == "quantises"]
    assert [log[i] for i in work] == [("handle 77", "quantises", (32, 16))] * 2 + [
        ("handle 77", "quantises", (16, 32))]
    before, after = log[:work[0]], log[work[-1] + 1:]
    fork = ("handle 77", "waits for", "current")
    assert fork in before and ("current", "waits for", "handle 77") in after
    assert all(e[1] != "allocates" for e in log[before.index(fork):])


def test_the_current_stream_waits_for_nothing(log):
    stack.quantise_layer(None, weights())
    assert {e[0] for e in log} == {"current"}
    assert not [e for e in log if e[1] == "waits for"]

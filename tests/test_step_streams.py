"""Whose memory a call allocates where it runs on a stream of its own.  The kernels of a call with
`stream` wait for nothing that is queued on the current stream, so their buffers must not come from the current
stream's part of the allocator.  Fakes instead of a GPU."""
import contextlib

import pytest
import torch

from lora_fine_tuning_mlp_b200 import api


class Stream:
    device = None


class Buffer:
    def __init__(self, stream):
        self.allocated, self.recorded, self.device = stream, set(), None

    def record_stream(self, stream):
        self.recorded.add(stream)

    def numel(self):
        return 1024


@pytest.fixture
def streams(monkeypatch):
    """The current stream and another; torch.empty says which was current."""
    now = [Stream()]

    @contextlib.contextmanager
    def on(stream):
        now.append(stream)
        yield
        now.pop()

    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: now[-1])
    monkeypatch.setattr(torch, "empty", lambda *a, **kw: Buffer(now[-1]))
    return now[0], Stream()


def test_scratch_of_one_call(streams):
    here, other = streams
    buf = api._scratch(None, 1024, None, other)
    assert buf.allocated is other
    assert api._scratch(None, 1024, None, None).allocated is here


def test_a_workspace_that_grows(streams):
    here, other = streams
    ws = api.Workspace()
    assert api._scratch(ws, 1024, None, other).allocated is other
    ws = api.Workspace()
    first = api._scratch(ws, 1024, None, None)
    assert first.allocated is here
    again = api._scratch(ws, 1024, None, other)      # kept from a call on the current stream
    assert again is first and other in again.recorded


def test_results(streams):
    here, other = streams
    out = api._allocate(other, lambda: torch.empty(4))
    assert out.allocated is other and here in out.recorded
    assert api._allocate(None, lambda: torch.empty(4)).allocated is here


def test_calls_of_the_dense_layers(streams):
    here, other = streams
    ws = api.Workspace()

    @api._allocates_for_its_stream
    def call(n, *, workspace=None, stream=None):
        return torch.empty(n), {"a": torch.empty(n), "none": None}, workspace.get(n, None)

    y, grads, buf = call(4, workspace=ws, stream=other)
    assert all(t.allocated is other and here in t.recorded for t in (y, grads["a"], buf))
    y, grads, again = call(4, workspace=ws)
    assert y.allocated is here and not y.recorded and again is buf


@pytest.mark.parametrize("name", ["forward", "backward", "linear_forward", "linear_backward", "rmsnorm_forward",
                                  "rmsnorm_backward", "block_forward", "block_backward", "ce_forward", "ce_backward",
                                  "ce_loss", "ce_backward_reduced"])
def test_every_one_of_them_does(name):
    assert getattr(api, name).__name__ == name and hasattr(getattr(api, name), "__wrapped__")

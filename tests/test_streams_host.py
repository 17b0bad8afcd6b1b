"""Which waits the binding queues when a call runs on a stream other than the
current one: host logic, with the streams, the allocator's record and the
entry replaced by recorders."""
import pytest
import torch

from transformer_head_scaled_sdpa_gb300 import binding

CURRENT = 7


class Recorder:
    def __init__(self, monkeypatch):
        self.events = events = []

        class Stream:
            def __init__(self, handle, device=None):
                self.cuda_stream = handle

            def wait_stream(self, other):
                events.append(("wait", self.cuda_stream, other.cuda_stream))

        class Tensor:
            def record_stream(self, stream):
                events.append(("record", stream.cuda_stream))

        def entry(*args):
            events.append(("call", args[-1]))
            return 0

        self.Stream, self.Tensor, self.entry = Stream, Tensor, entry
        monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: CURRENT, raising=False)
        monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
        monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: Stream(CURRENT))
        monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: Stream(0))

        def external(handle, device=None):
            assert handle, "handle 0 makes ExternalStream take a stream from its pool"
            return Stream(handle)

        monkeypatch.setattr(torch.cuda, "ExternalStream", external)

    def call(self, stream, made):
        binding._call_on(0, stream, made, self.entry, (1, 2))
        return self.events


@pytest.fixture
def rec(monkeypatch):
    return Recorder(monkeypatch)


@pytest.mark.parametrize("handle", [9, 0])
@pytest.mark.parametrize("as_int", [True, False], ids=["handle", "object"])
def test_other_stream_waits_before_the_call(rec, handle, as_int):
    """Memory from the current stream's pool may still be in use by what was
    queued there: the other stream waits for it, then the entry is called."""
    events = rec.call(handle if as_int else rec.Stream(handle), [rec.Tensor(), rec.Tensor()])
    assert events == [("wait", handle, CURRENT), ("record", handle), ("record", handle), ("call", handle)]


@pytest.mark.parametrize("stream", [None, CURRENT], ids=["default", "same"])
def test_current_stream_waits_for_nothing(rec, stream):
    assert rec.call(stream, [rec.Tensor()]) == [("call", CURRENT)]


def test_callers_buffers_need_no_wait(rec):
    """With every buffer the caller's own, streams stay independent."""
    assert rec.call(9, []) == [("call", 9)]


@pytest.mark.parametrize("handle", [9, 0])
@pytest.mark.parametrize("as_int", [True, False], ids=["handle", "object"])
def test_handle_of_another_stream(rec, handle, as_int):
    """The entries that take a handle: the wait comes with it."""
    rec.Tensor.get_device = lambda self: 0
    stream = handle if as_int else rec.Stream(handle)
    assert binding._stream_handle(stream, [rec.Tensor()]) == handle
    assert rec.events == [("wait", handle, CURRENT), ("record", handle)]
    rec.events.clear()
    assert binding._stream_handle(stream) == handle and binding._stream_handle(CURRENT, [rec.Tensor()]) == CURRENT
    assert rec.events == []

"""The workspaces that the tensor entry points take: on which stream, and for how long.  No GPU is needed."""
import contextlib

import pytest
import torch
from torch.utils._python_dispatch import TorchDispatchMode

from tiled_dense_gemm_relu_amd import groups

NEED = groups.COUNTER_BYTES + 4096


class Streams:
    """Stands in for torch.cuda's streams: which one is current, and which are capturing."""

    def __init__(self, monkeypatch, capturing=()):
        self.now = "main"
        monkeypatch.setattr(groups, "_current_device", lambda: 0)
        monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: self.now in capturing)
        monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: self.now)

        @contextlib.contextmanager
        def enter(stream):
            before, self.now = self.now, stream
            yield
            self.now = before
        monkeypatch.setattr(torch.cuda, "stream", enter)


class Record(TorchDispatchMode):
    def __init__(self, streams):
        super().__init__()
        self.streams, self.seen = streams, []

    def __torch_dispatch__(self, func, types, args=(), kwargs=None):
        self.seen.append((func.__name__.split(".")[0], self.streams.now))
        return func(*args, **(kwargs or {}))


@pytest.mark.parametrize("stream", [None, "side"])
def test_capture_takes_and_clears_memory_on_the_stream_of_the_kernels(monkeypatch, stream):
    # "side" forked from "main" into one capture: only what is enqueued on it comes before its kernels.
    streams, like = Streams(monkeypatch, capturing=("main", "side")), torch.zeros(1)
    with Record(streams) as ops:
        ptr, nbytes, keep = groups._workspace(None, NEED, like, 0, 7, stream)
    assert nbytes >= NEED and ptr == keep.data_ptr() and not keep[:groups.COUNTER_BYTES].any()
    done = [(name, where) for name, where in ops.seen if name in ("empty", "zeros", "zero_", "fill_")]
    assert {where for _, where in done} == {stream or "main"} and any(name.startswith("zero") for name, _ in done)


def test_capture_of_another_stream_than_the_current_one(monkeypatch):
    # The kernels' stream is being captured, the current one is not: memory of the capture all the same.
    Streams(monkeypatch, capturing=("side",))
    first, second = (groups._workspace(None, NEED, torch.zeros(1), 0, 7, "side")[2] for _ in range(2))
    assert first.data_ptr() != second.data_ptr() and (0, 7) not in groups._spaces

"""The workspaces that the tensor entry points take: on which stream, and for how long.  No GPU is needed."""
import contextlib

import pytest
import torch
from torch.utils._python_dispatch import TorchDispatchMode

import tiled_dense_gemm_relu_amd as gr
from tiled_dense_gemm_relu_amd import binding, groups

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


def test_cached_workspaces_grow_and_are_released(monkeypatch):
    Streams(monkeypatch)
    monkeypatch.setattr(groups, "_spaces", {})
    like = torch.zeros(1)
    first = groups._workspace(None, NEED, like, 0, 7, "side")
    assert first[1] == NEED and not first[2][:groups.COUNTER_BYTES].any()
    assert groups._workspace(None, NEED - 1, like, 0, 7, "side") is first
    assert groups._workspace(None, NEED, like, 0, 8, None)[0] != first[0]          # another stream's
    assert groups._workspace(None, 2 * NEED, like, 0, 7, "side")[1] == 2 * NEED
    gr.release_workspaces()
    assert not groups._spaces
    assert not groups._workspace(None, NEED, like, 0, 7, "side")[2][:groups.COUNTER_BYTES].any()


def test_splitk_keeps_its_own_workspace(monkeypatch):
    # A captured gemm_relu_splitk holds the address of its cached buffer: a larger grouped call on the same
    # stream must not replace it.
    class Stream(str):
        cuda_stream = 7
    side = Stream("side")
    Streams(monkeypatch)
    monkeypatch.setattr(groups, "_spaces", {})
    monkeypatch.setattr(binding, "_workspaces", {})
    like = torch.zeros(1)
    mine = binding.splitk_workspace(like.device, side, NEED)
    assert groups._workspace(None, 8 * NEED, like, 0, 7, side)[0] != mine.data_ptr()
    gr.release_workspaces()
    assert binding.splitk_workspace(like.device, side, NEED) is mine

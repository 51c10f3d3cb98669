"""Host-side checks of gemm_relu_groups.h: exported symbols, workspace sizes and the refusal of bad
arguments before any device work.  No GPU is needed and no kernel is launched."""
import ctypes
import os
import re

import pytest
import torch

import tiled_dense_gemm_relu_amd as gr
from tiled_dense_gemm_relu_amd import groups

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "gemm_relu_groups.h")

# Fake, well separated addresses that are never dereferenced.
A, B, E, C, D, U, V, W = (i << 40 for i in range(1, 9))


@pytest.fixture(scope="module")
def lib():
    return groups._library()


def test_library_exports_every_declared_symbol(lib):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"^\s*(?:int|int64_t)\s+(gemm_relu\w*)\s*\(", text, flags=re.M))
    assert names == {"gemm_relu_grouped", "gemm_relu_grouped_workspace", "gemm_relu_grouped_backward",
                     "gemm_relu_grouped_backward_workspace", "gemm_relu_adapters", "gemm_relu_adapters_workspace"}
    for name in names:
        assert ctypes.cast(getattr(lib, name), ctypes.c_void_p).value


def grouped(lib, a=A, b=B, ends=E, c=C, M=4, N=8, K=8, groups=2, dtype=0, layout=0, relu=1, config=-1, ws=W,
            ws_bytes=1 << 30):
    return lib.gemm_relu_grouped(a, b, ends, c, M, N, K, groups, dtype, layout, relu, config, ws, ws_bytes, None)


def backward(lib, dc=D, c=C, a=A, b=B, ends=E, da=U, db=V, M=4, N=8, K=8, groups=2, dtype=0, layout=0, relu=1, config=-1,
             ws=W, ws_bytes=1 << 30):
    return lib.gemm_relu_grouped_backward(dc, c, a, b, ends, da, db, M, N, K, groups, dtype, layout, relu, config,
                                          ws, ws_bytes, None)


def adapters(lib, x=A, w=B, u=U, v=V, scales=D, ends=E, ids=E + 4096, c=C, M=4, N=8, K=8, rank=4, count=3, segments=2,
             dtype=0, layout=0, relu=1, config=-1, ws=W, ws_bytes=1 << 30):
    return lib.gemm_relu_adapters(x, w, u, v, scales, ends, ids, c, M, N, K, rank, count, segments, dtype, layout,
                                  relu, config, ws, ws_bytes, None)


COMMON = [({"dtype": 2}, -2), ({"dtype": -1}, -2), ({"layout": 2}, -9), ({"layout": -1}, -9), ({"M": -1}, -1),
          ({"N": -1}, -1), ({"K": -1}, -1), ({"relu": 2}, -1), ({"relu": -1}, -1), ({"M": (1 << 20) + 1}, -7),
          ({"N": (1 << 20) + 1}, -7), ({"K": (1 << 20) + 1}, -7), ({"ends": 0}, -1), ({"ends": E + 2}, -4), ({"config": -2}, -8),
          ({"config": 99}, -8)]


@pytest.mark.parametrize("args,code", COMMON + [
    ({"groups": 0}, -1), ({"groups": 65536}, -7), ({"a": 0}, -1), ({"b": 0}, -1), ({"c": 0}, -1),
    ({"a": A + 1}, -4), ({"b": B + 1}, -4), ({"c": C + 1}, -4), ({"c": A + 2}, -3), ({"c": B + 2}, -3),
    ({"c": E}, -3)])
def test_grouped_refuses(lib, args, code):
    assert grouped(lib, **args) == code


@pytest.mark.parametrize("args,code", COMMON + [
    ({"groups": 0}, -1), ({"groups": 65536}, -7), ({"dc": 0}, -1), ({"c": 0}, -1), ({"a": 0}, -1), ({"b": 0}, -1),
    ({"da": 0, "db": 0}, -1), ({"da": U + 1}, -4), ({"db": V + 1}, -4), ({"dc": D + 1}, -4), ({"da": D}, -3),
    ({"db": A}, -3), ({"db": U + 2}, -3), ({"da": C}, -3), ({"ws": 0}, -10), ({"ws": W + 128}, -10),
    ({"ws_bytes": 100}, -10), ({"ws": D & ~255}, -3), ({"ws": V}, -3)])
def test_backward_refuses(lib, args, code):
    assert backward(lib, **args) == code


@pytest.mark.parametrize("args,code", COMMON + [
    ({"segments": 0}, -1), ({"segments": 65536}, -7), ({"count": 0}, -1), ({"count": 65536}, -7), ({"rank": 0}, -1),
    ({"rank": 257}, -7), ({"x": 0}, -1), ({"w": 0}, -1), ({"u": 0}, -1), ({"v": 0}, -1), ({"scales": 0}, -1),
    ({"ids": 0}, -1), ({"scales": D + 2}, -4), ({"ids": E + 4097}, -4), ({"u": U + 1}, -4), ({"v": V + 1}, -4),
    ({"c": U}, -3), ({"c": V}, -3), ({"c": D}, -3), ({"ws": 0}, -10), ({"ws": W + 8}, -10), ({"ws_bytes": 0}, -10),
    ({"ws": U}, -3)])
def test_adapters_refuse(lib, args, code):
    assert adapters(lib, **args) == code


def test_empty_outputs_need_no_device(lib):
    assert grouped(lib, a=0, c=0, M=0) == 0
    assert grouped(lib, c=0, N=0) == 0
    assert adapters(lib, x=0, c=0, M=0) == 0
    assert adapters(lib, c=0, N=0) == 0
    assert backward(lib, K=0) == 0


def test_workspace_sizes():
    # The masked gradient, 2 bytes an element, past the counters.
    none = gr.grouped_backward_workspace_bytes(100, 64, 32, 4, gr.F16, relu=False)
    assert none == groups.COUNTER_BYTES
    assert gr.grouped_backward_workspace_bytes(100, 64, 32, 4, gr.F16) == none + 100 * 64 * 2
    # Two 16-bit parts and a factor for each 32 columns of rank (12 rounds up to 32).
    want = groups.COUNTER_BYTES + 64 * 2 * 32 * 2 + 64 * 4
    assert gr.adapters_workspace_bytes(64, 64, 32, 12, 4, 4, gr.BF16) >= want
    for call in (lambda: gr.grouped_workspace_bytes(1, 1, 1, 0, gr.F16),
                 lambda: gr.grouped_backward_workspace_bytes(1, 1, 1, 1, 5),
                 lambda: gr.adapters_workspace_bytes(1, 1, 1, 300, 1, 1, gr.F16)):
        with pytest.raises(gr.GemmReluError):
            call()


def test_python_refuses_what_is_not_a_gpu_tensor():
    t = torch.zeros((2, 2), dtype=torch.float16)
    with pytest.raises(ValueError):
        gr.gemm_relu_grouped(t, t[None], torch.tensor([2], dtype=torch.int32))
    with pytest.raises(ValueError):
        gr.gemm_relu_grouped_backward(t, t, t, t[None], torch.tensor([2], dtype=torch.int32))
    with pytest.raises(ValueError):
        gr.gemm_relu_adapters(t, t, t[None], t[None], torch.ones(1), torch.tensor([2], dtype=torch.int32),
                              torch.tensor([0], dtype=torch.int32))
    for call in (gr.gemm_relu_grouped, gr.gemm_relu_grouped_backward, gr.gemm_relu_adapters):
        with pytest.raises(TypeError):
            call(*([None] * (3 if call is gr.gemm_relu_grouped else 5 if call is gr.gemm_relu_grouped_backward else 7)))

"""Gradients of the grouped products through autograd, on the GPU."""
import pytest
import torch

import tiled_dense_gemm_relu_amd as gr
from test_gpu_groups import ends_of, normal, weights

pytestmark = pytest.mark.gpu

SIZES, N, K = [40, 0, 3, 90], 72, 136


def inputs(dtype, layout, seed):
    M = sum(SIZES) + 2
    a, b = normal((M, K), dtype, seed).cuda(), weights(len(SIZES), N, K, dtype, layout, seed + 1).cuda()
    return a, b, ends_of(SIZES).cuda(), normal((M, N), dtype, seed + 2).cuda()


@pytest.mark.parametrize("needs", [(True, True), (True, False), (False, True)])
@pytest.mark.parametrize("relu", [True, False])
@pytest.mark.parametrize("layout", [gr.B_KN, gr.B_NK])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_autograd_gives_the_calls_gradients(dtype, layout, relu, needs):
    a, b, ends, dc = inputs(dtype, layout, 301)
    c = gr.gemm_relu_grouped(a, b, ends, b_layout=layout, relu=relu)
    da, db = gr.gemm_relu_grouped_backward(dc, c if relu else None, a, b, ends, b_layout=layout, relu=relu)
    a.requires_grad_(needs[0])
    b.requires_grad_(needs[1])
    y = gr.gemm_relu_grouped(a, b, ends, b_layout=layout, relu=relu)
    assert y.requires_grad and torch.equal(y, c)
    y.backward(dc)
    assert torch.equal(a.grad, da) if needs[0] else a.grad is None
    assert torch.equal(b.grad, db) if needs[1] else b.grad is None


def test_autograd_on_a_side_stream():
    a, b, ends, dc = inputs(torch.bfloat16, gr.B_KN, 311)
    c = gr.gemm_relu_grouped(a, b, ends)
    want = gr.gemm_relu_grouped_backward(dc, c, a, b, ends)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    y = gr.gemm_relu_grouped(a.requires_grad_(), b.requires_grad_(), ends, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    got = torch.autograd.grad(y, (a, b), dc)
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("sizes", [[1, 0, 2, 1], SIZES])
def test_captured_backward_pass(sizes):
    # Forward and backward in one graph; no eager graph of the leaves is alive.
    M = sum(sizes)
    a, b = normal((M, 512), torch.bfloat16, 341).cuda(), weights(4, 256, 512, torch.bfloat16, gr.B_KN, 342).cuda()
    ends, dc = ends_of(sizes).cuda(), normal((M, 256), torch.bfloat16, 343).cuda()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        gr.gemm_relu_grouped(a, b, ends)
    torch.cuda.synchronize()
    a.requires_grad_()
    b.requires_grad_()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = gr.gemm_relu_grouped(a, b, ends)
        da, db = torch.autograd.grad(y, (a, b), dc)
    for k in range(4):
        with torch.no_grad():
            a.copy_(normal((M, 512), torch.bfloat16, 350 + k))
            dc.copy_(normal((M, 256), torch.bfloat16, 360 + k))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        with torch.no_grad():
            c = gr.gemm_relu_grouped(a, b, ends)
            want = gr.gemm_relu_grouped_backward(dc, c, a, b, ends)
        torch.cuda.synchronize()
        assert torch.equal(y, c) and torch.equal(da, want[0]) and torch.equal(db, want[1]), k


def test_what_needs_no_graph_gets_none():
    a, b, ends, _ = inputs(torch.float16, gr.B_KN, 321)
    out = torch.empty((a.shape[0], N), dtype=a.dtype, device="cuda")
    assert gr.gemm_relu_grouped(a, b, ends, out=out) is out and not out.requires_grad
    b.requires_grad_()
    with pytest.raises(RuntimeError, match="no_grad"):
        gr.gemm_relu_grouped(a, b, ends, out=out)
    with torch.no_grad():
        assert gr.gemm_relu_grouped(a, b, ends, out=out) is out and not out.requires_grad
    da, db = gr.gemm_relu_grouped_backward(out, out, a, b, ends)
    assert not da.requires_grad and not db.requires_grad


def test_adapters_refuse_a_backward_pass():
    x, w = normal((3, 64), torch.float16, 331).cuda(), normal((64, 48), torch.float16, 332).cuda()
    u, v = normal((2, 64, 8), torch.float16, 333).cuda(), normal((2, 8, 48), torch.float16, 334).cuda()
    rest = (torch.ones(2, device="cuda"), torch.tensor([1, 3]).int().cuda(), torch.tensor([1, 0]).int().cuda())
    want = gr.gemm_relu_adapters(x, w, u, v, *rest)
    y = gr.gemm_relu_adapters(x, w.requires_grad_(), u, v, *rest)
    assert torch.equal(y, want)
    with pytest.raises(NotImplementedError, match="no_grad"):
        y.sum().backward()
    with pytest.raises(RuntimeError, match="no_grad"):
        gr.gemm_relu_adapters(x, w, u, v, *rest, out=want)
    with torch.no_grad():
        assert gr.gemm_relu_adapters(x, w, u, v, *rest, out=want) is want

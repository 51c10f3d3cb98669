"""What has no derivative says so: fp32 scales of 8-bit operands, and tangents of forward mode."""
import pytest
import torch

import tiled_dense_gemm_relu_amd as gr
from tiled_dense_gemm_relu_amd import blocks

from test_gpu_blocks_use import NotCompiled, randn, same_tensors

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(params=["compiled", "python"])
def route(request, monkeypatch):
    if request.param == "python":
        monkeypatch.setattr(blocks, "_calls", NotCompiled())


def test_scales_of_products(route):
    x, dc = randn((32, 48), 1).to(DEV), randn((32, 32), 2).to(DEV)
    q, s, qt, st = gr.quantize_blocks(x, transposed=True)
    w, sw, wt, swt = gr.quantize_blocks(x, tiles=True, transposed=True)
    want = gr.gemm_relu_blocks(q, s, w, sw)
    grads = gr.gemm_relu_blocks_backward(dc, want, qt, st, wt, swt)
    for t in (s, sw):
        t.requires_grad_()
        with pytest.raises(RuntimeError, match="_scales requires a gradient"):
            gr.gemm_relu_blocks(q, s, w, sw)
        with torch.no_grad():
            assert torch.equal(gr.gemm_relu_blocks(q, s, w, sw), want)
        t.requires_grad_(False)
    for t in (st, swt):
        t.requires_grad_()
        with pytest.raises(RuntimeError, match="t_scales requires a gradient"):
            gr.gemm_relu_blocks_backward(dc, want, qt, st, wt, swt)
        with torch.no_grad():
            assert all(same_tensors(u, v) for u, v in zip(gr.gemm_relu_blocks_backward(dc, want, qt, st, wt, swt), grads))
        t.requires_grad_(False)
    # one that is not needed is not looked at
    st.requires_grad_()
    assert torch.equal(gr.gemm_relu_blocks_backward(dc, want, None, st, wt, swt, need_dw=False)[0], grads[0])


def test_scales_of_an_expert_layer(route):
    x, logits = randn((4, 32), 1).to(DEV), torch.zeros((4, 2), device=DEV)
    w1, s1 = gr.quantize_blocks(randn((2, 16, 32), 2).to(DEV), tiles=True)
    w2, s2 = gr.quantize_blocks(randn((2, 32, 16), 3).to(DEV), tiles=True)

    def call(**kw):
        return gr.gemm_relu_experts(x, w1, w2, logits, 1, w1_scales=s1, w2_scales=s2, **kw)
    want = call()
    for s in (s1, s2):
        s.requires_grad_()
        y, ids, weights = call()
        assert y.requires_grad and not weights.requires_grad and torch.equal(y, want[0])
        with pytest.raises(NotImplementedError, match="no gradient"):
            y.sum().backward()
        with pytest.raises(RuntimeError, match="out="):
            call(out=torch.empty_like(x))
        with torch.no_grad():
            assert not call()[0].requires_grad
        s.requires_grad_(False)


def test_forward_mode(route):
    from torch.autograd import forward_ad
    x, w = randn((32, 48), 1).to(DEV), randn((16, 48), 2).to(DEV)
    w1, w2, logits = randn((2, 16, 48), 3).to(DEV), randn((2, 48, 16), 4).to(DEV), torch.zeros((32, 2), device=DEV)
    ends = torch.tensor([10, 32], dtype=torch.int32, device=DEV)
    q, s = gr.quantize_blocks(x)
    qw, sw = gr.quantize_blocks(w, tiles=True)
    scales, ids, one = torch.ones(1, device=DEV), torch.zeros(2, dtype=torch.int32, device=DEV), randn((1, 48, 8), 5).to(DEV)
    square, v = randn((48, 24), 6).to(DEV), randn((1, 8, 24), 7).to(DEV)
    calls = {
        "linear_blocks, x": (x, lambda t: gr.linear_blocks(t, w)), "linear_blocks, w": (w, lambda t: gr.linear_blocks(x, t)),
        "experts, x": (x, lambda t: gr.gemm_relu_experts(t, w1, w2, logits, 1)),
        "experts, w1": (w1, lambda t: gr.gemm_relu_experts(x, t, w2, logits, 1)),
        "experts, logits": (logits, lambda t: gr.gemm_relu_experts(x, w1, w2, t, 1)),
        "product, a_scales": (s, lambda t: gr.gemm_relu_blocks(q, t, qw, sw)),
        "product, b_scales": (sw, lambda t: gr.gemm_relu_blocks(q, s, qw, t)),
        "grouped, a": (x, lambda t: gr.gemm_relu_grouped(t, w2.transpose(1, 2).contiguous(), ends, b_layout=gr.B_NK)),
        "adapters, x": (x, lambda t: gr.gemm_relu_adapters(t, square, one, v, scales, ends, ids)),
    }
    for name, (t, call) in calls.items():
        call(t)                                          # takes the stream's workspace
        for enabled in (True, False):
            with torch.set_grad_enabled(enabled), forward_ad.dual_level():
                dual = forward_ad.make_dual(t, torch.ones_like(t))
                with pytest.raises(NotImplementedError, match="forward-mode"):
                    call(dual)
                call(t)                                  # others pass while a level is open
    with torch.no_grad():
        assert gr.linear_blocks(x, w).isfinite().all()

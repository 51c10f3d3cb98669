"""Gradients of 8-bit layers past the sizes of one launch for both: the quantizer, then two products by the kernels
that products of their sizes take.  Integers whose quantized values are exact, so gradients are known exactly too."""
import pytest
import torch

import tiled_dense_gemm_relu_amd as gr

from test_gpu_blocks import E4M3, E5M2, gen

pytestmark = pytest.mark.gpu
DEV = "cuda"

# Both gradients apart: long sums over few tiles; many tiles of 64, 128 and 256, with remainders; longest rows' pitches;
# few rows; and one launch for both, for comparison.
SHAPES = [(2048, 512, 512), (1100, 520, 500), (2100, 1500, 2100), (1300, 3100, 1111), (4100, 2056, 4100), (16, 2048, 2048),
          (1, 4100, 2050), (5000, 130, 100), (700, 640, 500)]


def integers(shape, seed):
    """-2 .. 2: multiples of a block's largest by 1, 1/2 and 0, which both formats hold."""
    return torch.randint(-2, 3, shape, generator=gen(seed)).half()


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("fx,fw", [(E4M3, E4M3), (E5M2, E4M3), (E4M3, E5M2)])
@pytest.mark.parametrize("relu", [True, False])
def test_gradients_of_integers(shape, fx, fw, relu):
    M, N, K = shape
    x, w, dc, c = (integers(s, i).to(DEV) for i, s in enumerate(((M, K), (N, K), (M, N), (M, N))))
    xt, sx = gr.quantize_blocks(x, fx, rows=False, transposed=True)
    wt, sw = gr.quantize_blocks(w, fw, tiles=True, rows=False, transposed=True)
    d = (torch.where(c > 0, dc, torch.zeros_like(dc)) if relu else dc).float()
    # (fp32 sums of integers below 2^24 are exact in any order; gradients are integers that fp16 holds)
    want_x, want_w = d @ w.float(), d.t().contiguous() @ x.float()
    assert max(float(want_x.abs().max()), float(want_w.abs().max())) <= 2048
    args = dc, c if relu else None, xt, sx, wt, sw
    for fmt in (E5M2, E4M3):
        dx, dw = gr.gemm_relu_blocks_backward(*args, relu=relu, dtype=fmt)
        # The scales are 2 / 448 and the like, no powers of two: a gradient is off by up to (blocks + 3) 2^-24 of its
        # partial sums, which are at most 512 a block of at most 64, so by less than 67 2^-24 2^15 = 0.14: the integer
        # is the nearest one (where it is not zero, fp16 holds no other number as close).
        assert torch.equal(dx.float().round(), want_x) and torch.equal(dw.float().round(), want_w)
        assert torch.equal(gr.gemm_relu_blocks_backward(*args, relu=relu, dtype=fmt, need_dw=False)[0], dx)
        assert torch.equal(gr.gemm_relu_blocks_backward(*args, relu=relu, dtype=fmt, need_dx=False)[1], dw)

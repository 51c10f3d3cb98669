"""The quantizer's values with their signs: zeros that stay zero, and what rounds to zero, bit for bit."""
import pytest
import torch

import tiled_dense_gemm_relu_amd as gr

from test_gpu_blocks import E4M3, E5M2, gen, reference_quantize

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("shape", [(3, 128), (130, 260), (70, 333)])
@pytest.mark.parametrize("fmt", [E4M3, E5M2])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("infinite", [False, True])
def test_signs_of_zeros(shape, fmt, dtype, infinite):
    R, C = shape
    x = torch.randn((R, C), generator=gen(R)).to(dtype)
    kind = torch.randint(0, 6, (R, C), generator=gen(C))
    x[kind == 0], x[kind == 1] = 0.0, -0.0
    x[kind == 2] *= 2.0 ** -13                       # to subnormal values, and to zeros of both signs
    x[0] = -0.0                                      # a block without a magnitude
    if infinite:
        x[-1, -1] = float("-inf")
    for tiles in (False, True):
        q, _, qt, _ = gr.quantize_blocks(x.to(DEV), fmt, tiles=tiles, transposed=True)
        for got, source in ((q, x), (qt, x.t())):
            want, _ = reference_quantize(source, fmt, tiles, False)
            number = ~want.isnan()
            assert torch.equal(got.cpu().view(torch.uint8)[number], want.to(fmt).view(torch.uint8)[number])
            assert torch.equal(got.cpu().float().isnan(), ~number)


def test_masked_places_are_positive_zeros():
    x = -torch.ones((5, 40), dtype=torch.bfloat16)
    mask = torch.ones_like(x)
    mask[:, ::2] = -1
    q, _ = gr.quantize_blocks(x.to(DEV), mask=mask.to(DEV))
    assert not q.cpu().view(torch.uint8)[:, ::2].any() and (q.cpu().view(torch.uint8)[:, 1::2] == 0xfe).all()

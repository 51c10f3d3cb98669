"""An expert layer whose 8-bit weights have scales far from 1: powers of two in rows and scales are powers of two in
the results, bit for bit, also where rows times stored values alone are out of range."""
import pytest
import torch

from test_gpu_experts import Layer

pytestmark = pytest.mark.gpu
DEV = "cuda"


def times(s, power):
    return (s.double() * 2.0 ** power).float()


# tokens, K, hidden, N, experts, top: rows by DMA, rows of odd length through registers, few and many units
@pytest.mark.parametrize("shape", [(3, 256, 128, 192, 8, 2), (5, 301, 130, 70, 6, 2), (24, 512, 640, 512, 32, 4), (40, 129, 1400, 1100, 16, 4)])
@pytest.mark.parametrize("kind", ["e4m3", "e5m2"])
def test_powers_of_two(shape, kind):
    T, K, H, N, E, top = shape
    layer = Layer(kind, torch.bfloat16, E, K, H, N, 3)
    g = torch.Generator().manual_seed(4)
    x = torch.randint(-8, 9, (T, K), generator=g).float()
    logits = torch.randn((T, E), generator=g).to(DEV)
    s1, s2 = (layer.args[f"w{i}_scales"].clone() for i in (1, 2))

    def call(px, p1, p2):
        layer.args["w1_scales"], layer.args["w2_scales"] = times(s1, p1), times(s2, p2)
        return layer((x * 2.0 ** px).bfloat16().to(DEV), logits, top)[0].cpu()
    base = call(0, 0, 0)
    assert base.isfinite().all() and base.any()
    # large and small rows, large and small intermediates, scales that a widened weight's exponent cannot hold
    for px, p1, p2 in ((124, -118, 0), (-120, 117, 0), (0, 116, -114), (0, -60, 119), (100, -95, -5), (3, 4, -8)):
        got, want = call(px, p1, p2), base.double() * 2.0 ** (px + p1 + p2)
        assert torch.equal(got.double(), want), (px, p1, p2, int((got.double() != want).sum()), want.numel())


@pytest.mark.parametrize("K", [256, 301])
@pytest.mark.parametrize("kind", ["e4m3", "e5m2"])
def test_terms_that_cancel_under_large_scales(K, kind):
    # Terms past the largest float, of a sum that is not: block sums are taken before they are scaled.
    layer = Layer(kind, torch.bfloat16, 2, K, 128, 64, 3)
    x = torch.zeros((3, K))
    w = torch.zeros((2, 128, K))
    x[:, 0], x[:, 70], w[:, :, 0], w[:, :, 70] = 1024.0, -1024.0, 256.0, 256.0
    x[:, 9], w[:, :, 9] = 1.0, 0.25
    layer.w[0][..., :] = w.to(layer.w[0].dtype).to(DEV)
    layer.args["w1_scales"] = torch.full_like(layer.args["w1_scales"], 0.75)
    s1, s2 = layer.args["w1_scales"].clone(), layer.args["w2_scales"].clone()
    x, logits = x.bfloat16().to(DEV), torch.zeros((3, 2), device=DEV)

    def call(power):
        layer.args["w1_scales"], layer.args["w2_scales"] = times(s1, power), times(s2, -power)
        return layer(x, logits, 1)[0].cpu()
    base = call(0)
    assert base.isfinite().all() and base.any()
    for power in (60, 110, 115):
        assert torch.equal(call(power), base), power


def test_scales_without_an_exponent():
    layer = Layer("e4m3", torch.bfloat16, 4, 128, 128, 64, 3)
    x, logits = torch.ones((2, 128), dtype=torch.bfloat16, device=DEV), torch.zeros((2, 4), device=DEV)
    layer.args["w2_scales"] = torch.zeros_like(layer.args["w2_scales"])
    assert (layer(x, logits, 2)[0] == 0).all()
    layer.args["w2_scales"] = torch.full_like(layer.args["w2_scales"], float("nan"))
    assert layer(x, logits, 2)[0].isnan().all()

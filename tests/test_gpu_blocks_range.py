"""8-bit products whose scales lie far from 1: powers of two in the scales are powers of two in the results, bit for bit,
wherever the results are in range, also where the product of two scales is not."""
import pytest
import torch

import tiled_dense_gemm_relu_amd as gr
from tiled_dense_gemm_relu_amd import blocks

from test_gpu_blocks import E4M3, E5M2, gen, nb, pitched

pytestmark = pytest.mark.gpu
DEV = "cuda"
CONFIGS = [blocks.CONFIG_AUTO, blocks.CONFIG_256, blocks.CONFIG_128, blocks.CONFIG_64, blocks.CONFIG_STREAM]


def values(shape, fmt, seed):
    """Multiples of the 2^4 (2^12) to 240 (28672): no product is far below the largest."""
    n, unit = (15, 16.0) if fmt == E4M3 else (7, 4096.0)
    return (torch.randint(-n, n + 1, shape, generator=gen(seed)).float() * unit).to(fmt)


class Operands:
    def __init__(self, M, N, K, fa, fb, b_rows, seed=1):
        self.a, self.b = values((M, K), fa, seed), values((N, K), fb, seed + 1)
        self.sa = torch.rand((nb(K), M), generator=gen(seed + 2)) + 0.5
        self.sb = torch.rand((nb(K), N) if b_rows else (nb(N), nb(K)), generator=gen(seed + 3)) + 0.5
        self.b_rows = b_rows
        self.pa, self.pb = pitched(self.a), pitched(self.b)

    def __call__(self, sa, sb, config):
        return gr.gemm_relu_blocks(self.pa, sa.to(DEV), self.pb, sb.to(DEV), relu=False, b_rows=self.b_rows, config=config).cpu()


def times(s, power):
    """s 2^power, rounded once where that is subnormal."""
    return (s.double() * 2.0 ** power).float()


def check_same(got, base, power):
    """got is base 2^power: exactly where that is at least 2^-120 (fp32 sums of that size have all their bits),
    and within 2^-128 where the terms cancelled to less."""
    want = base.double() * 2.0 ** power
    sure = want.abs() >= 2.0 ** -120
    assert sure.double().mean() > 0.5
    assert torch.equal(got[sure].double(), want[sure]), f"{int((got[sure].double() != want[sure]).sum())} of {int(sure.sum())}"
    assert ((got.double() - want).abs()[~sure] <= 2.0 ** -128).all()


# Results are some 2^18 (e4m3) to 2^32 (e5m2) times the scales: normal floats, of scales whose product is none.
SMALL = {(E4M3, E4M3): (-75, -62), (E4M3, E5M2): (-62, -80), (E5M2, E4M3): (-89, -50), (E5M2, E5M2): (-95, -56)}


@pytest.mark.parametrize("config", CONFIGS)
@pytest.mark.parametrize("b_rows", [False, True])
@pytest.mark.parametrize("fa,fb", list(SMALL))
def test_powers_of_two_in_the_scales(config, b_rows, fa, fb):
    op = Operands(70, 200, 300, fa, fb, b_rows)
    base = op(op.sa, op.sb, config)
    for p, q in [SMALL[fa, fb], SMALL[fa, fb][::-1], (-95, 93), (93, -95), (119, -110), (-110, 119), (126, -123), (-123, 126)]:
        check_same(op(times(op.sa, p), times(op.sb, q), config), base, p + q)
    check_same(op(-op.sa, times(op.sb, -3), config), -base, -3)


@pytest.mark.parametrize("shape", [(5, 13000, 130), (3, 25003, 300), (20, 13000, 1100), (20, 26000, 129), (64, 12500, 300),
                                   (64, 16384, 4200), (300, 700, 2000)])
@pytest.mark.parametrize("b_rows", [False, True])
def test_every_streaming_kernel(shape, b_rows):
    op = Operands(*shape, E5M2, E4M3, b_rows, 7)
    for config in (blocks.CONFIG_AUTO, blocks.CONFIG_STREAM):
        base = op(op.sa, op.sb, config)
        for p, q in [(-89, -50), (-95, 93), (119, -110)]:
            check_same(op(times(op.sa, p), times(op.sb, q), config), base, p + q)


@pytest.mark.parametrize("config", CONFIGS)
@pytest.mark.parametrize("b_rows", [False, True])
def test_subnormal_scales(config, b_rows):
    op = Operands(70, 200, 300, E4M3, E5M2, b_rows, 11)
    # what is left of the bits of subnormal scales, in range
    small, other = times(op.sa, -135), times(op.sb, -135)
    check_same(op(small, times(op.sb, 100), config), op(times(small, 135), op.sb, config), -35)
    check_same(op(times(op.sa, 100), other, config), op(op.sa, times(other, 135), config), -35)


@pytest.mark.parametrize("config", CONFIGS)
@pytest.mark.parametrize("b_rows", [False, True])
def test_blocks_of_zeros_under_large_scales(config, b_rows):
    # The product of the scales is past the largest float; the sums that it multiplies are zero.
    M, N, K = 70, 200, 300
    op = Operands(M, N, K, E4M3, E4M3, b_rows, 13)
    a = op.a.float()
    a[::2, 128:256] = 0
    op.pa = pitched(a.to(E4M3))
    sa, sb = op.sa.clone(), op.sb.clone()
    base = op(sa, sb, config)
    sa[1] *= 2.0 ** 100
    (sb[1] if b_rows else sb[:, 1]).mul_(2.0 ** 60)
    got = op(sa, sb, config)
    assert torch.equal(got[::2], base[::2]) and got[1::2].isinf().double().mean() > 0.9 and not got.isnan().any()
    # a scale of zero counts for nothing, however large the other is
    sa[1] = 0
    want = op(torch.where(torch.arange(nb(K))[:, None] == 1, torch.zeros(()), op.sa), op.sb, config)
    assert torch.equal(op(sa, sb, config), want)


@pytest.mark.parametrize("config", CONFIGS)
@pytest.mark.parametrize("b_rows", [False, True])
@pytest.mark.parametrize("fa,fb", list(SMALL))
@pytest.mark.parametrize("apart", [1, 8, 64])
def test_terms_that_cancel_under_large_scales(config, b_rows, fa, fb, apart):
    # Terms past the largest float, of a sum that is not: block sums are taken before they are scaled.
    M, N, K = 70, 200, 256
    op = Operands(M, N, K, fa, fb, b_rows, 17)
    a, b = torch.zeros((M, K)), torch.zeros((N, K))
    a[:, 0::128], a[:, apart::128], b[:, 0::128], b[:, apart::128] = 448.0, -448.0, 448.0, 448.0
    a[:, 9::128], b[:, 9::128] = 16.0 * torch.randint(1, 4, (M, 1), generator=gen(1)), 2.0
    op.pa, op.pb = pitched(a.to(fa)), pitched(b.to(fb))
    base = op(op.sa, op.sb, config)
    assert ((base >= 16) & (base <= 512)).all()
    for p, q in ((119, -1), (59, 58), (-1, 117), (30, 85)):
        assert torch.equal(op(times(op.sa, p), times(op.sb, q), config).double(), base.double() * 2.0 ** (p + q)), (p, q)


@pytest.mark.parametrize("sizes", [[300, 0, 1, 17, 128, 0, 260], [1] * 70, [64] * 5 + [0] * 80 + [3]])
@pytest.mark.parametrize("config", CONFIGS)
def test_groups(sizes, config):
    G, N, K, M = len(sizes), 200, 300, sum(sizes)
    a, b = pitched(values((M, K), E4M3, 1)), pitched(values((G, N, K), E4M3, 2))
    sa, sb = torch.rand((nb(K), M), generator=gen(3)) + 0.5, torch.rand((G, nb(N), nb(K)), generator=gen(4)) + 0.5
    ends = torch.tensor(sizes).cumsum(0).to(torch.int32).to(DEV)

    def call(p, q):
        return gr.gemm_relu_blocks(a, times(sa, p).to(DEV), b, times(sb, q).to(DEV), ends=ends, relu=False, config=config).cpu()
    base = call(0, 0)
    for p, q in ((-75, -62), (119, -110), (-95, 93)):
        check_same(call(p, q), base, p + q)


@pytest.mark.parametrize("shape", [(100, 200, 300), (640, 1100, 200), (300, 1500, 2000)])
def test_gradients(shape):
    # bf16 gradients and operands of magnitudes far from 1 (from 2^-80 on, which is the least that a scale covers)
    M, N, K = shape
    x, w, dc = (torch.randn(s, generator=gen(i)).bfloat16() for i, s in enumerate(((M, K), (N, K), (M, N))))

    def call(px, pw, pd):
        xt, sx = gr.quantize_blocks((x * 2.0 ** px).to(DEV), E5M2, rows=False, transposed=True)
        wt, sw = gr.quantize_blocks((w * 2.0 ** pw).to(DEV), E5M2, tiles=True, rows=False, transposed=True)
        return [t.cpu() for t in gr.gemm_relu_blocks_backward((dc * 2.0 ** pd).to(DEV), None, xt, sx, wt, sw, relu=False)]
    base = call(0, 0, 0)
    for px, pw, pd in ((-60, -60, -60), (110, 100, -75), (-70, -75, 80), (80, 80, -75)):
        dx, dw = call(px, pw, pd)
        for got, want, power in ((dx, base[0], pw + pd), (dw, base[1], px + pd)):
            want = want.double() * 2.0 ** power
            off = (got.double() - want).abs()
            # Small products may lose bits where they are subnormal, and a rounding go the other way.  Below 2^-126
            # a step of bf16 is 2^-133 however small the result is: half of it for the result, half for a result
            # that lies on the other side of a border.
            assert (off <= want.abs() * 2.0 ** -8 + want.abs().max() * 2.0 ** -20 + 2.0 ** -133).all() and got.isfinite().all()

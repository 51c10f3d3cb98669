"""The products whose rows choose their weights against plain 64-bit references.

Bars, derived from the arithmetic (u = half a step of the output dtype, relative): an output is a
sum held in fp32 and rounded once, so |got - ref| <= u |ref| + (1 + u) s + tiny, where s bounds the
sum's own error: each of its n additions is off by at most 2^-23 of the sum of |products| (a product
of two 16-bit values is exact in fp32; 2^-23, not 2^-24, allows for additions that truncate), and
tiny is half the smallest fp16 subnormal.  The adapters' intermediate adds its two-part rounding,
u^2 relative plus 2^-25 of its block's largest entry (fp16 subnormals of the second part).
"""
import itertools
import sys

import pytest
import torch

import tiled_dense_gemm_relu_amd as gr
from tiled_dense_gemm_relu_amd import binding, groups

pytestmark = pytest.mark.gpu

DT = {"fp16": torch.float16, "bf16": torch.bfloat16}
TINY = 2.0 ** -25


def say(msg):
    print(msg, file=sys.stderr, flush=True)


def ends_of(sizes):
    return torch.tensor(list(itertools.accumulate(sizes)), dtype=torch.int32)


def normal(shape, dtype, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(dtype)


def spans(sizes):
    ends = [0] + list(itertools.accumulate(sizes))
    return list(zip(range(len(sizes)), ends, ends[1:]))


def unaligned(t):
    """The same values 2 bytes off any wider alignment, on the GPU."""
    buf = torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")
    view = buf[1:].view(t.shape)
    view.copy_(t)
    return view


def guarded(shape, dtype, shift=0):
    """An output between two bands of a value that no kernel writes, and a check that they are whole."""
    n = 1
    for d in shape:
        n *= d
    buf = torch.full((n + 1024 + shift,), 777.0, dtype=dtype, device="cuda")
    view = buf[512 + shift:512 + shift + n].view(shape)

    def whole():
        return bool((buf[:512 + shift] == 777.0).all()) and bool((buf[512 + shift + n:] == 777.0).all())
    return view, whole


def assert_close(got, ref, err, what):
    """|got - ref| within u |ref| + (1 + u) err + tiny; exact where both are infinite or NaN."""
    u = torch.finfo(got.dtype).eps / 2
    g = got.detach().cpu().double()
    assert g.shape == ref.shape
    off = (g - ref).abs()
    bound = u * ref.abs() + (1 + u) * err + TINY
    bad = ~(off <= bound)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} out of tolerance, first at "
                           f"{bad.nonzero()[0].tolist()}: got {g[bad][0].item()}, want {ref[bad][0].item()} "
                           f"+- {bound[bad][0].item()}")


# ---------------------------------------------------------------- grouped products

def weights(groups_n, N, K, dtype, layout, seed, scale=None):
    b = normal((groups_n, K, N), dtype, seed, K ** -0.5 if scale is None else scale)
    return b.transpose(1, 2).contiguous() if layout == gr.B_NK else b


def as_kn(b, layout):
    return b.transpose(1, 2) if layout == gr.B_NK else b


def grouped_reference(a, b, sizes, layout, relu):
    a64, b64 = a.double(), as_kn(b, layout).double()
    M, K = a.shape
    ref = torch.zeros((M, b64.shape[2]), dtype=torch.float64)
    mag = torch.zeros_like(ref)
    for e, lo, hi in spans(sizes):
        if hi > lo:
            ref[lo:hi] = a64[lo:hi] @ b64[e]
            mag[lo:hi] = a64[lo:hi].abs() @ b64[e].abs()
    return (ref.clamp_min(0) if relu else ref), K * 2.0 ** -23 * mag


# (group sizes, spare rows, N, K)
SHAPES = [
    ([1], 0, 1, 1),
    ([3, 0, 5], 2, 33, 17),
    ([0, 0, 1, 0], 0, 64, 64),                       # one token
    ([1] * 16, 0, 256, 256),
    ([2, 0, 1, 7, 0, 0, 16, 3], 1, 512, 1024),       # a decoding step
    ([0, 1, 0, 2] * 40, 3, 128, 192),                # more groups than a wave has lanes, most of one or no row
    ([17, 31, 0, 64], 0, 136, 264),
    ([100, 28, 1], 0, 384, 320),
    ([130, 127, 3, 0, 257], 5, 200, 72),
    ([300], 0, 257, 129),
    ([5, 200, 95], 0, 130, 100),
    ([600, 0, 424], 0, 264, 136),
    ([0, 0], 9, 48, 40),                             # rows, none of them in a group
    ([40, 600, 900, 508], 0, 512, 512),
]


@pytest.mark.parametrize("relu", [True, False])
@pytest.mark.parametrize("layout", [gr.B_KN, gr.B_NK])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("shape", range(len(SHAPES)))
def test_grouped(shape, dtype, layout, relu):
    sizes, spare, N, K = SHAPES[shape]
    M = sum(sizes) + spare
    say(f"[grouped] {sizes[:6]} M={M} N={N} K={K} {dtype} layout={layout} relu={relu}")
    a, b = normal((M, K), DT[dtype], 1 + shape), weights(len(sizes), N, K, DT[dtype], layout, 2 + shape)
    ref, err = grouped_reference(a, b, sizes, layout, relu)
    out, whole = guarded((M, N), DT[dtype])
    got = gr.gemm_relu_grouped(a.cuda(), b.cuda(), ends_of(sizes).cuda(), out=out, b_layout=layout, relu=relu)
    torch.cuda.synchronize()
    assert got is out and whole()
    assert_close(out, ref, err, "C")
    if spare:
        assert (out[-spare:].view(torch.int16) == 0).all()        # +0.0


# Every kernel on shapes whose rows are 16-byte multiples (the others fall back to TILED): K-steps
# with and without a tail, fewer steps than stages, tiles that end inside a group, several tiles of
# work for a workgroup, more than 64 groups.
CONFIGS = [groups.CONFIG_TILED, groups.CONFIG_DMA_256, groups.CONFIG_DMA_128, groups.CONFIG_DMA_64,
           groups.CONFIG_STREAM]
CONFIG_SHAPES = [
    ([1, 0, 4], 1, 64, 64),
    ([40, 0, 256, 300], 3, 264, 136),
    ([513, 130], 0, 520, 320),
    ([0, 1, 5, 0, 70] * 17, 2, 136, 200),
    ([2000, 0, 1300], 30, 2056, 64),
    ([40, 0, 256, 300], 3, 262, 138),      # rows of an even length: K % 8 is 2
    ([1, 130, 64], 0, 134, 60),            # 4 (and less than a K-step)
    ([513, 130], 0, 518, 326),             # 6
    ([300, 40], 1, 261, 137),              # odd
]


@pytest.mark.parametrize("layout", [gr.B_KN, gr.B_NK])
@pytest.mark.parametrize("config", CONFIGS)
@pytest.mark.parametrize("shape", range(len(CONFIG_SHAPES)))
def test_grouped_kernels(shape, config, layout):
    sizes, spare, N, K = CONFIG_SHAPES[shape]
    M, dt = sum(sizes) + spare, (torch.float16, torch.bfloat16)[shape % 2]
    say(f"[grouped] {sizes[:6]} M={M} N={N} K={K} {dt} layout={layout} config={config}")
    a, b = normal((M, K), dt, 11 + shape), weights(len(sizes), N, K, dt, layout, 12 + shape)
    ends = ends_of(sizes).cuda()
    ref, err = grouped_reference(a, b, sizes, layout, True)
    out, whole = guarded((M, N), dt)
    gr.gemm_relu_grouped(a.cuda(), b.cuda(), ends, out=out, b_layout=layout, config=config)
    torch.cuda.synchronize()
    assert whole()
    assert_close(out, ref, err, "C")
    if spare:
        assert (out[-spare:].view(torch.int16) == 0).all()
    dc, c = normal((M, N), dt, 13 + shape), normal((M, N), dt, 14 + shape).clamp_min(0)
    ra, ea, rb, eb = backward_reference(dc, c, a, b, sizes, layout, True)
    da, whole_a = guarded((M, K), dt)
    db, whole_b = guarded(tuple(b.shape), dt)
    gr.gemm_relu_grouped_backward(dc.cuda(), c.cuda(), a.cuda(), b.cuda(), ends, b_layout=layout, da=da, db=db,
                                  config=config)
    torch.cuda.synchronize()
    assert whole_a() and whole_b()
    assert_close(da, ra, ea, "dA")
    assert_close(db, rb, eb, "dB")


@pytest.mark.parametrize("layout", [gr.B_KN, gr.B_NK])
@pytest.mark.parametrize("N,K", [(1101, 2051), (1100, 2051), (1101, 2048)])
def test_large_products_of_odd_rows(N, K, layout):
    # Large enough that rows of an odd length are copied to whole pieces first.
    sizes, spare, dt = [1100, 0, 900], 3, torch.bfloat16
    M = sum(sizes) + spare
    say(f"[odd rows] M={M} N={N} K={K} layout={layout}")
    a, b = normal((M, K), dt, 15), weights(3, N, K, dt, layout, 16)
    a[-1] = float("nan")                                           # a row of no group, behind the last group's
    ends = ends_of(sizes).cuda()
    ref, err = grouped_reference(a, b, sizes, layout, True)
    out, whole = guarded((M, N), dt)
    gr.gemm_relu_grouped(a.cuda(), b.cuda(), ends, out=out, b_layout=layout)
    torch.cuda.synchronize()
    assert whole()
    assert_close(out, ref, err, "C")
    for relu in (True, False):
        dc, c = normal((M, N), dt, 17), normal((M, N), dt, 18).clamp_min(0)
        ra, ea, rb, eb = backward_reference(dc, c, a, b, sizes, layout, relu)
        da, whole_a = guarded((M, K), dt)
        db, whole_b = guarded(tuple(b.shape), dt)
        gr.gemm_relu_grouped_backward(dc.cuda(), c.cuda(), a.cuda(), b.cuda(), ends, b_layout=layout, da=da, db=db, relu=relu)
        torch.cuda.synchronize()
        assert whole_a() and whole_b()
        assert_close(da, ra, ea, "dA")
        assert_close(db, rb, eb, "dB")


@pytest.mark.parametrize("layout", [gr.B_KN, gr.B_NK])
def test_adapters_of_odd_rows_in_large_products(layout):
    sizes, N, K = [900, 1, 1, 700, 398], 2051, 1901
    x, w, u, v, scales, ends, ids = adapter_inputs(sizes, 0, N, K, 20, 3, torch.float16, layout, 66)
    ref, err = adapter_reference(x, w, u, v, scales, sizes, ids, layout, True)
    out, whole = guarded((x.shape[0], N), torch.float16)
    gr.gemm_relu_adapters(*(t.cuda() for t in (x, w, u, v, scales, ends, ids)), out=out, b_layout=layout)
    torch.cuda.synchronize()
    assert whole()
    assert_close(out, ref, err, "C")


@pytest.mark.parametrize("layout", [gr.B_KN, gr.B_NK])
@pytest.mark.parametrize("N,K", [(64, 64), (66, 70), (40, 52)])
def test_grouped_unaligned_matrices(N, K, layout):
    sizes = [70, 0, 3, 60]
    a, b = normal((133, K), torch.bfloat16, 5), weights(4, N, K, torch.bfloat16, layout, 6)
    ref, err = grouped_reference(a, b, sizes, layout, True)
    out, whole = guarded((133, N), torch.bfloat16, shift=1)
    gr.gemm_relu_grouped(unaligned(a), unaligned(b), ends_of(sizes).cuda(), out=out, b_layout=layout)
    torch.cuda.synchronize()
    assert whole()
    assert_close(out, ref, err, "C")


@pytest.mark.parametrize("layout", [gr.B_KN, gr.B_NK])
@pytest.mark.parametrize("rows", [2, 40, 200])
def test_grouped_keeps_infinities_and_nan_to_their_group(rows, layout):
    # A group's weights and a row's entries may be anything: no other row sees them.
    sizes, N, K = [rows, rows + 1, rows], 72, 96
    M = sum(sizes) + 2
    a, b = normal((M, K), torch.float16, 7), weights(3, N, K, torch.float16, layout, 8)
    b[1] = float("nan")
    b[1].view(-1)[::3] = float("inf")
    a[0] = float("inf")
    a[-1] = float("nan")                                           # a row of no group
    got = gr.gemm_relu_grouped(a.cuda(), b.cuda(), ends_of(sizes).cuda(), b_layout=layout, relu=False).cpu()
    clean = [r for r in range(1, M) if not rows <= r < 2 * rows + 1 and r < M - 2]
    ref, err = grouped_reference(a, b, sizes, layout, False)
    assert_close(got[clean], ref[clean], err[clean], "C")
    assert not torch.isfinite(got[rows:2 * rows + 1]).any() and not torch.isfinite(got[0]).any()
    assert (got[-2:] == 0).all()


@pytest.mark.parametrize("ends", [[5, 2, 9], [-4, 100, 3], [2 ** 31 - 1, -2 ** 31, 7], [0, 0, 0], [50, 50, 50]])
def test_grouped_bad_ends_stay_inside(ends):
    # Ends that decrease or leave [0, M] give no error, and nothing outside C is written.
    M, N, K = 40, 72, 64
    a, b = normal((M, K), torch.float16, 9).cuda(), weights(3, N, K, torch.float16, gr.B_KN, 10).cuda()
    out, whole = guarded((M, N), torch.float16)
    gr.gemm_relu_grouped(a, b, torch.tensor(ends, dtype=torch.int32).cuda(), out=out)
    da, whole_a = guarded((M, K), torch.float16)
    db, whole_b = guarded((3, K, N), torch.float16)
    gr.gemm_relu_grouped_backward(out, out, a, b, torch.tensor(ends, dtype=torch.int32).cuda(), da=da, db=db)
    torch.cuda.synchronize()
    assert whole() and whole_a() and whole_b()
    assert not (out == 777.0).any() and not (da == 777.0).any() and not (db == 777.0).any()


def test_grouped_empty_calls():
    a = torch.zeros((0, 8), dtype=torch.float16, device="cuda")
    b = torch.ones((2, 8, 4), dtype=torch.float16, device="cuda")
    ends = torch.zeros(2, dtype=torch.int32, device="cuda")
    assert gr.gemm_relu_grouped(a, b, ends).shape == (0, 4)
    da, db = gr.gemm_relu_grouped_backward(a.new_zeros((0, 4)), a.new_zeros((0, 4)), a, b, ends)
    assert da.shape == (0, 8) and (db == 0).all()                  # no rows: the sums are empty
    out = gr.gemm_relu_grouped(a.new_zeros((5, 0)), b[:, :0].contiguous(), torch.tensor([2, 5]).int().cuda())
    assert out.shape == (5, 4) and (out.view(torch.int16) == 0).all()
    da, db = gr.gemm_relu_grouped_backward(a.new_zeros((5, 0)), a.new_zeros((5, 0)), a.new_ones((5, 8)),
                                           b[:, :, :0].contiguous(), torch.tensor([2, 5]).int().cuda())
    assert (da == 0).all() and da.shape == (5, 8) and db.shape == (2, 8, 0)


def test_grouped_refusals():
    a = torch.zeros((4, 8), dtype=torch.float16, device="cuda")
    b = torch.zeros((2, 8, 8), dtype=torch.float16, device="cuda")
    e = torch.tensor([1, 4], dtype=torch.int32, device="cuda")
    bad = [
        (lambda: gr.gemm_relu_grouped(a.float(), b.float(), e), TypeError),
        (lambda: gr.gemm_relu_grouped(a, b.bfloat16(), e), TypeError),
        (lambda: gr.gemm_relu_grouped(a, b, e.long()), TypeError),
        (lambda: gr.gemm_relu_grouped(a, b, e.cpu()), ValueError),
        (lambda: gr.gemm_relu_grouped(a, b, e[:1].contiguous()), ValueError),
        (lambda: gr.gemm_relu_grouped(a, b[0], e), ValueError),
        (lambda: gr.gemm_relu_grouped(a[:, :4], b, e), ValueError),
        (lambda: gr.gemm_relu_grouped(a[:, :4].contiguous(), b, e), ValueError),
        (lambda: gr.gemm_relu_grouped(a, b, e, out=a.new_zeros((4, 9))), ValueError),
        (lambda: gr.gemm_relu_grouped(a, b, e, b_layout=2), ValueError),
        (lambda: gr.gemm_relu_grouped(a, b, e, out=a), binding.GemmReluError),
        (lambda: gr.gemm_relu_grouped_backward(a, None, a, b, e), TypeError),
        (lambda: gr.gemm_relu_grouped_backward(a, a, a, b, e, need_da=False, need_db=False), ValueError),
        (lambda: gr.gemm_relu_grouped_backward(a, a[:3], a, b, e), ValueError),
        (lambda: gr.gemm_relu_grouped_backward(a, a, a, b, e, workspace=torch.zeros(64, device="cuda")),
         binding.GemmReluError),
        (lambda: gr.gemm_relu_adapters(a, b[0], b, b, torch.ones(2, device="cuda").double(), e, e), TypeError),
        (lambda: gr.gemm_relu_adapters(a, b[0], b, b, torch.ones(3, device="cuda"), e, e), ValueError),
        (lambda: gr.gemm_relu_adapters(a, b[0], b, b, torch.ones(2, device="cuda"), e, e[:1].contiguous()), ValueError),
        (lambda: gr.gemm_relu_adapters(a, b[0], b[:, :4].contiguous(), b, torch.ones(2, device="cuda"), e, e),
         ValueError),
    ]
    for call, error in bad:
        with pytest.raises(error):
            call()


# ---------------------------------------------------------------- gradients

def backward_reference(dc, c, a, b, sizes, layout, relu):
    d = dc.double()
    if relu:
        d = torch.where(c > 0, d, torch.zeros_like(d))
    a64, b64 = a.double(), as_kn(b, layout).double()
    da, da_mag = torch.zeros_like(a64), torch.zeros_like(a64)
    db, db_err = torch.zeros_like(b64), torch.zeros_like(b64)
    N = dc.shape[1]
    for e, lo, hi in spans(sizes):
        if hi > lo:
            da[lo:hi], da_mag[lo:hi] = d[lo:hi] @ b64[e].t(), d[lo:hi].abs() @ b64[e].abs().t()
            db[e] = a64[lo:hi].t() @ d[lo:hi]
            db_err[e] = (hi - lo) * 2.0 ** -23 * (a64[lo:hi].abs().t() @ d[lo:hi].abs())
    return da, N * 2.0 ** -23 * da_mag, as_kn(db, layout), as_kn(db_err, layout)


@pytest.mark.parametrize("relu", [True, False])
@pytest.mark.parametrize("layout", [gr.B_KN, gr.B_NK])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("shape", range(len(SHAPES)))
def test_grouped_backward(shape, dtype, layout, relu):
    sizes, spare, N, K = SHAPES[shape]
    M = sum(sizes) + spare
    say(f"[grouped_backward] {sizes[:6]} M={M} N={N} K={K} {dtype} layout={layout} relu={relu}")
    dt = DT[dtype]
    a, b = normal((M, K), dt, 21 + shape), weights(len(sizes), N, K, dt, layout, 22 + shape)
    dc, c = normal((M, N), dt, 23 + shape), normal((M, N), dt, 24 + shape).clamp_min(0)
    ra, ea, rb, eb = backward_reference(dc, c, a, b, sizes, layout, relu)
    da, whole_a = guarded((M, K), dt)
    db, whole_b = guarded(tuple(b.shape), dt)
    args = (dc.cuda(), c.cuda() if relu else None)
    gr.gemm_relu_grouped_backward(*args, a.cuda(), b.cuda(), ends_of(sizes).cuda(), b_layout=layout, relu=relu,
                                  da=da, db=db)
    torch.cuda.synchronize()
    assert whole_a() and whole_b()
    assert_close(da, ra, ea, "dA")
    assert_close(db, rb, eb, "dB")
    # one gradient at a time, without what it does not need
    only_a = gr.gemm_relu_grouped_backward(*args, None, b.cuda(), ends_of(sizes).cuda(), b_layout=layout, relu=relu,
                                           need_db=False)
    only_b = gr.gemm_relu_grouped_backward(*args, a.cuda(), None, ends_of(sizes).cuda(), b_layout=layout, relu=relu,
                                           need_da=False)
    assert only_a[1] is None and only_b[0] is None
    assert torch.equal(only_a[0], da) and torch.equal(only_b[1], db)


def test_grouped_backward_keeps_infinities_and_nan_to_their_rows():
    sizes, N, K = [40, 33, 50], 72, 96
    M = sum(sizes) + 3
    dt = torch.float16
    a, b = normal((M, K), dt, 31), weights(3, N, K, dt, gr.B_KN, 32)
    dc, c = normal((M, N), dt, 33), normal((M, N), dt, 34).abs().clamp_min(0.1)
    a[50], dc[51] = float("inf"), float("nan")                      # group 1
    a[-1], dc[-1], dc[-2] = float("nan"), float("inf"), float("nan")    # rows of no group
    c[3] = 0
    dc[3] = float("inf")                                            # masked: contributes nothing
    b[1] = float("nan")
    ra, ea, rb, eb = backward_reference(dc, c, a, b, sizes, gr.B_KN, True)
    da, db = gr.gemm_relu_grouped_backward(dc.cuda(), c.cuda(), a.cuda(), b.cuda(), ends_of(sizes).cuda())
    clean = [r for r in range(M - 3) if not 40 <= r < 73]
    assert_close(da.cpu()[clean], ra[clean], ea[clean], "dA")
    assert (da[-3:] == 0).all() and (da[3] == 0).all()
    for e in (0, 2):
        assert_close(db[e], rb[e], eb[e], "dB")


def test_grouped_backward_against_differences():
    # d(sum(dC * C))/dB along a direction: central differences of the 64-bit forward pass.
    sizes, N, K = [9, 0, 14], 24, 40
    dt = torch.float16
    a, b = normal((23, K), dt, 41), weights(3, N, K, dt, gr.B_KN, 42)
    dc = normal((23, N), dt, 43)
    c = gr.gemm_relu_grouped(a.cuda(), b.cuda(), ends_of(sizes).cuda())
    da, db = gr.gemm_relu_grouped_backward(dc.cuda(), c, a.cuda(), b.cuda(), ends_of(sizes).cuda())

    def loss(a64, b64):
        out = torch.zeros((23, N), dtype=torch.float64)
        for e, lo, hi in spans(sizes):
            out[lo:hi] = (a64[lo:hi] @ b64[e]).clamp_min(0)
        return float((out * dc.double()).sum())

    g = torch.Generator().manual_seed(44)
    h, u = 2.0 ** -20, torch.finfo(dt).eps / 2
    for base, grad in ((a, da), (b, db)):
        move = torch.randn(base.shape, generator=g, dtype=torch.float64)
        args = [a.double(), b.double()]
        at = 0 if base is a else 1
        plus, minus = list(args), list(args)
        plus[at], minus[at] = args[at] + h * move, args[at] - h * move
        diff = (loss(*plus) - loss(*minus)) / (2 * h)
        g64 = grad.cpu().double()
        # The gradient's entries are off by u relative (their fp32 sums by far less), the
        # difference by a kink within h: a sum crosses zero with odds of about h.
        assert abs(diff - float((g64 * move).sum())) <= 2 * u * float((g64 * move).abs().sum()) + 1e-3


# ---------------------------------------------------------------- adapters

def adapter_inputs(sizes, spare, N, K, rank, count, dtype, layout, seed):
    M = sum(sizes) + spare
    x, w = normal((M, K), dtype, seed), normal((K, N), dtype, seed + 1, K ** -0.5)
    u, v = normal((count, K, rank), dtype, seed + 2, K ** -0.5), normal((count, rank, N), dtype, seed + 3)
    g = torch.Generator().manual_seed(seed + 4)
    scales = torch.rand(count, generator=g) * 2 - 0.5
    ids = torch.randint(-1, count, (len(sizes),), generator=g, dtype=torch.int32)
    if layout == gr.B_NK:
        w, u, v = w.t().contiguous(), u.transpose(1, 2).contiguous(), v.transpose(1, 2).contiguous()
    return x, w, u, v, scales, ends_of(sizes), ids


def adapter_reference(x, w, u, v, scales, sizes, ids, layout, relu):
    x64, w64 = x.double(), (w.t() if layout == gr.B_NK else w).double()
    u64, v64 = as_kn(u, layout).double(), as_kn(v, layout).double()
    K, rank = x.shape[1], u64.shape[2]
    eps = 2.0 ** -23
    half = torch.finfo(x.dtype).eps / 2
    ref, mag, err = x64 @ w64, x64.abs() @ w64.abs(), 0.0
    err = K * eps * mag
    for s, lo, hi in spans(sizes):
        i = int(ids[s])
        if 0 <= i < u.shape[0] and hi > lo:
            z = float(scales[i]) * (x64[lo:hi] @ u64[i])
            dz = (K + 2) * eps * abs(float(scales[i])) * (x64[lo:hi].abs() @ u64[i].abs())
            dz = dz + half * half * z.abs() + 2.0 ** -24 * z.abs().max(dim=1, keepdim=True).values
            ref[lo:hi] += z @ v64[i]
            # the low-rank sum's own additions (two parts each), and the final one into the shared sum
            err[lo:hi] += dz @ v64[i].abs() + (2 * rank + 8) * eps * (z.abs() @ v64[i].abs() + mag[lo:hi])
    return (ref.clamp_min(0) if relu else ref), err


# (segment sizes, spare rows, N, K, rank, adapters)
ADAPTER_SHAPES = [
    ([1], 0, 1, 1, 1, 1),
    ([1], 0, 256, 512, 16, 3),                        # one token
    ([1] * 13, 0, 264, 136, 8, 4),                    # a decoding step
    ([1] * 70, 2, 192, 256, 16, 9),                   # more segments than a wave has lanes
    ([1, 1, 40, 1, 7, 0, 20, 1], 3, 130, 75, 12, 5),  # a mixed batch, odd sizes
    ([100, 0, 160], 0, 384, 320, 64, 2),              # prompts
    ([129, 1, 1, 300], 0, 128, 192, 33, 3),
    ([64, 64], 5, 72, 100, 256, 2),
    ([1] * 300, 0, 96, 64, 4, 40),
    ([700, 500], 0, 520, 264, 128, 2),
]


@pytest.mark.parametrize("relu", [True, False])
@pytest.mark.parametrize("layout", [gr.B_KN, gr.B_NK])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("shape", range(len(ADAPTER_SHAPES)))
def test_adapters(shape, dtype, layout, relu):
    sizes, spare, N, K, rank, count = ADAPTER_SHAPES[shape]
    say(f"[adapters] {sizes[:6]} N={N} K={K} rank={rank} {dtype} layout={layout} relu={relu}")
    x, w, u, v, scales, ends, ids = adapter_inputs(sizes, spare, N, K, rank, count, DT[dtype], layout, 51 + 7 * shape)
    ref, err = adapter_reference(x, w, u, v, scales, sizes, ids, layout, relu)
    out, whole = guarded((x.shape[0], N), DT[dtype])
    gr.gemm_relu_adapters(*(t.cuda() for t in (x, w, u, v, scales, ends, ids)), out=out, b_layout=layout, relu=relu)
    torch.cuda.synchronize()
    assert whole()
    assert_close(out, ref, err, "C")


@pytest.mark.parametrize("layout", [gr.B_KN, gr.B_NK])
@pytest.mark.parametrize("config", CONFIGS)
@pytest.mark.parametrize("sizes,N,K,rank", [([1] * 37 + [100, 0, 300], 264, 136, 16), ([1500, 1300], 2056, 64, 40),
                                            ([1] * 90, 64, 320, 64)])
def test_adapter_kernels(sizes, N, K, rank, config, layout):
    dt = torch.bfloat16 if rank == 16 else torch.float16
    say(f"[adapters] {sizes[:3]} N={N} K={K} rank={rank} {dt} layout={layout} config={config}")
    x, w, u, v, scales, ends, ids = adapter_inputs(sizes, 1, N, K, rank, 6, dt, layout, 65)
    ref, err = adapter_reference(x, w, u, v, scales, sizes, ids, layout, True)
    out, whole = guarded((x.shape[0], N), dt)
    gr.gemm_relu_adapters(*(t.cuda() for t in (x, w, u, v, scales, ends, ids)), out=out, b_layout=layout, config=config)
    torch.cuda.synchronize()
    assert whole()
    assert_close(out, ref, err, "C")


@pytest.mark.parametrize("layout", [gr.B_KN, gr.B_NK])
def test_adapters_unaligned_matrices(layout):
    sizes = [1, 30, 0, 2, 50]
    x, w, u, v, scales, ends, ids = adapter_inputs(sizes, 0, 72, 64, 16, 3, torch.bfloat16, layout, 61)
    ref, err = adapter_reference(x, w, u, v, scales, sizes, ids, layout, True)
    out, whole = guarded((83, 72), torch.bfloat16, shift=1)
    gr.gemm_relu_adapters(*(unaligned(t) for t in (x, w, u, v)), scales.cuda(), ends.cuda(), ids.cuda(), out=out,
                          b_layout=layout)
    torch.cuda.synchronize()
    assert whole()
    assert_close(out, ref, err, "C")


@pytest.mark.parametrize("rows", [1, 20, 150])
@pytest.mark.parametrize("layout", [gr.B_KN, gr.B_NK])
def test_adapters_never_reach_other_rows(layout, rows):
    # Neighbouring requests share MFMA blocks: an adapter full of infinities and NaN, and ids
    # outside the table, leave the others exactly as they are.
    sizes = [rows] * 5
    x, w, u, v, scales, ends, _ = adapter_inputs(sizes, 0, 80, 96, 20, 3, torch.float16, layout, 71)
    ids = torch.tensor([0, 1, -1, 3, 2], dtype=torch.int32)
    ref, err = adapter_reference(x, w, u, v, scales, sizes, ids, layout, False)
    u[1], v[1], scales[1] = float("inf"), float("nan"), float("inf")
    got = gr.gemm_relu_adapters(*(t.cuda() for t in (x, w, u, v, scales, ends, ids)), b_layout=layout, relu=False)
    keep = [r for r in range(5 * rows) if not rows <= r < 2 * rows]
    assert_close(got[keep], ref[keep], err[keep], "C")
    assert not torch.isfinite(got[rows:2 * rows]).any()


def test_adapters_intermediate_neither_overflows_nor_vanishes():
    # x @ U far outside fp16's range, and V the other way: the products are ordinary numbers.
    K, N, rank, dt = 64, 48, 8, torch.float16
    x, w = normal((3, K), dt, 81, 100.0), torch.zeros((K, N), dtype=dt)
    u, v = normal((2, K, rank), dt, 82, 2000.0), normal((2, rank, N), dt, 83, 2.0 ** -13)
    u[1] = u[1] * 2.0 ** -24
    scales = torch.tensor([0.1, 2.0 ** 14])
    sizes, ids = [1, 1, 1], torch.tensor([0, 1, 0], dtype=torch.int32)
    ref, err = adapter_reference(x, w, u, v, scales, sizes, ids, gr.B_KN, False)
    got = gr.gemm_relu_adapters(*(t.cuda() for t in (x, w, u, v, scales, ends_of(sizes), ids)), relu=False)
    assert_close(got, ref, err, "C")


# ---------------------------------------------------------------- streams, graphs, repeats

def calls(dt=torch.float16):
    """One call of each operator on fixed buffers, decode-sized and larger, and what it writes."""
    got = []
    for sizes, N, K in (([1, 0, 2, 1], 512, 1024), ([300, 0, 212], 256, 320)):
        M = sum(sizes)
        a, b = normal((M, K), dt, 91).cuda(), weights(len(sizes), N, K, dt, gr.B_KN, 92).cuda()
        ends, c = ends_of(sizes).cuda(), torch.empty((M, N), dtype=dt, device="cuda")
        got.append((lambda a=a, b=b, e=ends, c=c, **kw: gr.gemm_relu_grouped(a, b, e, out=c, **kw), [a], [c]))
        dc, cc = normal((M, N), dt, 93).cuda(), normal((M, N), dt, 94).clamp_min(0).cuda()
        da, db = torch.empty_like(a), torch.empty_like(b)
        got.append((lambda dc=dc, cc=cc, a=a, b=b, e=ends, da=da, db=db, **kw:
                    gr.gemm_relu_grouped_backward(dc, cc, a, b, e, da=da, db=db, **kw), [dc], [da, db]))
        x, w, u, v, scales, e2, ids = (t.cuda() for t in adapter_inputs(sizes, 0, N, K, 16, 3, dt, gr.B_KN, 95))
        y = torch.empty((M, N), dtype=dt, device="cuda")
        got.append((lambda x=x, w=w, u=u, v=v, s=scales, e=e2, i=ids, y=y, **kw:
                    gr.gemm_relu_adapters(x, w, u, v, s, e, i, out=y, **kw), [x], [y]))
    return got


@pytest.mark.parametrize("which", range(6))
def test_graph_replays_match_eager_calls(which):
    call, ins, outs = calls()[which]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        call()
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for k in range(4):
        for t in ins:
            t.copy_(normal(tuple(t.shape), t.dtype, 100 + k))
        for t in outs:
            t.fill_(777.0)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        first = [t.clone() for t in outs]
        for t in outs:
            t.fill_(777.0)
        call()                                       # eager, on the same inputs
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(first, outs)), (which, k)


@pytest.mark.parametrize("which", range(6))
def test_repeats_side_streams_and_a_shared_workspace(which):
    every = calls()
    call, ins, outs = every[which]
    call()
    torch.cuda.synchronize()
    want = [t.clone() for t in outs]
    need = 64 << 20
    ws = torch.zeros(need, dtype=torch.uint8, device="cuda")
    for k in range(3):
        for t in outs:
            t.fill_(777.0)
        every[(which + k) % len(every)][0](workspace=ws)          # another call leaves its scratch behind
        call(workspace=ws)
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(want, outs))
        assert (ws[:groups.COUNTER_BYTES] == 0).all()             # the counters are back at zero
    s = torch.cuda.Stream()
    for t in outs:
        t.fill_(777.0)
    torch.cuda.synchronize()
    call(stream=s)
    s.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(want, outs))


def test_two_streams_at_once():
    every = calls()
    for call, _, _ in every:
        call()
    torch.cuda.synchronize()
    want = [[t.clone() for t in outs] for _, _, outs in every]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        for k, (call, _, _) in enumerate(every):
            call(stream=streams[k % 2])
    torch.cuda.synchronize()
    for k, (_, _, outs) in enumerate(every):
        assert all(torch.equal(x, y) for x, y in zip(want[k], outs)), k

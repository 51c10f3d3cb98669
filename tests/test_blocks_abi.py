"""Host-side checks of gemm_relu_blocks.h: exported symbols, workspace sizes, the refusal of bad arguments before
any device work, and the quantizer's division.  No GPU is needed and no kernel is launched."""
import ctypes
import os
import re
from fractions import Fraction

import numpy as np
import pytest
import torch

import tiled_dense_gemm_relu_amd as gr
from tiled_dense_gemm_relu_amd import blocks, groups

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "gemm_relu_blocks.h")

# Fake, well separated addresses that are never dereferenced.
A, B, C, D, E, F, G, H, W = (i << 40 for i in range(1, 10))


@pytest.fixture(scope="module")
def lib():
    return blocks._library()


def test_library_exports_every_declared_symbol(lib):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"^\s*(?:int|int64_t)\s+(gemm_relu\w*)\s*\(", text, flags=re.M))
    assert names == {"gemm_relu_quantize_blocks", "gemm_relu_blocks", "gemm_relu_blocks_backward",
                     "gemm_relu_blocks_backward_workspace", "gemm_relu_experts", "gemm_relu_experts_workspace"}
    for name in names:
        assert ctypes.cast(getattr(lib, name), ctypes.c_void_p).value


def quantize(lib, x=A, mask=None, q=B, s=C, qt=D, st=E, count=1, R=4, cols=8, ldq=16, ldqt=16, dtype=0, fmt=0, form=0, power=0):
    return lib.gemm_relu_quantize_blocks(x, mask, q, s, qt, st, count, R, cols, ldq, ldqt, dtype, fmt, form, power, None)


def product(lib, a=A, sa=B, b=C, sb=D, ends=E, c=F, M=4, N=8, K=8, groups=2, lda=16, ldb=16, fa=0, fb=1, form=1, dtype=0,
            relu=1, config=-1):
    return lib.gemm_relu_blocks(a, sa, b, sb, ends, c, M, N, K, groups, lda, ldb, fa, fb, form, dtype, relu, config, None)


def backward(lib, dc=A, c=B, xt=C, sxt=D, wt=E, swt=F, dx=G, dw=H, M=4, N=8, K=8, ldxt=16, ldwt=16, fmt=1, fx=0, fw=0, dtype=0,
             relu=1, ws=W, ws_bytes=1 << 30):
    return lib.gemm_relu_blocks_backward(dc, c, xt, sxt, wt, swt, dx, dw, M, N, K, ldxt, ldwt, fmt, fx, fw, dtype, relu, ws,
                                         ws_bytes, None)


def experts(lib, x=A, w1=B, s1=C, w2=D, s2=E, logits=F, ids=G, weights=G + 4096, y=H, T=4, N=8, K=8, hidden=8, E_=3, top=2, ld1=16,
            ld2=16, renorm=1, dtype=0, fmt=0, layout=1, ws=W, ws_bytes=1 << 30):
    return lib.gemm_relu_experts(x, w1, s1, w2, s2, logits, ids, weights, y, T, N, K, hidden, E_, top, ld1, ld2, renorm, dtype,
                                 fmt, layout, ws, ws_bytes, None)


BIG = (1 << 20) + 1


@pytest.mark.parametrize("args,code", [
    ({"dtype": 2}, -2), ({"fmt": 2}, -2), ({"form": 2}, -9), ({"power": 2}, -1), ({"R": -1}, -1), ({"cols": BIG, "ldq": BIG + 15}, -7),
    ({"count": 65536}, -7), ({"q": None, "qt": None}, -1), ({"ldq": 7}, -4), ({"ldq": 24}, -4), ({"ldqt": 8}, -4),
    ({"ldq": (1 << 21) + 16}, -7), ({"x": None}, -1), ({"x": A + 1}, -4), ({"mask": A + 1}, -4), ({"q": B + 8}, -4), ({"s": C + 2}, -4),
    ({"st": None}, -1), ({"s": None}, -1), ({"q": A}, -3), ({"qt": B}, -3), ({"s": B}, -3), ({"mask": D}, -3), ({"st": C}, -3)])
def test_quantize_refuses(lib, args, code):
    assert quantize(lib, **args) == code


@pytest.mark.parametrize("args,code", [
    ({"dtype": 2}, -2), ({"fa": 2}, -2), ({"fb": -1}, -2), ({"form": 2}, -9), ({"M": -1}, -1), ({"N": BIG}, -7), ({"K": BIG, "lda": BIG + 15}, -7),
    ({"groups": 0}, -1), ({"groups": 65536}, -7), ({"relu": 2}, -1), ({"ends": None}, -1), ({"config": -2}, -8), ({"config": 4}, -8),
    ({"lda": 8}, -4), ({"ldb": 7}, -4), ({"lda": 1 << 22}, -7), ({"a": None}, -1), ({"b": None}, -1), ({"c": None}, -1), ({"sa": None}, -1),
    ({"sb": None}, -1), ({"a": A + 8}, -4), ({"b": C + 8}, -4), ({"c": F + 1}, -4), ({"sa": B + 2}, -4), ({"ends": E + 2}, -4),
    ({"c": A}, -3), ({"c": C}, -3), ({"c": B}, -3), ({"c": D}, -3), ({"c": E}, -3)])
def test_product_refuses(lib, args, code):
    assert product(lib, **args) == code


@pytest.mark.parametrize("args,code", [
    ({"dtype": 2}, -2), ({"fmt": 2}, -2), ({"fx": 2}, -2), ({"fw": 2}, -2), ({"relu": 2}, -1), ({"M": -1}, -1), ({"K": BIG}, -7),
    ({"dx": None, "dw": None}, -1), ({"ldxt": 8}, -4), ({"ldwt": 3}, -4), ({"dc": None}, -1), ({"c": None}, -1), ({"xt": None}, -1),
    ({"wt": None}, -1), ({"sxt": None}, -1), ({"swt": None}, -1), ({"xt": C + 8}, -4), ({"wt": E + 8}, -4), ({"dx": G + 1}, -4),
    ({"dx": A}, -3), ({"dw": B}, -3), ({"dw": G + 2}, -3), ({"dx": E}, -3), ({"dw": D}, -3), ({"ws": 0}, -10), ({"ws": W + 128}, -10),
    ({"ws_bytes": 1000}, -10), ({"ws": A}, -3), ({"ws": C}, -3), ({"ws": G}, -3)])
def test_backward_refuses(lib, args, code):
    assert backward(lib, **args) == code


@pytest.mark.parametrize("args,code", [
    ({"dtype": 2}, -2), ({"fmt": 2}, -2), ({"fmt": -2}, -2), ({"layout": 2}, -9), ({"layout": 0}, -9), ({"T": -1}, -1), ({"T": 65}, -7),
    ({"E_": 0}, -1), ({"E_": 1025}, -7), ({"top": 0}, -1), ({"top": 4}, -1), ({"top": 17, "E_": 20}, -7), ({"renorm": 2}, -1),
    ({"K": -1}, -1), ({"hidden": BIG}, -7), ({"N": BIG}, -7), ({"ld1": 8}, -4), ({"ld2": 24}, -4), ({"x": None}, -1), ({"w1": None}, -1),
    ({"w2": None}, -1), ({"s1": None}, -1), ({"s2": None}, -1), ({"ids": None}, -1), ({"weights": None}, -1), ({"y": None}, -1),
    ({"w1": B + 8}, -4), ({"x": A + 1}, -4), ({"logits": F + 2}, -4), ({"ids": G + 2}, -4), ({"y": A}, -3), ({"y": B}, -3), ({"y": F}, -3),
    ({"ids": F}, -3), ({"weights": G}, -3), ({"ws": 0}, -10), ({"ws": W + 8}, -10), ({"ws_bytes": 65536}, -10), ({"ws": D}, -3),
    ({"ws": G}, -3), ({"ws": H}, -3),
    # the intermediate, or the partial sums, past what a descriptor covers
    ({"T": 64, "top": 16, "E_": 16, "hidden": 1 << 20, "ld2": 1 << 20}, -7), ({"T": 64, "top": 16, "E_": 16, "N": 1 << 20}, -7)])
def test_experts_refuse(lib, args, code):
    assert experts(lib, **args) == code


def test_empty_outputs_need_no_device(lib):
    assert quantize(lib, x=None, R=0) == 0 and quantize(lib, x=None, cols=0) == 0 and quantize(lib, count=0) == 0
    assert product(lib, a=None, sa=None, c=None, M=0) == 0 and product(lib, b=None, sb=None, c=None, N=0) == 0
    assert backward(lib, K=0) == 0
    assert experts(lib, x=None, y=None, ids=None, weights=None, logits=None, T=0) == 0


def test_workspace_sizes():
    # 8-bit copies both ways at whole 16-byte pieces, and their scales
    need = gr.blocks_backward_workspace_bytes(100, 200, 300)
    assert need >= groups.COUNTER_BYTES + 100 * 208 + 200 * 112 + 4 * (100 * 2 + 200)
    # every choice's intermediate in two 16-bit parts, and its sums
    need = gr.experts_workspace_bytes(7, 70, 33, 5, 2)
    assert need >= groups.COUNTER_BYTES + 7 * 2 * (2 * 2 * 40 + 4 * 70)
    for sizes in ((0, 16, 16, 4, 2), (3, 0, 16, 4, 2), (3, 16, 0, 4, 2)):
        assert gr.experts_workspace_bytes(*sizes) >= groups.COUNTER_BYTES
    for call in (lambda: gr.blocks_backward_workspace_bytes(-1, 1, 1), lambda: gr.experts_workspace_bytes(65, 1, 1, 1, 1),
                 lambda: gr.experts_workspace_bytes(1, 1, 1, 1, 2), lambda: gr.experts_workspace_bytes(1, 1, 1, 1, 1, 7)):
        with pytest.raises(gr.GemmReluError):
            call()


def test_python_refuses_what_is_not_a_gpu_tensor():
    t, q, s = torch.zeros((2, 2), dtype=torch.float16), torch.zeros((2, 16), dtype=torch.float8_e4m3fn), torch.ones((1, 2))
    for call in (lambda: gr.quantize_blocks(t), lambda: gr.gemm_relu_blocks(q, s, q, s[:, :1]), lambda: gr.linear_blocks(t, t),
                 lambda: gr.gemm_relu_blocks_backward(t, t, q, s, q, s), lambda: gr.gemm_relu_experts(t, t[None], t[None], t, 1)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: gr.quantize_blocks(None), lambda: gr.gemm_relu_blocks(None, s, q, s), lambda: gr.linear_blocks(None, t),
                 lambda: gr.gemm_relu_blocks_backward(None, t, q, s, q, s), lambda: gr.gemm_relu_experts(None, t, t, t, 1)):
        with pytest.raises(TypeError):
            call()


def test_quotients_are_correctly_rounded():
    """The kernel's quotient (a product with the rounded reciprocal of the scale, corrected by its remainder) for
    every pair of 11-bit significands, of x and of the magnitude that the scale is made of (8-bit ones of bf16 are
    among them; the formats' largest values, 448 and 57344, have one significand, 1.75)."""
    m = np.arange(1024, 2048, dtype=np.float64) / 1024
    x = m.astype(np.float32)
    for amax in m:
        s = np.float32(amax / 448.0)                             # (a quotient of 11 and 3 bits in 64: one rounding)
        inverse = np.float32(1.0 / np.float64(s))
        t = (x.astype(np.float64) * np.float64(inverse)).astype(np.float32)          # 48 bits in 53: one rounding
        r = (x.astype(np.float64) - t.astype(np.float64) * np.float64(s)).astype(np.float32)
        wide = t.astype(np.longdouble) + r.astype(np.longdouble) * np.longdouble(inverse)
        q = wide.astype(np.float32)
        # wide was rounded to 64 bits: where that is half-way between two floats, by the exact sum
        ulp = np.spacing(np.abs(q)).astype(np.longdouble)
        for i in np.nonzero(np.abs(np.abs(wide - q.astype(np.longdouble)) - ulp / 2) < ulp * 2.0 ** -30)[0]:
            exact = Fraction(float(t[i])) + Fraction(float(r[i])) * Fraction(float(inverse))
            near = [np.nextafter(q[i], np.float32(-np.inf)), q[i], np.nextafter(q[i], np.float32(np.inf))]
            q[i] = min(near, key=lambda v: (abs(Fraction(float(v)) - exact), int(np.float32(v).view(np.int32)) & 1))
        # correctly rounded: x - q s is at most half a unit of q times s (products of 24 bits, exact in 64)
        off = np.abs(x.astype(np.float64) - q.astype(np.float64) * np.float64(s))
        assert (off <= np.spacing(q).astype(np.float64) / 2 * np.float64(s)).all()

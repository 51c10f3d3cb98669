"""The expert layer for a few tokens on the GPU, against 64-bit references."""
import math

import pytest
import torch

import tiled_dense_gemm_relu_amd as gr

pytestmark = pytest.mark.gpu

E4M3, E5M2 = torch.float8_e4m3fn, torch.float8_e5m2
DEV = "cuda"
KINDS = ["nk", "kn", "e4m3", "e5m2"]


def nb(n):
    return (n + 127) // 128


def pitched(q, pitch=None):
    """A GPU copy with rows at multiples of 16 bytes, NaN in the bytes between."""
    pitch = pitch or (q.shape[-1] + 15) // 16 * 16
    raw = torch.full(q.shape[:-1] + (pitch,), 0x7f, dtype=torch.uint8)
    raw[..., : q.shape[-1]] = q.view(torch.uint8)
    return raw.to(DEV)[..., : q.shape[-1]].view(q.dtype)


class Layer:
    """Random weights of one kind: on the GPU as the call takes them, and in 64 bits as (experts, in, out)."""

    def __init__(self, kind, dtype, E, K, H, N, seed, integers=False):
        g = torch.Generator().manual_seed(seed)

        def values(shape, scale):
            return torch.randint(-2, 3, shape, generator=g).float() if integers else torch.randn(shape, generator=g) * scale
        self.kind, self.args, self.wide = kind, {}, []
        self.w = []
        for i, (inner, out) in enumerate(((K, H), (H, N))):
            if kind in ("e4m3", "e5m2"):
                q = values((E, out, inner), 2.0).to(E4M3 if kind == "e4m3" else E5M2)
                s = torch.exp2(torch.randint(-1, 2, (E, nb(out), nb(inner)), generator=g).float())
                if not integers:
                    s = s * 0.37 * max(inner, 1) ** -0.5
                spread = s.double().repeat_interleave(128, 1)[:, :out].repeat_interleave(128, 2)[:, :, :inner]
                self.w.append(pitched(q, (inner + 47) // 16 * 16 if i else None))
                self.args["w%d_scales" % (i + 1)] = s.to(DEV)
                self.wide.append((q.double() * spread).transpose(1, 2))
            else:
                w = values((E, inner, out), max(inner, 1) ** -0.5).to(dtype)
                self.w.append((w if kind == "kn" else w.transpose(1, 2).contiguous()).to(DEV))
                self.wide.append(w.double())
        self.args["b_layout"] = gr.B_KN if kind == "kn" else gr.B_NK

    def __call__(self, x, *args, **kwargs):
        return gr.gemm_relu_experts(x, self.w[0], self.w[1], *args, **self.args, **kwargs)


def reference_route(logits, top, renormalize):
    ids = torch.full((logits.shape[0], top), -1, dtype=torch.int32)
    weights = torch.zeros((logits.shape[0], top), dtype=torch.float64)
    for t, row in enumerate(logits.double().tolist()):
        if any(not v < math.inf for v in row):
            weights[t] = math.nan
            continue
        order = [e for e in sorted(range(len(row)), key=lambda e: (-row[e], e)) if row[e] > -math.inf][:top]
        if not order:
            continue
        total = sum(math.exp(row[e] - row[order[0]]) for e in (order if renormalize else range(len(row))))
        for j, e in enumerate(order):
            ids[t, j], weights[t, j] = e, math.exp(row[e] - row[order[0]]) / total
    return ids, weights


def reference(x, layer, ids, weights):
    """(y, its terms' magnitudes, magnitudes of the second weights) in 64 bits."""
    w1, w2 = layer.wide
    T, N = x.shape[0], w2.shape[2]
    y, m, s = (torch.zeros((T, N), dtype=torch.float64) for _ in range(3))
    for t in range(T):
        for e, p in zip(ids[t].tolist(), weights[t].double().tolist()):
            if 0 <= e < w1.shape[0]:
                y[t] += p * ((x[t].double() @ w1[e]).relu() @ w2[e])
                m[t] += abs(p) * ((x[t].double().abs() @ w1[e].abs()) @ w2[e].abs())
                s[t] += w2[e].abs().sum(0)
    return y, m, s


def check_close(got, x, layer, ids, weights):
    """One rounding to the output's type; two fp32 sums (a rounding of 2^-23 of the magnitudes an addition, the
    second product's twice, for its high and low parts) and 16 roundings of weights, scales and partial sums; the
    intermediate kept as two 16-bit values (2^-16 of it in bf16; 2^-22 and an absolute 2^-25 in fp16)."""
    y, m, s = reference(x, layer, ids, weights)
    K, H = layer.wide[0].shape[1:]
    fine = torch.finfo(got.dtype)
    kept = 2.0 ** -16 if got.dtype == torch.bfloat16 else 2.0 ** -22
    allowed = (y.abs() * fine.eps / 2 + m * ((K + 2 * H + 16) * 2.0 ** -23 + kept) * 1.01 + fine.smallest_normal * fine.eps
               + (s * 2.0 ** -25 if got.dtype == torch.float16 else 0))
    off = (got.cpu().double() - y).abs()
    worst = (off / allowed).max()
    assert (off <= allowed).all(), f"off by {float(worst):.3g} of what is allowed"


# tokens, K, hidden, N, experts, top
SHAPES = [(1, 1, 1, 1, 1, 1), (1, 128, 64, 64, 8, 2), (2, 4100, 33, 70, 5, 2), (7, 1101, 130, 515, 12, 3),
          (24, 256, 384, 256, 16, 4), (64, 200, 136, 100, 4, 4), (64, 64, 48, 40, 1024, 16), (33, 130, 2100, 37, 2, 1)]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("renormalize", [True, False])
def test_routed(shape, kind, dtype, renormalize):
    T, K, H, N, E, top = shape
    g = torch.Generator().manual_seed(T + K)
    x, logits = torch.randn((T, K), generator=g).to(dtype), torch.randn((T, E), generator=g)
    layer = Layer(kind, dtype, E, K, H, N, 7)
    y, ids, weights = layer(x.to(DEV), logits.to(DEV), top, renormalize=renormalize)
    want_ids, want_weights = reference_route(logits, top, renormalize)
    assert torch.equal(ids.cpu(), want_ids)
    # a few roundings of exp (2 units) and of a sum of at most 1024 terms of one sign, added by lanes and halves
    assert ((weights.cpu().double() - want_weights).abs() <= want_weights * 40 * 2.0 ** -24).all()
    check_close(y, x, layer, want_ids, weights.cpu())


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("kind", KINDS)
def test_exact_on_integers(shape, kind):
    # small integers, weights and scales that are powers of two: every sum is exact in fp32
    T, K, H, N, E, top = shape
    K, H = min(K, 300), min(H, 300)
    g = torch.Generator().manual_seed(T + N)
    x = torch.randint(-1, 2, (T, K), generator=g).to(torch.bfloat16)
    layer = Layer(kind, torch.bfloat16, E, K, H, N, 3, integers=True)
    ids = torch.randint(-1, E + 1, (T, top), generator=g).to(torch.int32)        # some name no expert, some one twice
    weights = torch.exp2(torch.randint(-1, 2, (T, top), generator=g).float())
    y, got_ids, got_weights = layer(x.to(DEV), ids=ids.to(DEV), weights=weights.to(DEV))
    assert torch.equal(got_ids.cpu(), ids) and torch.equal(got_weights.cpu(), weights)
    assert torch.equal(y.cpu(), reference(x, layer, ids, weights)[0].to(torch.bfloat16))


@pytest.mark.parametrize("kind", KINDS)
def test_one_expert_for_all(kind):
    # 2 x 64 choices of the same expert: two passes over its weights
    x = torch.randn((64, 96), generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    layer = Layer(kind, torch.bfloat16, 3, 96, 80, 72, 2)
    ids, weights = torch.ones((64, 2), dtype=torch.int32), torch.rand((64, 2), generator=torch.Generator().manual_seed(4))
    y, _, _ = layer(x.to(DEV), ids=ids.to(DEV), weights=weights.to(DEV))
    check_close(y, x, layer, ids, weights)


def test_ties_and_logits_without_a_rank():
    T, E = 8, 70
    logits = torch.zeros((T, E))
    logits[0, [3, 66]] = 1.0                                     # two ties, then the lowest of the others
    logits[1] = -math.inf
    logits[2] = -math.inf
    logits[2, [69, 5]] = -2.0                                    # fewer than top
    logits[3, 10] = math.nan
    logits[4, 64] = math.inf
    logits[5] = -0.0
    logits[5, 40] = 0.0                                          # equal to -0
    logits[6] = -3.0e38
    logits[6, 1] = 3.0e38
    logits[7] = torch.randn(E, generator=torch.Generator().manual_seed(1))
    x = torch.randn((T, 64), generator=torch.Generator().manual_seed(2)).to(torch.bfloat16)
    layer = Layer("nk", torch.bfloat16, E, 64, 64, 64, 5)
    for renormalize in (True, False):
        y, ids, weights = layer(x.to(DEV), logits.to(DEV), 3, renormalize=renormalize)
        want, want_weights = reference_route(logits, 3, renormalize)
        assert torch.equal(ids.cpu(), want)
        assert torch.equal(weights.cpu().isnan(), want_weights.isnan())
        fine = [t for t in range(T) if t not in (3, 4)]
        torch.testing.assert_close(weights.cpu()[fine].double(), want_weights[fine], rtol=40 * 2.0 ** -24, atol=0)
        assert y[3].isnan().all() and y[4].isnan().all() and (y[1] == 0).all()
        check_close(y[fine], x[fine], layer, want[fine], weights.cpu()[fine])
    # nobody has a choice
    y, ids, _ = layer(x.to(DEV), torch.full((T, E), -math.inf, device=DEV), 3)
    assert (y == 0).all() and (ids == -1).all()
    y, ids, _ = layer(x.to(DEV), torch.full((T, E), math.nan, device=DEV), 3)
    assert y.isnan().all() and (ids == -1).all()


@pytest.mark.parametrize("kind", KINDS)
def test_empty_sizes(kind):
    for T, K, H, N in ((0, 16, 16, 16), (3, 0, 16, 16), (3, 16, 0, 16), (3, 16, 16, 0)):
        layer = Layer(kind, torch.float16, 4, K, H, N, 1)
        x, logits = torch.ones((T, K), dtype=torch.float16, device=DEV), torch.zeros((T, 4), device=DEV)
        y, ids, weights = layer(x, logits, 2)
        assert y.shape == (T, N) and (y == 0).all()
        assert (ids.cpu() == torch.tensor([0, 1])).all() and (weights == 0.5).all()


def test_another_tokens_infinities_stay_away():
    # x of one token and the weights of one expert are not finite: only who uses them is
    layer = Layer("nk", torch.float16, 4, 136, 72, 100, 1)
    layer.w[0][2] = math.nan
    layer.w[1][2] = math.inf
    x = torch.randn((5, 136), generator=torch.Generator().manual_seed(2)).to(torch.float16)
    x[1] = math.inf
    ids = torch.tensor([[0, 1], [0, 1], [3, 2], [1, 3], [0, 3]], dtype=torch.int32)
    weights = torch.full((5, 2), 0.5)
    y, _, _ = layer(x.to(DEV), ids=ids.to(DEV), weights=weights.to(DEV))
    assert y[[0, 3, 4]].isfinite().all() and not y[2].isfinite().any()
    check_close(y[[0, 3, 4]], x[[0, 3, 4]], layer, ids[[0, 3, 4]], weights[[0, 3, 4]])


def test_unaligned_inputs():
    # rows of X and of the weights that start 2 bytes into a dword
    for kind in ("nk", "kn"):
        layer = Layer(kind, torch.bfloat16, 3, 64, 48, 40, 1)
        for i in range(2):
            flat = torch.zeros(layer.w[i].numel() + 1, dtype=torch.bfloat16, device=DEV)
            flat[1:] = layer.w[i].reshape(-1)
            layer.w[i] = flat[1:].reshape(layer.w[i].shape)
        x = torch.randn(4 * 64 + 1, generator=torch.Generator().manual_seed(2)).to(torch.bfloat16).to(DEV)[1:].reshape(4, 64)
        ids, weights = torch.tensor([[0, 1], [2, 1], [0, 2], [1, 2]], dtype=torch.int32), torch.full((4, 2), 0.5)
        y, _, _ = layer(x, ids=ids.to(DEV), weights=weights.to(DEV))
        check_close(y, x.cpu(), layer, ids, weights)

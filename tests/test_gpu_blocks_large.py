"""Weights of more than 96 MiB, which the kernels read past the caches and from other blocks on: exact on integers."""
import pytest
import torch

import tiled_dense_gemm_relu_amd as gr
from tiled_dense_gemm_relu_amd import blocks

pytestmark = pytest.mark.gpu
DEV = "cuda"
E4M3 = torch.float8_e4m3fn


def integers(shape, seed, least=-2, most=2):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randint(least, most + 1, shape, generator=g, device=DEV)


def eight_bit(values):
    """An 8-bit copy with rows at multiples of 16 bytes, NaN in the bytes between."""
    raw = torch.full(values.shape[:-1] + ((values.shape[-1] + 15) // 16 * 16,), 0x7f, dtype=torch.uint8, device=DEV)
    raw[..., : values.shape[-1]] = values.float().to(E4M3).view(torch.uint8)
    return raw[..., : values.shape[-1]].view(E4M3)


def scale_tiles(shape, seed):
    return torch.exp2(integers(shape, seed, -1, 1).float())


def spread(s, rows, cols):
    return s.repeat_interleave(128, -2)[..., :rows, :].repeat_interleave(128, -1)[..., :cols]


@pytest.mark.parametrize("M", [1, 16, 40, 64])
def test_dense(M):
    N, K = 12345, 8200                                   # 8208 bytes a row: 97 MiB
    a, b, sa, sb = integers((M, K), 1), integers((N, K), 2), scale_tiles((65, M), 3), scale_tiles((97, 65), 4)
    c = gr.gemm_relu_blocks(eight_bit(a), sa, eight_bit(b), sb, relu=False)
    wide_a = a.float() * sa.t().repeat_interleave(128, 1)[:, :K]
    # sums of at most 8200 terms up to 16, in steps of a quarter: exact in fp32
    assert torch.equal(c, (wide_a @ (b.float() * spread(sb, N, K)).t()).to(torch.bfloat16))


@pytest.mark.parametrize("config", [blocks.CONFIG_AUTO, blocks.CONFIG_STREAM, blocks.CONFIG_64, blocks.CONFIG_128, blocks.CONFIG_256])
@pytest.mark.parametrize("most", [20, 300])
@pytest.mark.parametrize("K", [2050, 600])               # 17 blocks of k, the last of 2; 5 blocks
def test_grouped(config, most, K):
    G, N = 26 if K == 2050 else 84, 2000
    sizes = torch.randint(0, most, (G,), generator=torch.Generator().manual_seed(most))
    sizes[3] = 0
    ends = sizes.cumsum(0)
    M, kb = int(ends[-1]) + 5, (K + 127) // 128          # and 5 rows behind the last
    a, b, sa, sb = integers((M, K), 5), integers((G, N, K), 6), scale_tiles((kb, M), 7), scale_tiles((G, 16, kb), 8)
    assert M >= G and G * N * ((K + 15) // 16 * 16) >= 96 << 20
    c = gr.gemm_relu_blocks(eight_bit(a), sa, eight_bit(b), sb, ends=ends.to(torch.int32).to(DEV), relu=False, config=config)
    wide_a = a.float() * sa.t().repeat_interleave(128, 1)[:, :K]
    want, begin = torch.zeros((M, N), device=DEV), 0
    for g, end in enumerate(ends.tolist()):
        want[begin:end] = wide_a[begin:end] @ (b[g].float() * spread(sb[g], N, K)).t()
        begin = end
    assert torch.equal(c, want.to(torch.bfloat16))


@pytest.mark.parametrize("kind", ["nk", "kn", "e4m3"])
@pytest.mark.parametrize("tokens", [20, 40])
def test_expert_layer(kind, tokens):
    E, K, H, N, top = 40 if kind != "e4m3" else 60, 1500, 1200, 1300, 4
    assert E * min(K, N) * H * (1 if kind == "e4m3" else 2) >= 64 << 20 and E * H * K * (1 if kind == "e4m3" else 2) >= 96 << 20
    x = integers((tokens, K), 11, -1, 1).to(torch.bfloat16)
    w1, w2 = integers((E, H, K), 12, -1, 1), integers((E, N, H), 13, -1, 1)
    ids = integers((tokens, top), 14, 0, E - 1).to(torch.int32)
    weights = torch.exp2(integers((tokens, top), 15, -1, 1).float())
    kw = {}
    if kind == "e4m3":
        s1, s2 = scale_tiles((E, 10, 12), 16), scale_tiles((E, 11, 10), 17)
        args, kw = (eight_bit(w1), eight_bit(w2)), {"w1_scales": s1, "w2_scales": s2}
        wide = w1.float() * spread(s1, H, K), w2.float() * spread(s2, N, H)
    else:
        wide = w1.float(), w2.float()
        args = (w1.bfloat16(), w2.bfloat16())
        if kind == "kn":
            args, kw = tuple(w.transpose(1, 2).contiguous() for w in args), {"b_layout": gr.B_KN}
    y = gr.gemm_relu_experts(x, *args, ids=ids, weights=weights, **kw)[0]
    # hidden values are near 2^6 in steps of 2^-2, kept as two 16-bit values without loss; outputs near 2^13 in steps
    # of 2^-4, far from the 2^20 where fp32 sums would lose one
    want = torch.zeros((tokens, N), dtype=torch.float64, device=DEV)
    for t in range(tokens):
        for j in range(top):
            e = int(ids[t, j])
            hidden = (wide[0][e].double() @ x[t].double()).clamp_min(0) * float(weights[t, j])
            want[t] += wide[1][e].double() @ hidden
    assert torch.equal(y, want.to(torch.bfloat16))


@pytest.mark.parametrize("config", [blocks.CONFIG_64, blocks.CONFIG_128, blocks.CONFIG_STREAM])
@pytest.mark.parametrize("M", [3, 64, 100])
def test_dense_by_every_kernel(config, M):
    N, K = 12345, 8200
    a, b, sa, sb = integers((M, K), 21), integers((N, K), 22), scale_tiles((65, M), 23), scale_tiles((97, 65), 24)
    c = gr.gemm_relu_blocks(eight_bit(a), sa, eight_bit(b), sb, config=config)
    wide_a = a.float() * sa.t().repeat_interleave(128, 1)[:, :K]
    assert torch.equal(c, (wide_a @ (b.float() * spread(sb, N, K)).t()).relu().to(torch.bfloat16))


# ---------------------------------------------------------------- the longest rows, and places past 2^32 bytes


@pytest.mark.parametrize("M,N", [(3, 5), (70, 65), (300, 20)])
def test_longest_sums(M, N):
    K = 1 << 20
    a, b = integers((M, K), 31, -1, 1), integers((N, K), 32, -1, 1)
    ones = torch.ones((K // 128, M), device=DEV), torch.ones((1, K // 128), device=DEV)
    c = gr.gemm_relu_blocks(eight_bit(a), ones[0], eight_bit(b), ones[1], relu=False, out_dtype=torch.float16)
    assert torch.equal(c, (a.float() @ b.float().t()).half())


def test_longest_rows_of_an_expert_layer():
    for K, H, N in ((1 << 20, 3, 70), (70, 1 << 20, 3), (3, 70, 1 << 20)):
        x, w1, w2 = (integers(s, 33 + i, -1, 1).to(torch.bfloat16) for i, s in enumerate(((2, K), (2, H, K), (2, N, H))))
        ids, weights = torch.tensor([[1], [0]], dtype=torch.int32, device=DEV), torch.ones((2, 1), device=DEV)
        y = gr.gemm_relu_experts(x, w1, w2, ids=ids, weights=weights)[0]
        for t, e in ((0, 1), (1, 0)):
            hidden = (w1[e].double() @ x[t].double()).clamp_min(0)
            assert torch.equal(y[t], (w2[e].double() @ hidden).to(torch.bfloat16)), (K, H, N)


def test_quantizer_past_32_bits():
    R, C = 140000, 16384                                  # 4.6 GB
    x = torch.randint(-30000, 30000, (R, C), dtype=torch.int16, generator=torch.Generator(device=DEV).manual_seed(41), device=DEV)
    x = x.view(torch.bfloat16)                           # every finite magnitude (and no NaN: below 0x7f80)
    q, s, qt, st = gr.quantize_blocks(x, transposed=True)
    for r, c in ((0, 0), (139904, 16256), (139904, 0), (70016, 8192), (131072, 16256)):
        part = x[r:r + 128, c:c + 128].contiguous()
        pq, ps, pqt, pst = gr.quantize_blocks(part, transposed=True)
        rows = part.shape[0]
        assert torch.equal(q[r:r + 128, c:c + 128].view(torch.uint8), pq.view(torch.uint8)) and torch.equal(s[c // 128, r:r + 128], ps[0])
        assert torch.equal(qt[c:c + 128, r:r + 128].view(torch.uint8), pqt.view(torch.uint8)) and torch.equal(st[r // 128, c:c + 128], pst[0])
        assert rows == min(128, R - r)


@pytest.mark.parametrize("rows", [5, 100, 300])
def test_weights_past_32_bits(rows):
    G, N, K = 20, 16384, 16384                            # 5.4 GB
    a = integers((3 * rows, K), 51)
    b = torch.empty((G, N, K), dtype=torch.uint8, device=DEV)
    for g in (0, 16, 19):
        b[g] = eight_bit(integers((N, K), 52 + g)).view(torch.uint8)
    ends = torch.tensor([rows] * 16 + [2 * rows] * 3 + [3 * rows], dtype=torch.int32, device=DEV)
    ones = torch.ones((128, 3 * rows), device=DEV), torch.ones((G, 128, 128), device=DEV)
    c = gr.gemm_relu_blocks(eight_bit(a), ones[0], b.view(E4M3), ones[1], ends=ends, relu=False)
    for i, g in enumerate((0, 16, 19)):
        part = slice(i * rows, (i + 1) * rows)
        assert torch.equal(c[part], (a[part].float() @ b[g].view(E4M3).float().t()).to(torch.bfloat16)), g


def test_results_past_32_bits():
    M, N, K = 70000, 32800, 40                            # 4.6 GB of results
    a, b = integers((M, K), 61), integers((N, K), 62)
    for config in (blocks.CONFIG_AUTO, blocks.CONFIG_64):
        c = gr.gemm_relu_blocks(eight_bit(a), torch.ones((1, M), device=DEV), eight_bit(b), torch.ones((257, 1), device=DEV),
                                relu=False, config=config)
        for m in (0, 65400, M - 200):
            assert torch.equal(c[m:m + 200], (a[m:m + 200].float() @ b.float().t()).to(torch.bfloat16)), (config, m)
        del c


@pytest.mark.parametrize("kind", ["nk", "kn"])
def test_expert_layer_past_32_bits(kind):
    E, K, H = 18, 16384, 8192                             # 4.8 GB a stack
    x, logits = integers((3, K), 71, -1, 1).to(torch.bfloat16), torch.zeros((3, E), device=DEV)
    logits[0, 17] = logits[1, 16] = logits[2, 0] = 50.0
    w1, w2 = (torch.randint(-1, 2, s, dtype=torch.int8, generator=torch.Generator(device=DEV).manual_seed(72), device=DEV).to(torch.bfloat16)
              for s in (((E, H, K), (E, K, H)) if kind == "nk" else ((E, K, H), (E, H, K))))
    y = gr.gemm_relu_experts(x, w1, w2, logits, 1, b_layout=gr.B_NK if kind == "nk" else gr.B_KN)[0]
    for t, e in ((0, 17), (1, 16), (2, 0)):
        first, second = (w[e].double() if kind == "nk" else w[e].double().t() for w in (w1, w2))
        want = (second @ (first @ x[t].double()).clamp_min(0))
        assert torch.equal(y[t], want.to(torch.bfloat16)), t

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

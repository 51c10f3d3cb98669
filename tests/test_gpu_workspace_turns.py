"""Threads on one stream share its workspace: every entry point that keeps something there between its launches, at once."""
import threading

import pytest
import torch

import tiled_dense_gemm_relu_amd as gr

from test_gpu_blocks import gen
from test_gpu_experts import Layer

pytestmark = pytest.mark.gpu
DEV = "cuda"


def randn(shape, seed, dtype=torch.bfloat16):
    return torch.randn(shape, generator=gen(seed)).to(dtype).to(DEV)


def jobs(seed):
    M, N, K = 96, 160, 272
    out = []
    ends = torch.tensor([30, 30, M - 5], dtype=torch.int32, device=DEV)
    dc, c = randn((M, N), seed), randn((M, N), seed + 1)
    # gradients of grouped products: the masked gradient, or copies of odd rows, on their way
    for k in (1024, 1001):
        m, n = 1100, 1024 if k == 1024 else 1001
        gd, gc, a, b = randn((m, n), seed + 2), randn((m, n), seed + 3), randn((m, k), seed + 4), randn((3, k, n), seed + 5)
        rows = torch.tensor([300, 700, m - 5], dtype=torch.int32, device=DEV)
        out.append(lambda gd=gd, gc=gc, a=a, b=b, rows=rows: gr.gemm_relu_grouped_backward(gd, gc, a, b, rows))
    # a grouped product on copies of its odd rows
    a, b = randn((1500, 1501), seed + 6), randn((2, 1501, 1501), seed + 7)
    rows = torch.tensor([700, 1500], dtype=torch.int32, device=DEV)
    out.append(lambda a=a, b=b, rows=rows: (gr.gemm_relu_grouped(a, b, rows),))
    # adapters: the intermediates
    x, w, u, v = randn((M, K), seed + 8), randn((K, N), seed + 9), randn((3, K, 16), seed + 10), randn((3, 16, N), seed + 11)
    scales, ids = torch.ones(3, device=DEV), torch.tensor([0, 1, 2], dtype=torch.int32, device=DEV)
    out.append(lambda x=x, w=w, u=u, v=v: (gr.gemm_relu_adapters(x, w, u, v, scales, ends, ids),))
    # 8-bit gradients: the quantized gradient; an expert layer: the hidden values and the partial sums
    xt, sx = gr.quantize_blocks(randn((M, K), seed + 12), rows=False, transposed=True)
    wt, sw = gr.quantize_blocks(randn((N, K), seed + 13), tiles=True, rows=False, transposed=True)
    out.append(lambda dc=dc, c=c, xt=xt, sx=sx, wt=wt, sw=sw: gr.gemm_relu_blocks_backward(dc, c, xt, sx, wt, sw))
    layer = Layer("nk", torch.bfloat16, 6, 100, 300, 90, seed + 14)
    t, logits = randn((20, 100), seed + 15), torch.randn((20, 6), generator=gen(seed + 16)).to(DEV)
    out.append(lambda layer=layer, t=t, logits=logits: layer(t, logits, 2))
    # a split product with the same kind of space
    p, q = randn((64, 4096), seed + 17), randn((4096, 256), seed + 18)
    out.append(lambda p=p, q=q: (gr.gemm_relu_splitk(p, q, splits=8),))
    return out


def same(a, b):
    return all(torch.equal(u, v) for u, v in zip(a, b))


def test_threads_of_all_kinds_on_one_stream():
    work = jobs(100) + jobs(200)
    want, wrong = [job() for job in work], []
    torch.cuda.synchronize()

    def run(i):
        for _ in range(40):
            if not same(work[i](), want[i]):
                wrong.append(i)
    threads = [threading.Thread(target=run, args=(i,)) for i in range(len(work))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong, sorted(set(wrong))

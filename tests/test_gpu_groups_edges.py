"""Products whose rows choose their weights, at the edges of the rules that choose their kernels.

References, bars and helpers are test_gpu_groups.py's.
"""
import pytest
import torch

import tiled_dense_gemm_relu_amd as gr
from test_gpu_groups import (CONFIGS, adapter_inputs, adapter_reference, assert_close, backward_reference, calls,
                             ends_of, guarded, normal, say, weights)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("relu", [True, False])
@pytest.mark.parametrize("sizes,N,K", [([64], 12001, 1304), ([63], 13089, 1388), ([50, 0, 90, 12, 70], 15209, 298)])
def test_backward_of_few_odd_rows_and_a_long_sum(sizes, N, K, relu):
    # 17 to 64 rows a group of an odd length: copies for dB, while dA's weights are streamed.
    M, dt = sum(sizes), torch.bfloat16
    say(f"[odd rows] M={M} N={N} K={K} relu={relu}")
    a, b = normal((M, K), dt, 201), weights(len(sizes), N, K, dt, gr.B_NK, 202)
    dc, c = normal((M, N), dt, 203), normal((M, N), dt, 204).clamp_min(0)
    ra, ea, rb, eb = backward_reference(dc, c, a, b, sizes, gr.B_NK, relu)
    da, whole_a = guarded((M, K), dt)
    db, whole_b = guarded(tuple(b.shape), dt)
    args, ends = (dc.cuda(), c.cuda() if relu else None, a.cuda(), b.cuda()), ends_of(sizes).cuda()
    gr.gemm_relu_grouped_backward(*args, ends, b_layout=gr.B_NK, relu=relu, da=da, db=db)
    torch.cuda.synchronize()
    assert whole_a() and whole_b()
    assert_close(da, ra, ea, "dA")
    assert_close(db, rb, eb, "dB")
    only_a, _ = gr.gemm_relu_grouped_backward(*args, ends, b_layout=gr.B_NK, relu=relu, need_db=False)
    _, only_b = gr.gemm_relu_grouped_backward(*args, ends, b_layout=gr.B_NK, relu=relu, need_da=False)
    assert torch.equal(only_a, da) and torch.equal(only_b, db)


@pytest.mark.parametrize("layout", [gr.B_KN, gr.B_NK])
@pytest.mark.parametrize("N", [4, 68, 264, 1872])
@pytest.mark.parametrize("config", CONFIGS)
def test_many_adapters_in_a_block_whose_tile_passes_the_last_column(config, N, layout):
    # A decoding step: 16 rows, more than two adapters, the last of the table among them.
    sizes, count, dt = [1] * 16, 9, torch.bfloat16
    say(f"[adapters] N={N} layout={layout} config={config}")
    x, w, u, v, scales, ends, _ = adapter_inputs(sizes, 0, N, 192, 16, count, dt, layout, 211)
    ids = torch.arange(16, dtype=torch.int32) % count
    ref, err = adapter_reference(x, w, u, v, scales, sizes, ids, layout, False)
    out, whole = guarded((16, N), dt)
    gr.gemm_relu_adapters(*(t.cuda() for t in (x, w, u, v, scales, ends, ids)), out=out, b_layout=layout, relu=False,
                          config=config)
    torch.cuda.synchronize()
    assert whole()
    assert_close(out, ref, err, "C")


@pytest.mark.parametrize("which", range(6))
def test_graph_with_a_forked_side_stream(which):
    # The captured call runs on a stream forked from the capture's: its workspace is cleared there too.
    call, ins, outs = calls()[which]
    call()
    side, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        side.wait_stream(torch.cuda.current_stream())
        call(stream=side)
        torch.zeros(1 << 20, device="cuda").add_(7.0)          # memory that the other stream takes meanwhile
        torch.cuda.current_stream().wait_stream(side)
    for k in range(4):
        for t in ins:
            t.copy_(normal(tuple(t.shape), t.dtype, 220 + k))
        for t in outs:
            t.fill_(777.0)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        first = [t.clone() for t in outs]
        for t in outs:
            t.fill_(777.0)
        call()                                                 # eager, on the same inputs
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(first, outs)), (which, k)


@pytest.mark.parametrize("relu", [True, False])
@pytest.mark.parametrize("layout", [gr.B_KN, gr.B_NK])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("config", [-1, *CONFIGS])
@pytest.mark.parametrize("sizes,N", [([1] * 37 + [100, 0, 300], 264), ([1500, 1300], 512)])
def test_infinities_of_an_adapter_keep_their_sign(sizes, N, config, dtype, layout, relu):
    # A V with infinities and NaN, in rows that use it: what the products' signs make of them, whatever
    # the intermediate's parts are.
    say(f"[adapters] {sizes[-3:]} N={N} {dtype} layout={layout} config={config} relu={relu}")
    x, w, u, v, scales, ends, ids = adapter_inputs(sizes, 0, N, 136, 16, 3, dtype, layout, 231)
    ids = torch.arange(len(sizes), dtype=torch.int32) % 3
    inf, kn = float("inf"), v if layout == gr.B_KN else v.transpose(1, 2)
    clean = [n for n in range(N) if n not in (5, 40, 41, 77)]
    ref, err = adapter_reference(x, w, u, v, scales, sizes, ids, layout, relu)
    kn[0, 3, 5], kn[0, 7, 40], kn[1, 0, 41], kn[1, 9, 41], kn[2, 15, 77] = inf, -inf, inf, -inf, float("nan")
    want = adapter_reference(x, w, u, v, scales, sizes, ids, layout, False)[0][:, [5, 40, 41, 77]]
    if relu:
        want = torch.where(want > 0, want, torch.zeros_like(want))
    got = gr.gemm_relu_adapters(*(t.cuda() for t in (x, w, u, v, scales, ends, ids)), b_layout=layout, relu=relu,
                                config=config)
    assert_close(got[:, clean], ref[:, clean], err[:, clean], "C")
    got = got[:, [5, 40, 41, 77]].cpu().double()
    odd = ~torch.isfinite(want)
    assert odd.sum() > 0.1 * odd.numel() and torch.equal(torch.isnan(got), torch.isnan(want))
    assert torch.equal(torch.isfinite(got), ~odd) and torch.equal(got[want.abs() == inf], want[want.abs() == inf])


def test_released_workspaces_give_their_memory_back():
    call, _, outs = calls()[4]
    call()
    want = [t.clone() for t in outs]
    a, b = torch.ones((1500, 2051), device="cuda").half(), torch.ones((2, 2051, 2051), device="cuda").half()
    gr.gemm_relu_grouped(a, b, torch.tensor([700, 1500]).int().cuda())         # odd rows: copies of a and b
    torch.cuda.synchronize()
    held = torch.cuda.memory_allocated()
    gr.release_workspaces()
    assert held - torch.cuda.memory_allocated() >= 2 * (a.numel() + b.numel())
    for t in outs:
        t.fill_(777.0)
    call()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(want, outs))

"""The 8-bit products and the expert layer for a few tokens as programs use them: through autograd, in graphs, on
side streams, two at once, and together as a served layer."""
import pytest
import torch

import tiled_dense_gemm_relu_amd as gr
from tiled_dense_gemm_relu_amd import blocks

from test_gpu_blocks import E4M3, E5M2, check_close, gen, pitched, reference_quantize, stands_for
from test_gpu_experts import Layer
from test_gpu_experts import check_close as check_layer

pytestmark = pytest.mark.gpu
DEV = "cuda"


def randn(shape, seed, dtype=torch.bfloat16, scale=1.0):
    return (torch.randn(shape, generator=gen(seed)) * scale).to(dtype)


# ---------------------------------------------------------------- autograd


@pytest.mark.parametrize("relu", [True, False])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_linear_and_gradients_match_the_formulas(relu, dtype):
    M, N, K = 200, 150, 300
    x, w, dc = randn((M, K), 1, dtype), randn((N, K), 2, dtype, K ** -0.5), randn((M, N), 3, dtype)
    xg, wg = x.to(DEV).requires_grad_(), w.to(DEV).requires_grad_()
    c = gr.linear_blocks(xg, wg, relu=relu)
    c.backward(dc.to(DEV))
    qx, qw = (stands_for(*reference_quantize(t, E4M3, tiles, False), tiles) for t, tiles in ((x, False), (w, True)))
    check_close(c.detach(), qx, qw, relu)
    # gradients of what was kept: x along its columns, w's tiles, the masked gradient both ways
    d = torch.where(c.detach().cpu() > 0, dc, torch.zeros_like(dc)) if relu else dc
    d_rows, d_columns = (stands_for(*reference_quantize(t, E5M2, False, False), False) for t in (d, d.t()))
    x_columns = stands_for(*reference_quantize(x.t(), E4M3, False, False), False)
    check_close(xg.grad, d_rows, qw.t().contiguous())
    check_close(wg.grad, d_columns, x_columns)
    # one gradient alone is the same
    for which in (0, 1):
        xs, ws = x.to(DEV).requires_grad_(which == 0), w.to(DEV).requires_grad_(which == 1)
        gr.linear_blocks(xs, ws, relu=relu).backward(dc.to(DEV))
        assert torch.equal((xs, ws)[which].grad, (xg, wg)[which].grad) and (xs, ws)[1 - which].grad is None
    with torch.no_grad():
        assert torch.equal(gr.linear_blocks(xg, wg, relu=relu), c)


def test_captured_backward_pass():
    # Forward and backward in one graph; no eager graph of the leaves is alive.
    M, N, K = 130, 144, 200
    x, w, dc = (torch.zeros(s, dtype=torch.bfloat16, device=DEV) for s in ((M, K), (N, K), (M, N)))
    x.requires_grad_()
    w.requires_grad_()
    gr.linear_blocks(x.detach(), w.detach())
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dx, dw = torch.autograd.grad(gr.linear_blocks(x, w), (x, w), dc)
    for seed in range(1, 6):
        with torch.no_grad():
            for i, t in enumerate((x, w, dc)):
                t.copy_(randn(t.shape, 20 * seed + i))
            torch.cuda.synchronize()
            graph.replay()
            q, s, xt, sxt = gr.quantize_blocks(x, transposed=True)
            qw, sw, wt, swt = gr.quantize_blocks(w, tiles=True, transposed=True)
            c = gr.gemm_relu_blocks(q, s, qw, sw)
            want = gr.gemm_relu_blocks_backward(dc, c, xt, sxt, wt, swt)
            torch.cuda.synchronize()
            assert torch.equal(dx, want[0]) and torch.equal(dw, want[1]) and want[0].any() and want[1].any()


@pytest.mark.parametrize("shape", [(0, 5, 7), (5, 0, 7), (5, 7, 0), (1, 1, 1)])
def test_linear_of_nothing(shape):
    M, N, K = shape
    x, w = (torch.ones(s, dtype=torch.float16, device=DEV, requires_grad=True) for s in ((M, K), (N, K)))
    c = gr.linear_blocks(x, w)
    assert c.shape == (M, N) and (c == K).all()
    c.backward(torch.ones_like(c))
    assert (x.grad == N).all() and (w.grad == M).all() and x.grad.shape == x.shape and w.grad.shape == w.shape


def test_linear_on_a_side_stream():
    M, N, K = 520, 300, 700
    x, w, dc = randn((M, K), 1).to(DEV), randn((N, K), 2).to(DEV), randn((M, N), 3).to(DEV)
    results = []
    for stream in (None, torch.cuda.Stream()):
        xg, wg = x.clone().requires_grad_(), w.clone().requires_grad_()
        if stream is not None:
            stream.wait_stream(torch.cuda.current_stream())
        c = gr.linear_blocks(xg, wg, stream=stream)
        if stream is not None:
            torch.cuda.current_stream().wait_stream(stream)
        results.append((c.detach(),) + torch.autograd.grad(c, (xg, wg), dc))
        torch.cuda.synchronize()
    assert same(*results)


def test_gradients_match_differences():
    """Values that 8 bits hold exactly (integers up to 15 in blocks whose largest is 448, gradients of 1 and 2):
    there the layer is the product itself, so a step of 1 changes sum(dc c) by exactly the gradient's entry."""
    M, N, K = 5, 130, 140
    g = gen(7)
    x, w = (torch.randint(-7, 8, (r, K), generator=g).to(torch.float16) for r in (M, N))
    # each row's, column's and tile's largest magnitude: rows and columns of their own, so steps leave the scales alone
    x[:, 0] = x[:, 128] = 448
    x[4] = 448
    w[::128, ::128] = 448
    dc = torch.randint(1, 3, (M, N), generator=g).to(torch.float16)
    dc[:, 0] = dc[:, 128] = 2
    dc[4] = 2

    def total(x, w):
        # 64-bit sums of exact outputs (integers below 2^24 in fp32; c itself is rounded to fp16, so sum it by parts)
        q, s = gr.quantize_blocks(x.to(DEV))
        qw, sw = gr.quantize_blocks(w.to(DEV), tiles=True)
        return float((dc.double() * (stands_for(q, s, False) @ stands_for(qw, sw, True).t())).sum())
    xg, wg = x.to(DEV).requires_grad_(), w.to(DEV).requires_grad_()
    gr.linear_blocks(xg, wg, relu=False).backward(dc.to(DEV))
    base = total(x, w)
    for (m, k) in ((0, 1), (1, 60), (3, 139), (2, 129)):
        step = x.clone()
        step[m, k] += 1
        assert total(step, w) - base == float((dc[m].double() @ w[:, k].double()))
        assert float(xg.grad[m, k]) == float(torch.tensor(total(step, w) - base).half())
    for (n, k) in ((1, 1), (60, 61), (129, 139), (2, 129)):
        step = w.clone()
        step[n, k] += 1
        assert float(wg.grad[n, k]) == float(torch.tensor(total(x, step) - base).half())


def test_refusals_of_gradients():
    x, w = randn((4, 32), 1).to(DEV), randn((2, 16, 32), 2).to(DEV)
    w2, logits = randn((2, 32, 16), 3).to(DEV), torch.zeros((4, 2), device=DEV)
    y, ids, weights = gr.gemm_relu_experts(x.requires_grad_(), w, w2, logits, 1)
    assert y.requires_grad and not weights.requires_grad
    with pytest.raises(NotImplementedError, match="no gradient"):
        y.sum().backward()
    with pytest.raises(RuntimeError, match="out="):
        gr.gemm_relu_experts(x, w, w2, logits, 1, out=torch.empty_like(x))
    with torch.no_grad():
        again = gr.gemm_relu_experts(x, w, w2, logits, 1, out=torch.empty((4, 32), dtype=x.dtype, device=DEV))[0]
    assert torch.equal(again, y)
    q, s = gr.quantize_blocks(x.detach())
    with pytest.raises(RuntimeError, match="requires a gradient"):
        gr.gemm_relu_blocks(q.requires_grad_(), s, q.detach(), torch.ones((1, 1), device=DEV))


@pytest.mark.parametrize("what", ["strided", "short storage", "wrong scales", "odd pitch", "other device", "formats", "layout",
                                  "both routes", "no route", "out dtype"])
def test_python_refusals(what):
    q, s = gr.quantize_blocks(randn((8, 40), 1).to(DEV))
    w, sw = gr.quantize_blocks(randn((6, 40), 2).to(DEV), tiles=True)
    x, w1, w2 = randn((4, 32), 1).to(DEV), randn((2, 16, 32), 2).to(DEV), randn((2, 32, 16), 3).to(DEV)
    logits = torch.zeros((4, 2), device=DEV)
    stack = pitched(torch.zeros((2, 16, 32), dtype=E4M3))
    ones = torch.ones((2, 1, 1), device=DEV)
    calls = {
        "strided": lambda: gr.gemm_relu_blocks(pitched(torch.zeros((40, 8), dtype=E4M3)).t(), s, w, sw),
        "short storage": lambda: gr.gemm_relu_blocks(torch.zeros(7 * 48 + 40, dtype=torch.uint8, device=DEV).view(E4M3).as_strided((8, 40), (48, 1)), s, w, sw),
        "wrong scales": lambda: gr.gemm_relu_blocks(q, s.t().contiguous(), w, sw),
        "odd pitch": lambda: gr.gemm_relu_blocks(torch.zeros((8, 40), dtype=torch.uint8, device=DEV).view(E4M3), s, w, sw),
        "other device": lambda: gr.gemm_relu_blocks(q, s, w.cpu(), sw),
        "formats": lambda: gr.gemm_relu_experts(x, stack, stack.view(torch.uint8).view(E5M2), logits, 1, w1_scales=ones, w2_scales=ones),
        "layout": lambda: gr.gemm_relu_experts(x, stack, stack, logits, 1, w1_scales=ones, w2_scales=ones, b_layout=gr.B_KN),
        "both routes": lambda: gr.gemm_relu_experts(x, w1, w2, logits, 1, ids=torch.zeros((4, 1), dtype=torch.int32, device=DEV)),
        "no route": lambda: gr.gemm_relu_experts(x, w1, w2),
        "out dtype": lambda: gr.gemm_relu_blocks(q, s, w, sw, out_dtype=torch.float32),
    }
    with pytest.raises((ValueError, TypeError)):
        calls[what]()


# ---------------------------------------------------------------- streams and graphs


class Work:
    """Calls of every operator on buffers whose contents can be replaced, and their eager results."""

    def __init__(self):
        M, N, K = 96, 160, 272
        self.x, self.w = torch.empty((M, K), dtype=torch.bfloat16, device=DEV), torch.empty((N, K), dtype=torch.bfloat16, device=DEV)
        self.dc, self.c = (torch.empty((M, N), dtype=torch.bfloat16, device=DEV) for _ in range(2))
        self.logits = torch.empty((40, 6), device=DEV)
        self.w1, self.w2 = (torch.empty(s, dtype=torch.bfloat16, device=DEV) for s in ((6, 130, K), (6, K, 130)))
        self.ends = torch.tensor([40, 40, M - 3], dtype=torch.int32, device=DEV)

    def fill(self, seed):
        for i, t in enumerate((self.x, self.w, self.dc, self.c, self.logits, self.w1, self.w2)):
            t.copy_(torch.randn(t.shape, generator=gen(10 * seed + i)) * (t.shape[-1] ** -0.5 if t.dim() == 3 else 1.0))

    def __call__(self, **kw):
        q, s, xt, sxt = gr.quantize_blocks(self.x, transposed=True, **kw)
        qw, sw, wt, swt = gr.quantize_blocks(self.w, tiles=True, transposed=True, **kw)
        out = [q.view(torch.uint8), s, xt.view(torch.uint8), sxt]
        for config in (blocks.CONFIG_AUTO, blocks.CONFIG_256, blocks.CONFIG_128, blocks.CONFIG_64):
            out.append(gr.gemm_relu_blocks(q, s, qw, sw, config=config, **kw))
        q1, s1 = gr.quantize_blocks(self.w1, tiles=True, **kw)
        out.append(gr.gemm_relu_blocks(q, s, q1[:3], s1[:3].contiguous(), ends=self.ends, relu=False, **kw))
        out += gr.gemm_relu_blocks_backward(self.dc, self.c, xt, sxt, wt, swt, **kw)
        for tokens in (1, 8, 40):
            out += gr.gemm_relu_experts(self.x[:tokens], self.w1, self.w2, self.logits[:tokens], 2, **kw)
        q2, s2 = gr.quantize_blocks(self.w2, tiles=True, **kw)
        out += gr.gemm_relu_experts(self.x[:8], q1, q2, self.logits[:8], 3, w1_scales=s1, w2_scales=s2, **kw)
        return out


def same(a, b):
    return all(torch.equal(u, v) for u, v in zip(a, b))


def test_graph_replays_match_eager_calls():
    work = Work()
    work.fill(0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        work()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = work()
    for seed in range(1, 6):
        work.fill(seed)
        torch.cuda.synchronize()
        graph.replay()
        eager = work()
        torch.cuda.synchronize()
        assert same(captured, eager), f"replay {seed}"
        assert same(work(), eager)                      # and run to run


def test_two_graphs_and_eager_calls_share_nothing():
    # captured on one stream, replayed on another, with eager calls between and a larger workspace taken
    work, other = Work(), Work()
    work.fill(1)
    other.fill(2)
    graphs = []
    for w in (work, other):
        w()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = w()
        graphs.append((g, out, w))
    gr.release_workspaces()
    big = Layer("nk", torch.bfloat16, 2, 64, 4096, 4096, 1)
    big(torch.ones((64, 64), dtype=torch.bfloat16, device=DEV), torch.zeros((64, 2), device=DEV), 2)
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(3):
        torch.cuda.synchronize()
        for (g, _, _), s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for g, out, w in graphs:
            assert same(out, w())


def test_side_stream_and_two_streams_at_once():
    work, other = Work(), Work()
    work.fill(3)
    other.fill(4)
    want, want_other = work(), other()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(4):
        got = [w(stream=s) for w, s in zip((work, other), streams)]
        torch.cuda.synchronize()
        assert same(got[0], want) and same(got[1], want_other)
    for _ in range(4):                                   # and as the current streams
        got = []
        for w, s in zip((work, other), streams):
            with torch.cuda.stream(s):
                got.append(w())
        torch.cuda.synchronize()
        assert same(got[0], want) and same(got[1], want_other)


def test_two_threads_on_one_stream():
    # They share the stream's workspace: the launches of a call stay together.
    import threading
    layer = Layer("nk", torch.bfloat16, 6, 100, 300, 90, 5)
    M, N, K = 96, 160, 272
    jobs = []
    for seed in (1, 2):
        x, logits = randn((20, 100), seed).to(DEV), torch.randn((20, 6), generator=gen(10 + seed)).to(DEV)
        xt, sx = gr.quantize_blocks(randn((M, K), 20 + seed).to(DEV), rows=False, transposed=True)
        wt, sw = gr.quantize_blocks(randn((N, K), 30 + seed).to(DEV), tiles=True, rows=False, transposed=True)
        dc, c = randn((M, N), 40 + seed).to(DEV), randn((M, N), 50 + seed).to(DEV)
        jobs.append(lambda x=x, logits=logits: layer(x, logits, 2))
        jobs.append(lambda dc=dc, c=c, xt=xt, sx=sx, wt=wt, sw=sw: gr.gemm_relu_blocks_backward(dc, c, xt, sx, wt, sw))
    want, wrong = [job() for job in jobs], []

    def run(i):
        for _ in range(100):
            if not same(jobs[i](), want[i]):
                wrong.append(i)
    threads = [threading.Thread(target=run, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong


def test_own_workspace_is_left_clean():
    layer = Layer("nk", torch.bfloat16, 5, 136, 200, 520, 3)
    x, logits = randn((9, 136), 1).to(DEV), torch.randn((9, 5), generator=gen(2)).to(DEV)
    need = gr.experts_workspace_bytes(9, 520, 200, 5, 2)
    space = torch.full((need,), 0xFF, dtype=torch.uint8, device=DEV)
    space[:65536] = 0
    want = layer(x, logits, 2)
    for _ in range(3):
        assert same(layer(x, logits, 2, workspace=space), want)
        assert not space[:65536].any()
    with pytest.raises(gr.GemmReluError, match="WORKSPACE"):
        layer(x, logits, 2, workspace=space[:-256])


# ---------------------------------------------------------------- together


def test_masked_places_may_hold_anything():
    # A ReLU's gradient: infinities and NaN where the output is not above zero change nothing.
    M, N, K = 140, 150, 130
    xt, sx = gr.quantize_blocks(randn((M, K), 1).to(DEV), rows=False, transposed=True)
    wt, sw = gr.quantize_blocks(randn((N, K), 2).to(DEV), tiles=True, rows=False, transposed=True)
    dc, c = randn((M, N), 3), randn((M, N), 4)
    c[7] = -1.0                                          # a row and a column without any
    c[:, 9] = 0.0
    c[3, 5], c[4, 6] = float("nan"), -float("inf")       # not above zero either
    bad = dc.clone()
    holes = ~(c > 0)
    bad[holes] = torch.tensor([float("inf"), -float("inf"), float("nan"), torch.finfo(torch.bfloat16).min])[
        torch.arange(int(holes.sum())) % 4].to(torch.bfloat16)
    clean = torch.where(holes, torch.zeros_like(dc), dc)
    for f in (lambda d: gr.gemm_relu_blocks_backward(d.to(DEV), c.to(DEV), xt, sx, wt, sw),
              lambda d: gr.quantize_blocks(d.to(DEV), E5M2, mask=c.to(DEV), transposed=True)):
        got, want = f(bad), f(clean)
        assert all(same_tensors(u, v) for u, v in zip(got, want))
    dx, dw = gr.gemm_relu_blocks_backward(bad.to(DEV), c.to(DEV), xt, sx, wt, sw)
    assert not dx[7].any() and not dw[9].any() and dx.isfinite().all() and dw.isfinite().all()


def test_calls_as_the_documentation_has_them():
    M, N, K, top = 33, 70, 150, 2
    x, w, dc = randn((M, K), 1).to(DEV), randn((N, K), 2).to(DEV), randn((M, N), 3).to(DEV)
    q, s, qt, st = gr.quantize_blocks(x, transposed=True)
    qw, sw, wt, sw_t = gr.quantize_blocks(w, tiles=True, transposed=True)
    c = gr.gemm_relu_blocks(q, s, qw, sw)
    dx, dw = gr.gemm_relu_blocks_backward(dc, c, qt, st, wt, sw_t)
    x.requires_grad_()
    w.requires_grad_()
    layer = gr.linear_blocks(x, w)
    assert torch.equal(layer, c)
    layer.backward(dc)
    assert torch.equal(x.grad, dx) and torch.equal(w.grad, dw)
    w1, w2, logits = randn((4, 20, K), 4).to(DEV), randn((4, K, 20), 5).to(DEV), randn((M, 4), 6).float().to(DEV)
    with torch.no_grad():
        y, ids, weights = gr.gemm_relu_experts(x, w1, w2, logits, top)
    assert y.shape == x.shape and ids.shape == weights.shape == (M, top)


def test_served_layer():
    from tiled_dense_gemm_relu_amd.expert_layer import ServedExperts, serve_experts
    decoded, prompt, layer, (x, logits) = serve_experts(tokens=24, prompt=300, experts=8, width=136, hidden=200, top=2)
    served = ServedExperts(layer, 2)
    w1, w2 = (torch.stack([stands_for(q, s, True) for q, s in zip(w, sc)]) for w, sc in ((served.w1, served.s1), (served.w2, served.s2)))
    for e in range(8):
        # (out, in), as the training weights (in, out) transposed, half a step of e4m3 of a tile's largest away
        trained = layer.weights[0][e].t().cpu().double()
        assert ((w1[e] - trained).abs() <= trained.abs() * 2.0 ** -4 + trained.abs().max() * 2.0 ** -9 / 448).all()

    class Wide:
        wide = [w1.transpose(1, 2).contiguous(), w2.transpose(1, 2).contiguous()]
    best, ids = logits.cpu().topk(2, dim=1)
    check_layer(decoded, x[:24].cpu(), Wide, ids[:24], best.double().softmax(1)[:24])
    # the prompt's activations are quantized twice: half a step of e4m3 (2^-4) of each, and the sums' signs vary
    y = torch.stack([sum(p * ((x[t].cpu().double() @ Wide.wide[0][e]).relu() @ Wide.wide[1][e])
                         for e, p in zip(ids[t].tolist(), best.double().softmax(1)[t].tolist())) for t in range(300)])
    assert float((prompt.cpu().double() - y).norm() / y.norm()) <= 2 * 2.0 ** -4
    served.decode(x[:1], logits[:1])


def test_module_runs():
    from tiled_dense_gemm_relu_amd import expert_layer
    decoded, prompt, _, _ = expert_layer.serve_experts()
    assert decoded.isfinite().all() and prompt.isfinite().all() and prompt.shape == (500, 256)


# ---------------------------------------------------------------- compiled marshalling


class NotCompiled:
    """Leaves every call to Python."""

    def quantize(self, *args):
        return None

    multiply = backward = experts = quantize


def both_routes(monkeypatch, call):
    """What a call returns through the compiled marshalling (which has to take it) and through Python's."""
    class Counting:
        taken = 0

        def __init__(self, calls):
            self.calls = calls

        def __getattr__(self, name):
            def call(*args):
                out = getattr(self.calls, name)(*args)
                Counting.taken += out is not None
                return out
            return call
    with monkeypatch.context() as m:
        m.setattr(blocks, "_calls", Counting(blocks._compiled()))
        compiled = call()
        m.setattr(blocks, "_calls", NotCompiled())
        return compiled, call(), Counting.taken


def same_tensors(u, v):
    assert u.shape == v.shape and u.dtype == v.dtype and u.stride() == v.stride() and not u.requires_grad
    return torch.equal(u.view(torch.uint8) if u.element_size() == 1 else u, v.view(torch.uint8) if v.element_size() == 1 else v)


@pytest.mark.parametrize("shape", [(1, 16), (48, 160), (3, 32, 144), (1, 1), (17, 130), (2, 33, 31), (3, 1040), (1100, 5), (2, 20, 2049)])
@pytest.mark.parametrize("kw", [{}, {"tiles": True, "transposed": True}, {"rows": False, "transposed": True, "power_of_two": True},
                                {"dtype": E5M2, "masked": True, "transposed": True}])
def test_compiled_quantizer_is_the_same(monkeypatch, shape, kw):
    kw = dict(kw)
    x = randn(shape, 1).to(DEV).requires_grad_()
    if kw.pop("masked", False):
        kw["mask"] = randn(shape, 2).to(DEV)
    a, b, taken = both_routes(monkeypatch, lambda: gr.quantize_blocks(x, **kw))
    assert taken == 1 and len(a) == len(b)
    assert all(same_tensors(u, v) for u, v in zip(a, b))


@pytest.mark.parametrize("K", [32, 150])
@pytest.mark.parametrize("grouped", [False, True])
@pytest.mark.parametrize("kw", [{}, {"out_dtype": torch.float16, "relu": False}, {"b_rows": True, "config": blocks.CONFIG_64}])
def test_compiled_product_is_the_same(monkeypatch, K, grouped, kw):
    q, s = gr.quantize_blocks(randn((40, K), 1).to(DEV))
    w, sw = gr.quantize_blocks(randn((2, 24, K) if grouped else (24, K), 2).to(DEV), E5M2, tiles=not kw.get("b_rows", False))
    ends = torch.tensor([10, 37], dtype=torch.int32, device=DEV) if grouped else None
    a, b, taken = both_routes(monkeypatch, lambda: gr.gemm_relu_blocks(q, s, w, sw, ends=ends, **kw))
    assert taken == 1 and same_tensors(a, b)


@pytest.mark.parametrize("shape", [(32, 48, 64), (33, 50, 70)])
@pytest.mark.parametrize("kw", [{}, {"relu": False}, {"dtype": E4M3}])
def test_compiled_gradients_are_the_same(monkeypatch, shape, kw):
    M, N, K = shape
    xt, sx = gr.quantize_blocks(randn((M, K), 1).to(DEV), rows=False, transposed=True)
    wt, sw = gr.quantize_blocks(randn((N, K), 2).to(DEV), tiles=True, rows=False, transposed=True)
    dc, c = randn((M, N), 3).to(DEV).requires_grad_(), randn((M, N), 4).to(DEV)
    call = lambda: gr.gemm_relu_blocks_backward(dc, c if kw.get("relu", True) else None, xt, sx, wt, sw, **kw)  # noqa: E731
    call()                                               # takes the stream's workspace
    a, b, taken = both_routes(monkeypatch, call)
    assert taken == 1 and all(same_tensors(u, v) for u, v in zip(a, b))
    gr.release_workspaces()
    again, _, taken = both_routes(monkeypatch, call)     # without one Python does the call
    assert taken == 0 and all(same_tensors(u, v) for u, v in zip(a, again))


@pytest.mark.parametrize("kind", ["nk", "kn", "e4m3"])
@pytest.mark.parametrize("renormalize", [True, False])
def test_compiled_expert_layer_is_the_same(monkeypatch, kind, renormalize):
    layer = Layer(kind, torch.bfloat16, 6, 100, 70, 90, 5)
    x, logits = randn((5, 100), 1).to(DEV), torch.randn((5, 6), generator=gen(2)).to(DEV)
    call = lambda: layer(x, logits, 2, renormalize=renormalize)  # noqa: E731
    call()
    a, b, taken = both_routes(monkeypatch, call)
    assert taken == 1 and len(a) == len(b) == 3 and all(same_tensors(u, v) for u, v in zip(a, b))
    x.requires_grad_()
    a, b, taken = both_routes(monkeypatch, call)         # (taken inside the node of autograd's graph)
    assert taken == 1 and a[0].requires_grad and b[0].requires_grad and torch.equal(a[0], b[0])
    with torch.no_grad():
        assert both_routes(monkeypatch, call)[2] == 1


def test_compiled_marshalling_refuses_what_python_refuses(monkeypatch):
    x = randn((32, 32), 1).to(DEV)
    q, s = gr.quantize_blocks(x)
    w, sw = gr.quantize_blocks(x, tiles=True)
    e, logits = x.expand(2, 32, 32).contiguous(), torch.zeros((32, 2), device=DEV)
    short = torch.zeros(31 * 48 + 20, dtype=torch.uint8, device=DEV).view(E4M3).as_strided((32, 20), (48, 1))
    bad = [lambda: gr.quantize_blocks(x.float()), lambda: gr.quantize_blocks(x, torch.float16), lambda: gr.quantize_blocks(x.t()),
           lambda: gr.quantize_blocks(x.cpu()), lambda: gr.quantize_blocks(x[0]), lambda: gr.quantize_blocks(x, mask=x[:16]),
           lambda: gr.quantize_blocks(x, rows=False), lambda: gr.quantize_blocks(None), lambda: gr.quantize_blocks(x, mask=3),
           lambda: gr.gemm_relu_blocks(q, s, w, sw.cpu()), lambda: gr.gemm_relu_blocks(q, s[:, :16], w, sw),
           lambda: gr.gemm_relu_blocks(q, s, w, sw, ends=sw), lambda: gr.gemm_relu_blocks(q, s, w[:, :16], sw),
           lambda: gr.gemm_relu_blocks(q, s, w, sw, config=9), lambda: gr.gemm_relu_blocks(x, s, w, sw),
           lambda: gr.gemm_relu_blocks(q, s, w, s), lambda: gr.gemm_relu_blocks(q, s, w, sw, b_rows=True),
           lambda: gr.gemm_relu_blocks(short, s, short, sw), lambda: gr.gemm_relu_blocks(q.t(), s, w, sw),
           lambda: gr.gemm_relu_blocks_backward(x, x, q, s, w, sw[:, :0]), lambda: gr.gemm_relu_blocks_backward(x, None, q, s, w, sw),
           lambda: gr.gemm_relu_blocks_backward(x, x[:16], q, s, w, sw), lambda: gr.gemm_relu_blocks_backward(x, x, q, s, w[:16], sw),
           lambda: gr.gemm_relu_blocks_backward(x, x, q, s, w, sw, dtype=torch.float16),
           lambda: gr.gemm_relu_blocks_backward(x.float(), x, q, s, w, sw),
           lambda: gr.gemm_relu_experts(x, e, e, logits, 3), lambda: gr.gemm_relu_experts(x, e, e, logits, None),
           lambda: gr.gemm_relu_experts(x, e, e, logits[:, :1], 1), lambda: gr.gemm_relu_experts(x, e, e.half(), logits, 1),
           lambda: gr.gemm_relu_experts(x, e, e, logits, 1, w1_scales=s), lambda: gr.gemm_relu_experts(x, e, e, logits, 1, b_layout=7),
           lambda: gr.gemm_relu_experts(x, e, e[:, :16], logits, 1), lambda: gr.gemm_relu_experts(x, q, q, logits, 1),
           lambda: gr.gemm_relu_experts(x.repeat(3, 1), e, e, logits.repeat(3, 1), 1)]
    for i, call in enumerate(bad):
        errors = []
        for calls in (blocks._compiled(), NotCompiled()):
            with monkeypatch.context() as m:
                m.setattr(blocks, "_calls", calls)
                with pytest.raises(Exception) as e:
                    call()
                errors.append((type(e.value), str(e.value)))
        assert errors[0] == errors[1], i

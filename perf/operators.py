"""The operators whose rows choose their weights, as measured cases: products grouped by expert, their
gradient, and a shared projection with low-rank adapters.

Plain forms are elementary torch operations in 32 bits, rounded once; with ``own`` the calls are the
framework's.  ``ends`` holds the row after each group's (segment's) last row, on the GPU.
"""
import math

import numpy as np
import torch

own = False

_DT = {"fp16": torch.float16, "bf16": torch.bfloat16}


def listed():
    return [
        # Products grouped by expert.  The smallest call: 16 tokens of a toy layer (latency).
        {"name": "expert_smallest", "op": "grouped", "rows": 16, "spare": 0, "groups": 8, "skew": 0.0,
         "k": 256, "n": 256, "dtype": "fp16", "layout": "kn", "relu": True},
        # A decoding step: 64 tokens over 64 experts, a third of them without a token: weights are streamed.
        {"name": "expert_decode", "op": "grouped", "rows": 64, "spare": 0, "groups": 64, "skew": 0.0,
         "k": 2048, "n": 2048, "dtype": "bf16", "layout": "nk", "relu": True},
        # Ragged sizes, rows that are no multiple of 16 bytes, and spare rows past the last group.
        {"name": "expert_ragged", "op": "grouped", "rows": 4000, "spare": 37, "groups": 5, "skew": 0.7,
         "k": 4100, "n": 1100, "dtype": "bf16", "layout": "kn", "relu": False},
        # A prompt's tokens over many experts: groups of about half a large tile.
        {"name": "expert_prompt", "op": "grouped", "rows": 4096, "spare": 0, "groups": 32, "skew": 0.3,
         "k": 2048, "n": 2048, "dtype": "bf16", "layout": "kn", "relu": True},
        # A training batch's forward pass (the largest).
        {"name": "expert_batch", "op": "grouped", "rows": 16384, "spare": 0, "groups": 16, "skew": 0.2,
         "k": 4096, "n": 8192, "dtype": "fp16", "layout": "nk", "relu": True},
        # Gradients.  A small layer's.
        {"name": "expert_grad_small", "op": "grouped_backward", "rows": 256, "spare": 0, "groups": 8, "skew": 0.0,
         "k": 512, "n": 512, "dtype": "fp16", "layout": "kn", "relu": True},
        # A training batch's.
        {"name": "expert_grad", "op": "grouped_backward", "rows": 8192, "spare": 0, "groups": 16, "skew": 0.2,
         "k": 2048, "n": 4096, "dtype": "bf16", "layout": "kn", "relu": True},
        # Odd row lengths, spare rows, no activation.
        {"name": "expert_grad_odd", "op": "grouped_backward", "rows": 1000, "spare": 9, "groups": 7, "skew": 0.5,
         "k": 1101, "n": 517, "dtype": "fp16", "layout": "nk", "relu": False},
        # Adapters beside a shared projection.  One token of one request.
        {"name": "adapter_one_token", "op": "adapters", "rows": 1, "segments": 1, "adapters": 8, "rank": 16,
         "k": 4096, "n": 4096, "dtype": "bf16", "layout": "nk", "relu": True},
        # A decoding step of 64 requests with 32 adapters between them, over a wide projection.
        {"name": "adapter_decode", "op": "adapters", "rows": 64, "segments": 64, "adapters": 32, "rank": 16,
         "k": 8192, "n": 16384, "dtype": "bf16", "layout": "kn", "relu": True},
        # Prompts of six requests.
        {"name": "adapter_prompt", "op": "adapters", "rows": 4096, "segments": 6, "adapters": 4, "rank": 64,
         "k": 4096, "n": 8192, "dtype": "fp16", "layout": "kn", "relu": True},
        # A mixed batch (prompt chunks and single tokens) with odd sizes and an odd rank.
        {"name": "adapter_mixed_odd", "op": "adapters", "rows": 700, "segments": 40, "adapters": 12, "rank": 12,
         "k": 1100, "n": 2050, "dtype": "fp16", "layout": "nk", "relu": False},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    """A row length: mostly whole cache lines, some of 16 bytes' multiples, some of any length."""
    v, kind = _log(rng, lo, hi), rng.random()
    step = 64 if kind < 0.6 else 8 if kind < 0.8 else 1
    return max(lo, v // step * step)


def draw(rng):
    most = max((work(c) for c in listed()), key=lambda w: w["flops"])
    while True:
        op = rng.choice(["grouped", "grouped_backward", "adapters"])
        c = {"op": op, "rows": _log(rng, 1, 16384), "k": _width(rng, 256, 8192), "n": _width(rng, 256, 16384),
             "dtype": rng.choice(["fp16", "bf16"]), "layout": rng.choice(["kn", "nk"]),
             "relu": rng.random() < 0.6}
        if op == "adapters":
            c["segments"] = c["rows"] if c["rows"] <= 256 and rng.random() < 0.4 else _log(rng, 1, min(64, c["rows"]))
            c["adapters"] = _log(rng, 1, 64)
            c["rank"] = rng.choice([8, 16, 16, 32, 64, 64, 128, rng.randint(1, 100)])
        else:
            c["groups"] = _log(rng, 1, 128)
            c["spare"] = rng.choice([0, 0, _log(rng, 1, 64)])
            c["skew"] = round(rng.uniform(0.0, 1.0), 2)
        w = work(c)
        stored = c.get("groups", 1) * c["k"] * c["n"] * 2
        if w["flops"] <= 0.9 * most["flops"] and w["bytes"] <= 0.9 * most["bytes"] and stored <= 0.9 * most["bytes"]:
            return c


def _shares(case):
    p = np.arange(1, case["groups"] + 1, dtype=np.float64) ** -case["skew"]
    return p / p.sum()


def _sizes(case, g):
    """Rows of each group (drawn from the router's shares) or segment (chunks and single tokens)."""
    if case["op"] == "adapters":
        s, rows = case["segments"], case["rows"]
        if s == rows:
            return [1] * s
        cuts = torch.randperm(rows - 1, generator=g)[: s - 1].sort().values + 1 if rows > 1 else torch.empty(0)
        cuts = [0] + [int(v) for v in cuts] + [rows]
        return [b - a for a, b in zip(cuts, cuts[1:])]
    shares = torch.from_numpy(_shares(case))[torch.randperm(case["groups"], generator=g)]
    picks = torch.multinomial(shares, case["rows"], replacement=True, generator=g)
    return torch.bincount(picks, minlength=case["groups"]).tolist()


def prepare(case, seed):
    host = torch.Generator().manual_seed(int(seed))
    dev = "cuda" if torch.cuda.is_available() else "cpu"
    g = torch.Generator(device=dev).manual_seed(int(seed) + 17)
    dt, k, n, nk = _DT[case["dtype"]], case["k"], case["n"], case["layout"] == "nk"

    def normal(shape, scale):
        return (torch.randn(shape, generator=g, device=dev, dtype=torch.float32) * scale).to(dt)

    sizes = _sizes(case, host)
    s = {"case": case, "cap": max(1, max(sizes)),
         "ends": torch.tensor(np.cumsum(sizes), dtype=torch.int32, device=dev)}
    if case["op"] == "adapters":
        rows, count, rank = case["rows"], case["adapters"], case["rank"]
        s["x"] = normal((rows, k), 1.0)
        s["w"] = normal((n, k) if nk else (k, n), k ** -0.5)
        s["u"] = normal((count, rank, k) if nk else (count, k, rank), k ** -0.5)
        s["v"] = normal((count, n, rank) if nk else (count, rank, n), 1.0)
        s["scales"] = torch.rand(count, generator=g, device=dev) * 0.5 / rank ** 0.5 + 0.1 / rank ** 0.5
        # One request in eight of a batch uses no adapter.
        ids = torch.randint(0, count, (case["segments"],), generator=host, dtype=torch.int32)
        none = torch.rand(case["segments"], generator=host) < 0.125
        none[0] = False
        s["ids"] = torch.where(none, torch.full_like(ids, -1), ids).to(dev)
        return s
    rows, groups = case["rows"] + case["spare"], case["groups"]
    s["a"] = normal((rows, k), 1.0)
    s["b"] = torch.empty((groups, n, k) if nk else (groups, k, n), dtype=dt, device=dev)
    for e in range(groups):
        s["b"][e] = normal((n, k) if nk else (k, n), k ** -0.5)
    if case["op"] == "grouped_backward":
        s["dc"] = normal((rows, n), 0.5)
        s["c"] = normal((rows, n), 1.0)
        if case["relu"]:
            s["c"] = s["c"].clamp_min_(0)
    return s


def run(s):
    return _RUN[s["case"]["op"]](s)


def _layout(gr, s):
    return gr.B_NK if s["case"]["layout"] == "nk" else gr.B_KN


# ---------------------------------------------------------------- plain forms


def _slots(s, rows, count):
    """For each row its group (``count``: none) and its place in the group."""
    at = torch.arange(rows, device=s["ends"].device)
    ends = s["ends"].long()
    group = torch.searchsorted(ends, at, right=True)
    starts = torch.cat([ends.new_zeros(1), ends])
    place = torch.where(group < count, at - starts[group], torch.zeros_like(at))
    return group, place, group < count


def _padded(s, x, group, place, inside, count):
    """Rows laid out by group, (count, cap, width), in 32 bits; rows of no group are left out."""
    out = torch.zeros((count, s["cap"], x.shape[1]), dtype=torch.float32, device=x.device)
    out[group[inside], place[inside]] = x[inside].float()
    return out


def _back(y, group, place, inside, rows):
    out = torch.zeros((rows, y.shape[2]), dtype=y.dtype, device=y.device)
    out[inside] = y[group[inside], place[inside]]
    return out


def _wide(t, swap):
    """A stack of matrices in 32 bits, each transposed if ``swap``, laid out densely."""
    return (t.transpose(1, 2) if swap else t).to(torch.float32, memory_format=torch.contiguous_format)


def _act(y, case):
    return y.clamp_min(0) if case["relu"] else y


def _grouped(s):
    case = s["case"]
    if own:
        import tiled_dense_gemm_relu_amd as gr
        return gr.gemm_relu_grouped(s["a"], s["b"], s["ends"], b_layout=_layout(gr, s), relu=case["relu"])
    rows, count = s["a"].shape[0], case["groups"]
    where = _slots(s, rows, count)
    y = torch.bmm(_padded(s, s["a"], *where, count), _wide(s["b"], case["layout"] == "nk"))
    return _act(_back(y, *where, rows), case).to(s["a"].dtype)


def _grouped_backward(s):
    case = s["case"]
    if own:
        import tiled_dense_gemm_relu_amd as gr
        da, db = gr.gemm_relu_grouped_backward(s["dc"], s["c"], s["a"], s["b"], s["ends"], b_layout=_layout(gr, s),
                                               relu=case["relu"])
        return {"da": da, "db": db}
    rows, count, nk, dt = s["a"].shape[0], case["groups"], case["layout"] == "nk", s["a"].dtype
    where = _slots(s, rows, count)
    d = s["dc"].float()
    if case["relu"]:
        d = d * (s["c"] > 0)
    dp, ap = _padded(s, d, *where, count), _padded(s, s["a"], *where, count)
    da = _back(torch.bmm(dp, _wide(s["b"], not nk)), *where, rows)
    db = torch.bmm(_wide(dp, True), ap) if nk else torch.bmm(_wide(ap, True), dp)
    return {"da": da.to(dt), "db": db.to(dt)}


def _adapters(s):
    case = s["case"]
    if own:
        import tiled_dense_gemm_relu_amd as gr
        return gr.gemm_relu_adapters(s["x"], s["w"], s["u"], s["v"], s["scales"], s["ends"], s["ids"],
                                     b_layout=_layout(gr, s), relu=case["relu"])
    rows, count, nk = case["rows"], case["segments"], case["layout"] == "nk"
    where = _slots(s, rows, count)
    ids = s["ids"].long()
    pick = ids.clamp_min(0)
    scale = torch.where(ids >= 0, s["scales"][pick], torch.zeros((), device=ids.device))
    t = torch.bmm(_padded(s, s["x"], *where, count), _wide(s["u"][pick], nk)) * scale[:, None, None]
    low = _back(torch.bmm(t, _wide(s["v"][pick], nk)), *where, rows)
    w = s["w"].float()
    return _act(s["x"].float() @ (w.t() if nk else w) + low, case).to(s["x"].dtype)


_RUN = {"grouped": _grouped, "grouped_backward": _grouped_backward, "adapters": _adapters}


# ---------------------------------------------------------------- work and exact values


def work(case):
    k, n = case["k"], case["n"]
    if case["op"] == "adapters":
        m, r = case["rows"], case["rank"]
        used = case["adapters"] * (1 - (1 - 1 / case["adapters"]) ** (case["segments"] * 0.875))
        return {"bytes": 2 * (m * k + k * n + m * n + max(1.0, used) * r * (k + n)),
                "flops": 2 * m * k * n + 2 * m * r * (k + n) * 0.875}
    m, rows = case["rows"], case["rows"] + case["spare"]
    used = float((1 - (1 - _shares(case)) ** m).sum())          # groups that get a row
    if case["op"] == "grouped":
        return {"bytes": 2 * (m * k + used * k * n + rows * n), "flops": 2 * m * k * n}
    return {"bytes": 2 * (m * k + used * k * n + (2 if case["relu"] else 1) * m * n + rows * k + case["groups"] * k * n),
            "flops": 4 * m * k * n}


def exact(case, seed):
    """The definitions, group by group, in 64 bits."""
    s = prepare(case, seed)
    nk, ends = case["layout"] == "nk", [0] + s["ends"].tolist()
    spans = list(zip(range(len(ends) - 1), ends, ends[1:]))

    def kn(w):
        w = w.double()
        return w.t().contiguous() if nk else w

    if case["op"] == "adapters":
        x = s["x"].double()
        y = x @ kn(s["w"])
        for e, lo, hi in spans:
            i = int(s["ids"][e])
            if i >= 0:
                y[lo:hi] += float(s["scales"][i]) * ((x[lo:hi] @ kn(s["u"][i])) @ kn(s["v"][i]))
        return y.relu() if case["relu"] else y
    rows = s["a"].shape[0]
    if case["op"] == "grouped":
        y = torch.zeros((rows, case["n"]), dtype=torch.float64, device=s["a"].device)
        for e, lo, hi in spans:
            if hi > lo:
                y[lo:hi] = s["a"][lo:hi].double() @ kn(s["b"][e])
        return y.relu() if case["relu"] else y
    d = s["dc"].double()
    if case["relu"]:
        d[s["c"] <= 0] = 0
    da = torch.zeros((rows, case["k"]), dtype=torch.float64, device=d.device)
    db = torch.zeros(s["b"].shape, dtype=torch.float64, device=d.device)
    for e, lo, hi in spans:
        if hi > lo:
            da[lo:hi] = d[lo:hi] @ kn(s["b"][e]).t().contiguous()
            grad = s["a"][lo:hi].double().t().contiguous() @ d[lo:hi]
            db[e] = grad.t() if nk else grad
    return {"da": da, "db": db}

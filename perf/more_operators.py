"""Products of 8-bit floating-point matrices scaled by blocks of 128, as measured cases: the quantizer that
makes such matrices, the product (dense, and grouped by expert), its gradients, and a whole expert layer for
a few tokens.

Plain forms are elementary torch operations in 32 bits, rounded once; with ``own`` the calls are the
framework's.  A quantized matrix is a float8 tensor whose rows start at multiples of 16 bytes, with one
float32 scale for 128 elements of a row (``scales[block, row]``) or for a tile of 128 x 128
(``scales[row block, block]``); an element stands for its 8-bit value times its scale.
"""
import math

import numpy as np
import torch

own = False

_DT = {"fp16": torch.float16, "bf16": torch.bfloat16}
_F8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
_MOST = {"e4m3": 448.0, "e5m2": 57344.0}       # the formats' largest values
_FLOOR = 2.0 ** -80                            # magnitude that a block's scale covers at least
_B = 128


def listed():
    return [
        # The quantizer.  One token's activations on their way into a decoding step's product (latency).
        {"name": "quantize_token", "op": "quantize", "rows": 1, "k": 4096, "dtype": "bf16", "format": "e4m3",
         "form": "rows", "mask": False, "power": False},
        # A training batch's gradient behind a ReLU, by rows and transposed by rows, as both its products want it.
        {"name": "quantize_gradient", "op": "quantize", "rows": 8192, "k": 4096, "dtype": "bf16", "format": "e5m2",
         "form": "both", "mask": True, "power": False},
        # The product.  The small correctness shape of the dense product (latency).
        {"name": "blocks_small", "op": "product", "rows": 256, "spare": 0, "groups": 0, "skew": 0.0, "k": 256, "n": 256,
         "dtype": "fp16", "format": "e4m3", "format_b": "e4m3", "b_rows": False, "relu": True},
        # A decoding step: 64 tokens, the weights are streamed.
        {"name": "blocks_decode", "op": "product", "rows": 64, "spare": 0, "groups": 0, "skew": 0.0, "k": 8192, "n": 16384,
         "dtype": "bf16", "format": "e4m3", "format_b": "e4m3", "b_rows": False, "relu": True},
        # Ragged tails in all three sizes, no activation.
        {"name": "blocks_ragged", "op": "product", "rows": 4000, "spare": 0, "groups": 0, "skew": 0.0, "k": 4100, "n": 11000,
         "dtype": "fp16", "format": "e4m3", "format_b": "e4m3", "b_rows": False, "relu": False},
        # The benchmark's square (the largest).
        {"name": "blocks_square", "op": "product", "rows": 8192, "spare": 0, "groups": 0, "skew": 0.0, "k": 8192, "n": 8192,
         "dtype": "bf16", "format": "e4m3", "format_b": "e4m3", "b_rows": False, "relu": True},
        # A prompt's tokens over many experts, with spare rows past the last group.
        {"name": "blocks_experts", "op": "product", "rows": 4096, "spare": 37, "groups": 32, "skew": 0.3, "k": 2048,
         "n": 2048, "dtype": "bf16", "format": "e4m3", "format_b": "e4m3", "b_rows": False, "relu": True},
        # Gradients of a layer.  Odd sizes.
        {"name": "blocks_grad_odd", "op": "gradient", "rows": 1000, "k": 1101, "n": 517, "dtype": "fp16", "format": "e5m2",
         "relu": True},
        # A training batch's.
        {"name": "blocks_grad", "op": "gradient", "rows": 8192, "k": 4096, "n": 4096, "dtype": "bf16", "format": "e5m2",
         "relu": True},
        # The expert layer for a few tokens.  One token, 4 of 64 experts, 16-bit weights (latency).
        {"name": "layer_token", "op": "experts", "rows": 1, "experts": 64, "top": 4, "k": 2048, "hidden": 2048,
         "dtype": "bf16", "weights": "nk", "renormalize": True},
        # A decoding step of 24 requests with 8-bit weights.
        {"name": "layer_decode", "op": "experts", "rows": 24, "experts": 64, "top": 4, "k": 2048, "hidden": 4096,
         "dtype": "bf16", "weights": "e4m3", "renormalize": True},
        # Odd sizes, weights stored (in, out), weights of the softmax over all experts.
        {"name": "layer_odd", "op": "experts", "rows": 7, "experts": 12, "top": 3, "k": 1101, "hidden": 1300,
         "dtype": "fp16", "weights": "kn", "renormalize": False},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    """A row length: mostly whole blocks, some multiples of 16, some of any length."""
    v, kind = _log(rng, lo, hi), rng.random()
    step = 128 if kind < 0.6 else 16 if kind < 0.8 else 1
    return max(lo, v // step * step)


def draw(rng):
    most = [work(c) for c in listed()]
    flops, moved = max(w["flops"] for w in most), max(w["bytes"] for w in most)
    while True:
        op = rng.choice(["quantize", "product", "product", "gradient", "experts"])
        c = {"op": op, "dtype": rng.choice(["fp16", "bf16"]), "k": _width(rng, 128, 8192)}
        form = rng.choice(["e4m3", "e4m3", "e5m2"])
        if op == "quantize":
            c.update(rows=_log(rng, 1, 16384), format=form, form=rng.choice(["rows", "rows", "both", "transposed", "tiles"]),
                     mask=rng.random() < 0.4, power=rng.random() < 0.3)
        elif op == "product":
            groups = rng.choice([0, 0, _log(rng, 1, 64)])
            c.update(rows=_log(rng, 1, 16384), spare=rng.choice([0, _log(rng, 1, 64)]) if groups else 0, groups=groups,
                     skew=round(rng.uniform(0.0, 1.0), 2) if groups else 0.0, n=_width(rng, 128, 16384), format=form,
                     format_b=rng.choice(["e4m3", "e4m3", "e5m2"]), b_rows=rng.random() < 0.2, relu=rng.random() < 0.6)
        elif op == "gradient":
            c.update(rows=_log(rng, 1, 16384), n=_width(rng, 128, 8192), format=form, relu=rng.random() < 0.6)
        else:
            experts = _log(rng, 2, 128)
            c.update(rows=_log(rng, 1, 64), experts=experts, top=rng.randint(1, min(8, experts)), k=_width(rng, 128, 4096),
                     hidden=_width(rng, 128, 8192), weights=rng.choice(["nk", "kn", "e4m3", "e4m3", "e5m2"]),
                     renormalize=rng.random() < 0.7)
        w = work(c)
        stored = (4 * c["experts"] * c["k"] * c["hidden"] if op == "experts" else
                  max(1, c.get("groups", 1)) * c["k"] * c.get("n", 1))
        if w["flops"] <= 0.9 * flops and w["bytes"] <= 0.9 * moved and stored <= 5e9:
            return c


def _shares(case):
    p = np.arange(1, case["groups"] + 1, dtype=np.float64) ** -case["skew"]
    return p / p.sum()


def _blocks(n):
    return (n + _B - 1) // _B


# ---------------------------------------------------------------- quantized matrices in elementary operations


def _pitched(shape, dtype, device):
    """A float8 tensor whose rows start at multiples of 16 bytes."""
    pitch = (shape[-1] + 15) // 16 * 16
    return torch.zeros(shape[:-1] + (pitch,), dtype=torch.uint8, device=device)[..., : shape[-1]].view(dtype)


def _cast(v, form):
    """8-bit values, in rows that start at multiples of 16 bytes."""
    out = _pitched(tuple(v.shape), _F8[form], v.device)
    out.copy_(v.to(_F8[form]))
    return out


def _scale(amax, form, power):
    amax = amax.clamp_min(_FLOOR)
    s = amax / torch.full_like(amax, _MOST[form])       # (by a number, the GPU multiplies with its reciprocal)
    if power:
        fraction, exponent = torch.frexp(s)
        s = torch.ldexp(torch.ones_like(s), torch.where(fraction > 0.5, exponent, exponent - 1))
    return s


def _to_blocks(x, tiles):
    """(..., rows, cols) of float32 as (..., row blocks, rows a block, col blocks, 128), zeros behind the ends."""
    rows, cols = x.shape[-2:]
    high = _B if tiles else 1
    padded = torch.nn.functional.pad(x, (0, -cols % _B, 0, -rows % high))
    return padded.reshape(x.shape[:-2] + (-(-rows // high), high, _blocks(cols), _B))


def _quantize(x, form, tiles=False, power=False):
    """(8-bit matrix, scales) of float32 x (..., rows, cols): scales (..., blocks, rows), or (..., row blocks, blocks)."""
    parts = _to_blocks(x, tiles)
    s = _scale(parts.abs().amax(dim=(-3, -1), keepdim=True), form, power)
    q = (parts / s).reshape(x.shape[:-2] + (parts.shape[-4] * parts.shape[-3], -1))[..., : x.shape[-2], : x.shape[-1]]
    s = s[..., 0, :, 0]
    return _cast(q, form), (s if tiles else s.transpose(-1, -2).contiguous())


def _wide(q, s, tiles, dt=torch.float32):
    """What a quantized matrix stands for."""
    rows, cols = q.shape[-2:]
    if tiles:
        s = s.repeat_interleave(_B, dim=-2)[..., :rows, :]
    else:
        s = s.transpose(-1, -2)
    return q.to(dt) * s.to(dt).repeat_interleave(_B, dim=-1)[..., :cols]


# ---------------------------------------------------------------- inputs


def prepare(case, seed):
    host = torch.Generator().manual_seed(int(seed))
    dev = "cuda" if torch.cuda.is_available() else "cpu"
    g = torch.Generator(device=dev).manual_seed(int(seed) + 17)
    dt, k = _DT[case["dtype"]], case["k"]

    def normal(shape, scale):
        return torch.randn(shape, generator=g, device=dev, dtype=torch.float32) * scale

    def spread(rows, cols, scale=1.0):
        """Rows and columns of different magnitudes, as activations have."""
        return normal((rows, cols), scale) * normal((rows, 1), 0.4).exp() * normal((1, cols), 0.4).exp()

    s = {"case": case}
    if case["op"] == "quantize":
        s["x"] = spread(case["rows"], k).to(dt)
        s["above"] = normal((case["rows"], k), 1.0).clamp_min_(0).to(dt) if case["mask"] else None
    elif case["op"] == "product":
        groups, n, rows = case["groups"], case["n"], case["rows"] + case["spare"]
        s["a"], s["sa"] = _quantize(spread(rows, k), case["format"])
        one = lambda: _quantize(normal((n, k), k ** -0.5), case["format_b"], tiles=not case["b_rows"])  # noqa: E731
        s["ends"] = None
        if groups:
            shares = torch.from_numpy(_shares(case))[torch.randperm(groups, generator=host)]
            picks = torch.multinomial(shares, case["rows"], replacement=True, generator=host)
            sizes = torch.bincount(picks, minlength=groups)
            s["cap"] = int(sizes.max())
            s["ends"] = sizes.cumsum(0).to(torch.int32).to(dev)
            s["b"], first = _pitched((groups, n, k), _F8[case["format_b"]], dev), one()
            s["sb"] = torch.empty((groups,) + tuple(first[1].shape), dtype=torch.float32, device=dev)
            for e in range(groups):
                s["b"][e], s["sb"][e] = one() if e else first
        else:
            s["b"], s["sb"] = one()
    elif case["op"] == "gradient":
        rows, n = case["rows"], case["n"]
        s["dc"] = spread(rows, n, 2.0 ** -6).to(dt)
        s["c"] = normal((rows, n), 1.0).clamp_min_(0).to(dt) if case["relu"] else None
        s["xt"], s["sxt"] = _quantize(spread(rows, k).t().contiguous(), "e4m3")
        s["wt"], s["swt"] = _quantize(normal((k, n), k ** -0.5), "e4m3", tiles=True)
    else:
        experts, hidden, kind = case["experts"], case["hidden"], case["weights"]
        s["x"] = normal((case["rows"], k), 1.0).to(dt)
        # some experts are chosen more often than others
        s["logits"] = normal((case["rows"], experts), 1.0) + normal((1, experts), 0.5)
        shapes = [(hidden, k), (k, hidden)]                       # (out, in)
        if kind in _F8:
            for i, shape in enumerate(shapes):
                w = _pitched((experts,) + shape, _F8[kind], dev)
                scale = torch.empty((experts, _blocks(shape[0]), _blocks(shape[1])), dtype=torch.float32, device=dev)
                for e in range(experts):
                    w[e], scale[e] = _quantize(normal(shape, shape[1] ** -0.5), kind, tiles=True)
                s["w%d" % (i + 1)], s["s%d" % (i + 1)] = w, scale
        else:
            for i, (out, inner) in enumerate(shapes):
                w = torch.empty((experts, out, inner) if kind == "nk" else (experts, inner, out), dtype=dt, device=dev)
                for e in range(experts):
                    w[e] = normal(tuple(w.shape[1:]), inner ** -0.5).to(dt)
                s["w%d" % (i + 1)], s["s%d" % (i + 1)] = w, None
    return s


def run(s):
    return _RUN[s["case"]["op"]](s)


# ---------------------------------------------------------------- plain forms


def _run_quantize(s):
    case, form = s["case"], s["case"]["form"]
    if own:
        import tiled_dense_gemm_relu_amd as gr
        return gr.quantize_blocks(s["x"], dtype=_F8[case["format"]], tiles=form == "tiles", mask=s["above"],
                                  rows=form != "transposed", transposed=form in ("both", "transposed"),
                                  power_of_two=case["power"])
    x = s["x"].float()
    if case["mask"]:
        x = x * (s["above"] > 0)
    out = ()
    if form != "transposed":
        out += _quantize(x, case["format"], form == "tiles", case["power"])
    if form in ("both", "transposed"):
        out += _quantize(x.t().contiguous(), case["format"], False, case["power"])
    return out


def _run_product(s):
    case = s["case"]
    dt, n = _DT[case["dtype"]], case["n"]
    if own:
        import tiled_dense_gemm_relu_amd as gr
        return gr.gemm_relu_blocks(s["a"], s["sa"], s["b"], s["sb"], ends=s["ends"], out_dtype=dt, relu=case["relu"],
                                   b_rows=case["b_rows"])
    a, b = _wide(s["a"], s["sa"], False), _wide(s["b"], s["sb"], not case["b_rows"])
    if s["ends"] is None:
        y = a @ b.t()
    else:
        # rows laid out by group, (groups, most rows of one, k)
        rows, groups = a.shape[0], case["groups"]
        at, ends = torch.arange(rows, device=a.device), s["ends"].long()
        group = torch.searchsorted(ends, at, right=True)
        place = at - torch.cat([ends.new_zeros(1), ends])[group]
        inside = group < groups
        padded = torch.zeros((groups, s["cap"], a.shape[1]), device=a.device)
        padded[group[inside], place[inside]] = a[inside]
        z = torch.bmm(padded, b.transpose(1, 2).contiguous())
        y = torch.zeros((rows, n), device=a.device)
        y[inside] = z[group[inside], place[inside]]
    return (y.clamp_min(0) if case["relu"] else y).to(dt)


def _run_gradient(s):
    case = s["case"]
    dt, form = _DT[case["dtype"]], case["format"]
    if own:
        import tiled_dense_gemm_relu_amd as gr
        dx, dw = gr.gemm_relu_blocks_backward(s["dc"], s["c"], s["xt"], s["sxt"], s["wt"], s["swt"], relu=case["relu"],
                                              dtype=_F8[form])
        return {"dx": dx, "dw": dw}
    d = s["dc"].float()
    if case["relu"]:
        d = d * (s["c"] > 0)
    q, scale = _quantize(d, form)
    qt, scale_t = _quantize(d.t().contiguous(), form)
    dx = _wide(q, scale, False) @ _wide(s["wt"], s["swt"], True).t()
    dw = _wide(qt, scale_t, False) @ _wide(s["xt"], s["sxt"], False).t()
    return {"dx": dx.to(dt), "dw": dw.to(dt)}


def _route(logits, top, renormalize):
    """The largest logits of each row, ties to the lowest index, and their softmax weights."""
    best, ids = torch.sort(logits, dim=1, descending=True, stable=True)
    e = (best - best[:, :1]).exp()
    chosen = e[:, :top]
    return ids[:, :top], chosen / (chosen if renormalize else e).sum(1, keepdim=True)


def _run_experts(s):
    case, top = s["case"], s["case"]["top"]
    kind, dt = case["weights"], _DT[case["dtype"]]
    if own:
        import tiled_dense_gemm_relu_amd as gr
        y, ids, weights = gr.gemm_relu_experts(s["x"], s["w1"], s["w2"], s["logits"], top, w1_scales=s["s1"],
                                               w2_scales=s["s2"], b_layout=gr.B_KN if kind == "kn" else gr.B_NK,
                                               renormalize=case["renormalize"])
        return {"y": y, "ids": ids, "weights": weights}
    x, rows = s["x"].float(), case["rows"]
    ids, weights = _route(s["logits"], top, case["renormalize"])
    few = rows * top < case["experts"]

    def stack(i):
        """(experts or slots, in, out) in 32 bits."""
        w, scale = s["w%d" % i], s["s%d" % i]
        if few:
            w = (w.view(torch.uint8)[ids.reshape(-1)].view(w.dtype) if scale is not None else w[ids.reshape(-1)])
            scale = scale[ids.reshape(-1)] if scale is not None else None
        w = w.float() if scale is None else _wide(w, scale, True)
        return w if kind == "kn" else w.transpose(1, 2).contiguous()

    if few:      # each slot's expert
        h = torch.bmm(x.repeat_interleave(top, dim=0)[:, None], stack(1)).clamp_min(0)
        y = (torch.bmm(h, stack(2))[:, 0].reshape(rows, top, -1) * weights[:, :, None]).sum(1)
    else:        # every expert on every token
        share = torch.zeros((rows, case["experts"]), device=x.device).scatter_(1, ids, weights)
        h = torch.bmm(x[None].expand(case["experts"], -1, -1).contiguous(), stack(1)).clamp_min(0)
        y = (torch.bmm(h, stack(2)) * share.t()[:, :, None]).sum(0)
    return {"y": y.to(dt), "ids": ids.to(torch.int32), "weights": weights}


_RUN = {"quantize": _run_quantize, "product": _run_product, "gradient": _run_gradient, "experts": _run_experts}


# ---------------------------------------------------------------- work and exact values


def work(case):
    m, k = case["rows"], case["k"]
    if case["op"] == "quantize":
        both = 2 if case["form"] == "both" else 1
        scales = m * k / (_B * _B if case["form"] == "tiles" else _B)
        return {"bytes": m * k * (2 + 2 * case["mask"] + both) + 4 * scales * both, "flops": 4 * m * k * both}
    if case["op"] == "gradient":
        n = case["n"]
        return {"bytes": 2 * m * n * (1 + case["relu"]) + m * k + k * n + 4 * m * k / _B + 2 * m * k + 2 * n * k,
                "flops": 4 * m * n * k}
    if case["op"] == "product":
        n, groups = case["n"], case["groups"]
        used = float((1 - (1 - _shares(case)) ** m).sum()) if groups else 1.0     # groups that get a row
        weights = used * n * k * (1 + 4 / (_B if case["b_rows"] else _B * _B))
        return {"bytes": m * k * (1 + 4 / _B) + weights + 2 * (m + case["spare"]) * n, "flops": 2 * m * n * k}
    # experts: weights of the experts that are chosen (as if all were as likely)
    share = case["top"] / case["experts"]
    used = case["experts"] * (1 - (1 - share) ** m)
    size = 1 + 4 / (_B * _B) if case["weights"] in _F8 else 2
    return {"bytes": used * 2 * k * case["hidden"] * size + 2 * 2 * m * k + 4 * m * case["experts"] + 8 * m * case["top"],
            "flops": 4 * m * case["top"] * k * case["hidden"]}


def _exact_quantize(x, form, tiles, power):
    """(values, scales) of a matrix of 64-bit values: the definition with a search for the nearest value by
    the grid's spacing.  The quotient is rounded to 32 bits, as the definition says, then to 8."""
    rows, cols = x.shape
    high = _B if tiles else 1
    bits, low = (3, -6) if form == "e4m3" else (2, -14)           # fraction bits, smallest normal exponent
    amax = torch.zeros((-(-rows // high), _blocks(cols)), dtype=torch.float64, device=x.device)
    for b in range(amax.shape[1]):
        part = x[:, b * _B:(b + 1) * _B].abs().amax(1)
        if tiles:
            part = torch.cat([part, part.new_zeros(-rows % high)]).reshape(-1, high).amax(1)
        amax[:, b] = part
    s = (amax.clamp_min(_FLOOR) / _MOST[form]).float().double()
    if power:
        s = torch.exp2(torch.ceil(torch.log2(s)))
    spread = s.repeat_interleave(high, 0)[:rows].repeat_interleave(_B, 1)[:, :cols]
    t = (x / spread).float().double()
    unit = torch.exp2(torch.floor(torch.log2(t.abs().clamp_min(2.0 ** (low - 8)))).clamp_min(low) - bits)
    return torch.round(t / unit) * unit, (s if tiles else s.t().contiguous())


def exact(case, seed):
    """The definitions in 64 bits."""
    s, op = prepare(case, seed), case["op"]

    def full(q, scale, tiles):
        """A quantized matrix in 64 bits."""
        out = q.double()
        for b in range(scale.shape[1] if tiles else scale.shape[0]):
            cols = out[:, b * _B:(b + 1) * _B]
            cols *= (scale[:, b].double().repeat_interleave(_B)[: out.shape[0], None] if tiles else scale[b].double()[:, None])
        return out

    if op == "quantize":
        x = s["x"].double()
        if case["mask"]:
            x = torch.where(s["above"] > 0, x, torch.zeros_like(x))
        out, form = (), case["form"]
        if form != "transposed":
            out += _exact_quantize(x, case["format"], form == "tiles", case["power"])
        if form in ("both", "transposed"):
            out += _exact_quantize(x.t().contiguous(), case["format"], False, case["power"])
        return out
    if op == "product":
        a = full(s["a"], s["sa"], False)
        if s["ends"] is None:
            y = a @ full(s["b"], s["sb"], not case["b_rows"]).t().contiguous()
        else:
            y, lo = torch.zeros((a.shape[0], case["n"]), dtype=torch.float64, device=a.device), 0
            for e, hi in enumerate(s["ends"].tolist()):
                if hi > lo:
                    y[lo:hi] = a[lo:hi] @ full(s["b"][e], s["sb"][e], not case["b_rows"]).t().contiguous()
                lo = hi
        return y.relu() if case["relu"] else y
    if op == "gradient":
        d = s["dc"].double()
        if case["relu"]:
            d[s["c"] <= 0] = 0
        q, scale = _exact_quantize(d, case["format"], False, False)
        qt, scale_t = _exact_quantize(d.t().contiguous(), case["format"], False, False)
        dx = full(q, scale, False) @ full(s["wt"], s["swt"], True).t().contiguous()
        dw = full(qt, scale_t, False) @ full(s["xt"], s["sxt"], False).t().contiguous()
        return {"dx": dx, "dw": dw}
    x, logits = s["x"].double(), s["logits"].double()
    y = torch.zeros((case["rows"], case["k"]), dtype=torch.float64, device=x.device)
    weights = torch.zeros((case["rows"], case["top"]), dtype=torch.float64, device=x.device)
    ids = torch.zeros((case["rows"], case["top"]), dtype=torch.int32, device=x.device)
    for t in range(case["rows"]):
        row = logits[t].tolist()
        order = sorted(range(len(row)), key=lambda e: (-row[e], e))[: case["top"]]
        total = sum(math.exp(v - row[order[0]]) for v in ([row[e] for e in order] if case["renormalize"] else row))
        for j, e in enumerate(order):
            p = math.exp(row[e] - row[order[0]]) / total
            if s["s1"] is None:
                w1, w2 = s["w1"][e].double(), s["w2"][e].double()
            else:
                w1, w2 = full(s["w1"][e], s["s1"][e], True), full(s["w2"][e], s["s2"][e], True)
            if case["weights"] != "kn":
                w1, w2 = w1.t(), w2.t()
            y[t] += p * ((x[t] @ w1).relu() @ w2)
            ids[t, j], weights[t, j] = e, p
    return {"y": y, "ids": ids, "weights": weights}

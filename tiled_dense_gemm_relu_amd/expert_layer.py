"""An expert layer trained for a few steps and served in 8 bits, then a projection served with adapters.

    python -m tiled_dense_gemm_relu_amd.expert_layer

The layer routes each token to one of ``experts`` two-matrix networks, y = ReLU(x @ B1[e]) @ B2[e].
Tokens are sorted by expert once; the running sum of the experts' token counts, made and kept on the
GPU, is the row table of both products and of all four gradients.  For serving its weights are quantized
once: prompts take the same products on 8-bit matrices, a few tokens the whole layer in one call.
"""
from __future__ import annotations

import torch

from .blocks import gemm_relu_blocks, gemm_relu_experts, quantize_blocks
from .groups import gemm_relu_adapters, gemm_relu_grouped, gemm_relu_grouped_backward


class ExpertLayer:
    """y[m] = ReLU(x[m] @ B1[e]) @ B2[e] for token m's expert e; weights in ``dtype``, fp32 masters."""

    def __init__(self, experts: int, width: int, hidden: int, dtype=torch.bfloat16, device="cuda", seed: int = 0):
        g = torch.Generator(device=device).manual_seed(seed)

        def normal(*shape):
            return torch.randn(shape, generator=g, device=device) * shape[1] ** -0.5
        self.masters = [normal(experts, width, hidden), normal(experts, hidden, width)]
        self.weights = [m.to(dtype) for m in self.masters]
        self.experts = experts

    def route(self, expert: torch.Tensor):
        """(order, ends): the tokens sorted by expert, and the row after each expert's last token."""
        order = torch.argsort(expert, stable=True)
        counts = torch.zeros(self.experts, dtype=torch.int64, device=expert.device).scatter_add_(
            0, expert, torch.ones_like(expert))
        return order, counts.cumsum(0).to(torch.int32)

    def forward(self, x: torch.Tensor, expert: torch.Tensor):
        """The layer's outputs in the order of ``x``, and what backward needs."""
        order, ends = self.route(expert)
        rows = x[order]
        hidden = gemm_relu_grouped(rows, self.weights[0], ends)
        y = gemm_relu_grouped(hidden, self.weights[1], ends, relu=False)
        out = torch.empty_like(y)
        out[order] = y
        return out, (rows, hidden, order, ends)

    def backward(self, dy: torch.Tensor, saved):
        """Gradients with respect to x and to both weights."""
        rows, hidden, order, ends = saved
        dhidden, db2 = gemm_relu_grouped_backward(dy[order], None, hidden, self.weights[1], ends, relu=False)
        drows, db1 = gemm_relu_grouped_backward(dhidden, hidden, rows, self.weights[0], ends)
        dx = torch.empty_like(drows)
        dx[order] = drows
        return dx, [db1, db2]

    def step(self, gradients, rate: float):
        for master, weight, grad in zip(self.masters, self.weights, gradients):
            master.add_(grad.float(), alpha=-rate)
            weight.copy_(master)


class ServedExperts:
    """An ExpertLayer's weights in 8 bits, stored (out, in), with the softmax of its chosen experts' logits.

    ``prompt`` sorts the chosen (token, expert) pairs by expert and multiplies quantized rows; ``decode`` takes
    up to 64 tokens, whose activations it does not quantize.  Both choose alike: ties to the lowest index, logits
    of -inf never, rows of zeros for tokens without a choice and of NaN for those with a logit of NaN or +inf.
    """

    def __init__(self, layer: ExpertLayer, top: int, dtype=torch.float8_e4m3fn):
        if not 1 <= top <= layer.experts:
            raise ValueError(f"top must be 1 to {layer.experts}, got {top}")
        self.top, self.experts, self.dtype = top, layer.experts, dtype
        (self.w1, self.s1), (self.w2, self.s2) = (quantize_blocks(w, dtype, tiles=True, rows=False, transposed=True)
                                                  for w in layer.weights)

    def decode(self, x: torch.Tensor, logits: torch.Tensor):
        return gemm_relu_experts(x, self.w1, self.w2, logits, self.top, w1_scales=self.s1, w2_scales=self.s2)[0]

    def prompt(self, x: torch.Tensor, logits: torch.Tensor):
        best, ids = (t[:, : self.top] for t in logits.sort(dim=1, descending=True, stable=True))
        share, none = best.softmax(dim=1).reshape(-1), (best == -float("inf")).reshape(-1)
        expert, order = ids.reshape(-1).sort(stable=True)
        ends = torch.searchsorted(expert, torch.arange(self.experts, device=x.device), right=True).to(torch.int32)
        rows = order // self.top
        hidden = gemm_relu_blocks(*quantize_blocks(x[rows], self.dtype), self.w1, self.s1, ends=ends, out_dtype=x.dtype)
        y = gemm_relu_blocks(*quantize_blocks(hidden, self.dtype), self.w2, self.s2, ends=ends, out_dtype=x.dtype, relu=False)
        parts = torch.empty(y.shape, dtype=torch.float32, device=x.device)
        parts[order] = (y.float() * share[order][:, None]).masked_fill_(none[order][:, None], 0.0)
        return parts.view(*ids.shape, y.shape[1]).sum(dim=1).to(x.dtype)      # (in the order of the choices, every time)


def train(steps: int = 8, tokens: int = 512, experts: int = 8, width: int = 128, hidden: int = 256, rate: float = 0.1):
    """Fits a fixed random target; returns the mean squared error before each step."""
    torch.manual_seed(1)
    layer = ExpertLayer(experts, width, hidden)
    x = torch.randn(tokens, width, device="cuda").bfloat16()
    target = torch.randn(tokens, width, device="cuda") * 0.5
    expert = torch.randint(0, experts, (tokens,), device="cuda")
    losses = []
    for _ in range(steps):
        y, saved = layer.forward(x, expert)
        off = y.float() - target
        losses.append(float((off * off).mean()))
        _, gradients = layer.backward((off * (2.0 / tokens)).bfloat16(), saved)
        layer.step(gradients, rate)
    return losses


def serve_experts(tokens: int = 24, prompt: int = 500, experts: int = 8, width: int = 256, hidden: int = 512, top: int = 2):
    """A decoding step and a prompt through one layer in 8 bits: (decoded, prompt's outputs, layer, inputs)."""
    layer = ExpertLayer(experts, width, hidden, seed=3)
    served = ServedExperts(layer, top)
    g = torch.Generator(device="cuda").manual_seed(4)
    x = torch.randn(prompt, width, generator=g, device="cuda").bfloat16()
    logits = torch.randn(prompt, experts, generator=g, device="cuda")
    return served.decode(x[:tokens], logits[:tokens]), served.prompt(x, logits), layer, (x, logits)


def serve(requests=((0, 5), (2, 1), (-1, 3), (2, 1)), width: int = 256, out: int = 512, rank: int = 16, adapters: int = 3):
    """A batch of requests, each an (adapter or -1, tokens) pair, through one shared projection."""
    torch.manual_seed(2)
    x = torch.randn(sum(n for _, n in requests), width, device="cuda").bfloat16()
    w = (torch.randn(width, out, device="cuda") * width ** -0.5).bfloat16()
    u = (torch.randn(adapters, width, rank, device="cuda") * width ** -0.5).bfloat16()
    v = torch.randn(adapters, rank, out, device="cuda").bfloat16()
    scales = torch.full((adapters,), rank ** -0.5, device="cuda")
    ids = torch.tensor([i for i, _ in requests], dtype=torch.int32, device="cuda")
    ends = torch.tensor([n for _, n in requests], device="cuda").cumsum(0).to(torch.int32)
    return gemm_relu_adapters(x, w, u, v, scales, ends, ids), (x, w, u, v, scales)


if __name__ == "__main__":
    losses = train()
    print("mean squared error by step: " + " ".join(f"{v:.4f}" for v in losses))
    decoded, prompt, _, _ = serve_experts()
    off = float((decoded.float() - prompt[: len(decoded)].float()).norm() / decoded.float().norm())
    print(f"8-bit experts: {len(decoded)} tokens decoded, {len(prompt)} of a prompt; activations in 8 bits change {off:.1%}")
    y, _ = serve()
    print(f"served {y.shape[0]} tokens of 4 requests: outputs {tuple(y.shape)}, mean {float(y.float().mean()):.4f}")

"""An expert layer trained for a few steps, then a projection served with adapters.

    python -m tiled_dense_gemm_relu_amd.expert_layer

The layer routes each token to one of ``experts`` two-matrix networks, y = ReLU(x @ B1[e]) @ B2[e].
Tokens are sorted by expert once; the running sum of the experts' token counts, made and kept on the
GPU, is the row table of both products and of all four gradients.
"""
from __future__ import annotations

import torch

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
    y, _ = serve()
    print(f"served {y.shape[0]} tokens of 4 requests: outputs {tuple(y.shape)}, mean {float(y.float().mean()):.4f}")

"""A mixture-of-experts feed-forward layer on the grouped operators.

    python examples/expert_layer.py

Trains a small layer for a few steps (row grouping, grouped products and their
gradients), then quantizes its experts to 4 bits and decodes a batch of tokens
through them, one launch per projection, without grouping the rows.
"""
import os
import sys

import torch

if __name__ == "__main__":
    sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from dense_tiled_gemm_02_amd import grouped, w4


class ExpertLayer(torch.nn.Module):
    """Each token goes through its `top` best experts: down(silu(gate x) * up x),
    weighted by the router's normalized probabilities."""

    def __init__(self, width, hidden, experts, top, dtype=torch.bfloat16, device="cuda"):
        super().__init__()
        self.experts, self.top = experts, top
        init = lambda *s: torch.nn.Parameter(torch.randn(s, dtype=dtype, device=device) * s[-2] ** -0.5)
        self.router = init(width, experts)
        self.gate_up = init(experts, width, 2 * hidden)
        self.down = init(experts, hidden, width)

    def route(self, x):
        p, ids = torch.softmax((x @ self.router).float(), -1).topk(self.top)
        return (p / p.sum(-1, keepdim=True)).to(x.dtype), ids

    @staticmethod
    def act(h):
        gate, up = h.chunk(2, -1)
        return torch.nn.functional.silu(gate) * up

    def forward(self, x):
        p, ids = self.route(x)
        offsets, order = grouped.group_rows(ids.reshape(-1), self.experts)
        order = order.long()
        h = self.act(grouped.grouped_linear(x[order // self.top], self.gate_up, offsets))
        y = grouped.grouped_linear(h.contiguous(), self.down, offsets)
        back = torch.empty_like(order)
        back[order] = torch.arange(order.numel(), device=order.device)
        return (y[back].unflatten(0, (-1, self.top)) * p[..., None]).sum(1)

    def quantize(self, group=64):
        """The experts' weights in 4 bits, for decode()."""
        q = lambda weight: w4.w4_quantize(weight.detach().transpose(1, 2), group, zeros=True) + (group,)
        return q(self.gate_up), q(self.down)

    @torch.no_grad()
    def decode(self, x, quantized):
        p, ids = self.route(x)
        ids = ids.reshape(-1)
        project = lambda rows, t: w4.w4_matvec(rows, t[0], t[1], zeros=t[2], group=t[3], experts=ids)
        h = self.act(project(x.repeat_interleave(self.top, 0), quantized[0]))
        y = project(h.contiguous(), quantized[1])
        return (y.unflatten(0, (-1, self.top)) * p[..., None]).sum(1)


def main(width=256, hidden=384, experts=8, top=2, tokens=512, steps=20):
    torch.manual_seed(0)
    layer = ExpertLayer(width, hidden, experts, top)
    teacher = ExpertLayer(width, hidden, experts, top)
    optimizer = torch.optim.Adam(layer.parameters(), lr=2e-3)
    losses = []
    for _ in range(steps):
        x = torch.randn(tokens, width, dtype=torch.bfloat16, device="cuda")
        with torch.no_grad():
            target = teacher(x)
        loss = (layer(x) - target).float().square().mean()
        optimizer.zero_grad()
        loss.backward()
        optimizer.step()
        losses.append(loss.item())
    x = torch.randn(16, width, dtype=torch.bfloat16, device="cuda")
    with torch.no_grad():
        full = layer(x).float()
    four = layer.decode(x, layer.quantize()).float()
    error = ((four - full).norm() / full.norm()).item()
    return losses, error


if __name__ == "__main__":
    losses, error = main()
    print("loss %.4f -> %.4f over %d steps; 4-bit decode differs by %.1f %% from the layer" % (
        losses[0], losses[-1], len(losses), 100 * error))

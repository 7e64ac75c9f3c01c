"""The expert layer example: its output and gradients against the plain layer
in float64, its 4-bit decode against the dequantized weights, and its run."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def example():
    spec = importlib.util.spec_from_file_location("expert_layer", os.path.join(ROOT, "examples", "expert_layer.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def plain(x, gate_up, down, p, ids):
    """Every token through its experts, one by one, in the tensors' type."""
    out = []
    for t in range(x.shape[0]):
        y = 0
        for j in range(ids.shape[1]):
            h = x[t] @ gate_up[ids[t, j]]
            gate, up = h.chunk(2, -1)
            y = y + p[t, j] * ((torch.nn.functional.silu(gate) * up) @ down[ids[t, j]])
        out.append(y)
    return torch.stack(out)


def test_layer_and_gradients():
    torch.manual_seed(1)
    layer = example().ExpertLayer(64, 72, 4, 2)
    x = torch.randn(50, 64, dtype=torch.bfloat16, device="cuda")
    c = torch.randn(50, 64, dtype=torch.bfloat16, device="cuda")
    p, ids = layer.route(x)
    y = layer(x)
    (y * c).sum().backward()
    gu, dn = (w.detach().double().cpu().requires_grad_() for w in (layer.gate_up, layer.down))
    ref = plain(x.double().cpu(), gu, dn, p.detach().double().cpu(), ids.cpu())
    (ref * c.double().cpu()).sum().backward()
    # bf16 intermediates: about ten roundings of 2^-8 on the way
    for got, want in ((y.detach(), ref.detach()), (layer.gate_up.grad, gu.grad), (layer.down.grad, dn.grad)):
        assert (got.cpu().double() - want).norm() <= 10 * 2.0 ** -8 * want.norm()


def test_decode_uses_the_quantized_weights():
    torch.manual_seed(2)
    layer = example().ExpertLayer(64, 96, 4, 2)
    x = torch.randn(9, 64, dtype=torch.bfloat16, device="cuda")
    quantized = layer.quantize(group=32)
    weights = []
    for q, s, z, group in quantized:
        v = torch.stack((q & 15, q >> 4), -1).flatten(-2).double().cpu()
        K = v.shape[-1]
        spread = lambda t: t.double().cpu().repeat_interleave(group, -1)[..., :K]
        weights.append(((v - spread(z)) * spread(s)).transpose(1, 2))
    p, ids = layer.route(x)
    ref = plain(x.double().cpu(), weights[0], weights[1], p.double().detach().cpu(), ids.cpu())
    got = layer.decode(x, quantized).cpu().double()
    assert (got - ref).norm() <= 10 * 2.0 ** -8 * ref.norm()


def test_example_runs():
    losses, error = example().main(width=64, hidden=64, experts=4, tokens=128, steps=8)
    assert all(torch.isfinite(torch.tensor(losses))) and losses[-1] < losses[0]
    assert error < 0.25

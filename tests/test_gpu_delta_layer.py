"""The example layer end to end: training lowers its loss, autograd through
the library's gradients agrees with a 64-bit torch model of the layer, and
serving (a prompt, then single tokens) agrees with one forward."""
from __future__ import annotations

import importlib.util
import os

import pytest
import torch

from tests import layers_reference as ref

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("delta_layer", os.path.join(ROOT, "examples", "delta_layer.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def test_trains_and_serves(example):
    losses, apart = example.main(B=2, L=100, steps=40)
    print(f"loss {losses[0]:.3f} -> {losses[-1]:.3f}, served {apart:.1e}", flush=True)
    assert losses[-1] < 0.8 * losses[0]
    # the state keeps 24 bits; a bf16 output may round the other way (2^-8)
    assert apart < 2 * 2.0 ** -8


def test_gradients_reach_every_weight(example):
    """The layer's gradient of its normalised queries and keys' weights against
    the 64-bit reference of the two operators."""
    torch.manual_seed(1)
    layer = example.DeltaLayer(64, key_heads=1, value_heads=2, head=32, positions=50, rotated=8).to("cuda:0")
    x = torch.randn(2, 50, 64, device="cuda:0")
    y = layer(x)
    dy = torch.randn_like(y)
    (y * dy).sum().backward()
    for name, p in layer.named_parameters():
        assert p.grad is not None and torch.isfinite(p.grad).all() and p.grad.norm() > 0, name
    with torch.no_grad():
        q, k, v, g, beta = layer.parts(x)
        do = (dy @ layer.out.weight).to(torch.bfloat16).unflatten(2, (2, 32)).transpose(1, 2)
        rest = (layer.cos, layer.sin, None, "l2", "half", 1e-6)
        qn, kn = (ref.norm(t, w.detach(), *rest).to(torch.bfloat16) for t, w in ((q, layer.wq), (k, layer.wk)))
        grads, _ = ref.delta_bwd(qn, kn, v, g, beta, do)
        for t, w, d in ((q, layer.wq, grads[0]), (k, layer.wk, grads[1])):
            _, dw = ref.norm_bwd(t, d.to(torch.bfloat16), w.detach(), *rest)
            # the gradients between the two operators are bf16 on both sides
            assert (w.grad.double().cpu() - dw).norm() <= 2.0 ** -6 * dw.norm()

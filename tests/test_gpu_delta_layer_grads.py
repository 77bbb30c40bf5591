"""The example's autograd functions under the gradients that autograd hands
them: the expanded one of a sum, and a second differentiation."""
from __future__ import annotations

import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
DEV = "cuda:0"


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("delta_layer", os.path.join(ROOT, "examples", "delta_layer.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def functions(example):
    gen = torch.Generator().manual_seed(41)
    r = lambda *s: torch.randn(s, generator=gen).to(DEV)  # noqa: E731
    need = lambda *ts: [t.requires_grad_() for t in ts]  # noqa: E731
    q, k, v = ((r(2, 2, 70, 32) / 6).to(torch.bfloat16) for _ in range(3))
    w, angle = r(32), r(70, 8)
    delta = need(q, k, v, -r(2, 2, 70).abs(), torch.sigmoid(r(2, 2, 70)))
    norm = need(q.detach().clone(), k.detach().clone(), w, w.clone())
    return {"delta": (lambda: example.DeltaRule.apply(*delta), delta),
            "norm": (lambda: example.QkNormRope.apply(*norm, angle.cos(), angle.sin()), norm)}


@pytest.mark.parametrize("name", ["delta", "norm"])
def test_the_gradient_of_a_sum(example, name):
    call, leaves = functions(example)[name]
    outs = call()
    outs = outs if isinstance(outs, tuple) else (outs,)
    want = torch.autograd.grad(outs, leaves, [torch.ones_like(o) for o in outs], retain_graph=True)
    got = torch.autograd.grad(sum(o.sum() for o in outs), leaves)
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("name", ["delta", "norm"])
def test_no_second_gradient(example, name):
    call, leaves = functions(example)[name]
    outs = call()
    first = torch.autograd.grad(sum(o.sum() for o in (outs if isinstance(outs, tuple) else (outs,))), leaves,
                                create_graph=True)
    with pytest.raises(RuntimeError):
        first[0].float().square().sum().backward()

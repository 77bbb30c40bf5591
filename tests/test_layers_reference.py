"""The 64-bit references of the layer operators: gradients against central
differences of the forward, and hand-worked values (CPU)."""
import math

import pytest
import torch

from tests import layers_reference as ref


def _delta_inputs(seed, B=1, Hk=1, Hv=2, L=9, Dk=3, Dv=4):
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=gen, dtype=torch.float64)  # noqa: E731
    return {"q": r(B, Hk, L, Dk), "k": r(B, Hk, L, Dk), "v": r(B, Hv, L, Dv), "g": -r(B, Hv, L).abs(),
            "beta": torch.sigmoid(r(B, Hv, L)), "s0": r(B, Hv, Dk, Dv)}, r(B, Hv, L, Dv), r(B, Hv, Dk, Dv)


def test_delta_by_hand():
    """Two steps of one-dimensional keys: S = 2, then 0.5 * 2 corrected towards 5 by half."""
    q = k = torch.ones(1, 1, 2, 1)
    v = torch.tensor([2.0, 5.0]).reshape(1, 1, 2, 1)
    g = torch.tensor([0.0, math.log(0.5)]).reshape(1, 1, 2)
    beta = torch.tensor([1.0, 0.5]).reshape(1, 1, 2)
    o, s, _ = ref.delta(q, k, v, g, beta, scale=1.0)
    assert torch.allclose(o.flatten(), torch.tensor([2.0, 1.0 + 0.5 * 4.0], dtype=torch.float64))
    assert torch.allclose(s.flatten(), torch.tensor([3.0], dtype=torch.float64))


@pytest.mark.parametrize("seed", [1, 2])
def test_delta_gradients_are_differences(seed):
    x, do, ds = _delta_inputs(seed)
    loss = lambda y: sum((a * b).sum() for a, b in zip(ref.delta(**y)[:2], (do, ds)))  # noqa: E731
    grads, _ = ref.delta_bwd(x["q"], x["k"], x["v"], x["g"], x["beta"], do, x["s0"], ds)
    gen = torch.Generator().manual_seed(seed + 10)
    for name, grad in zip(("q", "k", "v", "g", "beta", "s0"), grads):
        d = torch.randn(x[name].shape, generator=gen, dtype=torch.float64)
        h = 1e-6
        diff = (loss({**x, name: x[name] + h * d}) - loss({**x, name: x[name] - h * d})) / (2 * h)
        assert abs(diff - (grad * d).sum()) < 1e-6 * (1 + abs(diff)), name   # h^2 and the loss's 1e-16 / h


@pytest.mark.parametrize("kind", ["rms", "l2"])
@pytest.mark.parametrize("pairs", ["half", "adjacent"])
def test_norm_gradients_are_differences(kind, pairs):
    gen = torch.Generator().manual_seed(3)
    r = lambda *s: torch.randn(s, generator=gen, dtype=torch.float64)  # noqa: E731
    x, dy, w, angle = r(2, 3, 5, 7), r(2, 3, 5, 7), r(7), r(9, 2)
    pos = torch.tensor([[0, 1, 2, 3, 4], [4, 8, 7, 0, 0]])
    how = (angle.cos(), angle.sin(), pos, kind, pairs, 1e-5)
    dx, dw = ref.norm_bwd(x, dy, w, *how)
    h = 1e-6
    for grad, move in ((dx, lambda s, d: (x + s * d, w)), (dw, lambda s, d: (x, w + s * d))):
        d = torch.randn(grad.shape, generator=gen, dtype=torch.float64)
        up, down = ((ref.norm(*move(s, d), *how) * dy).sum() for s in (h, -h))
        assert abs((up - down) / (2 * h) - (grad * d).sum()) < 1e-6 * (1 + abs((grad * d).sum()))


def test_rotation_by_hand():
    y = torch.tensor([1.0, 2.0, 3.0, 4.0, 5.0], dtype=torch.float64).reshape(1, 1, 1, 5)
    cos, sin = torch.zeros(1, 2, dtype=torch.float64), torch.ones(1, 2, dtype=torch.float64)   # a quarter turn
    assert ref.rotate(y, cos, sin, None, "half").flatten().tolist() == [-3.0, -4.0, 1.0, 2.0, 5.0]
    assert ref.rotate(y, cos, sin, None, "adjacent").flatten().tolist() == [-2.0, 1.0, -4.0, 3.0, 5.0]

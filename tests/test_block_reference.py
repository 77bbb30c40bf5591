"""The 64-bit references of the block's operators on the CPU: gradients against
central differences and autograd, the generator against its published answers."""
import numpy as np
import pytest
import torch

from tests import block_reference as ref

F64 = torch.float64


def test_generator_gives_the_published_answers():
    """Known answers of Philox 4x32-10 published with the generator."""
    F = 0xFFFFFFFF
    for counter, key, want in (
            ((0, 0, 0, 0), (0, 0), (0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8)),
            ((F, F, F, F), (F, F), (0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD)),
            ((0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344), (0xA4093822, 0x299F31D0),
             (0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1))):
        assert tuple(int(x) for x in ref.philox(counter, key)) == want


def test_bits_are_spread_evenly():
    """65536 bins of 2^20 values would hold 16 each; sixteen bins hold 65536 +- 6 sqrt(65536)."""
    b = ref.bits(1 << 10, 1 << 10, 12345, 6)
    counts = np.bincount(b.flatten().numpy() >> 12, minlength=16)
    assert (abs(counts - 65536) < 6 * 256).all()


@pytest.mark.parametrize("gates", ["steps", "heads", "none"])
def test_linear_gradients_against_autograd(gates):
    gen = torch.Generator().manual_seed(1)
    r = lambda *s: torch.randn(s, generator=gen, dtype=F64)  # noqa: E731
    q, k, v, do, s0, ds = r(2, 2, 9, 5), r(2, 2, 9, 5), r(2, 4, 9, 3), r(2, 4, 9, 3), r(2, 4, 5, 3), r(2, 4, 5, 3)
    g = {"steps": -r(2, 4, 9).abs(), "heads": -r(4).abs(), "none": None}[gates]
    leaves = [t for t in (q, k, v, s0, g) if t is not None]
    for t in leaves:
        t.requires_grad_()
    o, s, _ = ref.linear(q, k, v, g, s0)
    want = torch.autograd.grad((o * do).sum() + (s * ds).sum(), leaves)
    with torch.no_grad():
        (dq, dk, dv, dg, ds0), size = ref.linear_bwd(q, k, v, g, do, s0, ds)
    got = [dq, dk, dv, ds0] + ([] if g is None else [dg if g.dim() == 3 else dg.sum((0, 2))])
    for a, b in zip(got, want):
        assert torch.allclose(a, b, rtol=1e-10, atol=1e-12)
    assert (dg.abs() <= size * (1 + 1e-9)).all()


@pytest.mark.parametrize("p", [0.0, 0.3])
def test_layer_norm_gradients_against_autograd(p):
    gen = torch.Generator().manual_seed(2)
    r = lambda *s: torch.randn(s, generator=gen, dtype=F64)  # noqa: E731
    x, res, w, b, dy, dh = r(3, 4, 11), r(3, 4, 11), r(11), r(11), r(3, 4, 11), r(3, 4, 11)
    for t in (x, res, w, b):
        t.requires_grad_()
    y, h = ref.layer_norm(x, w, b, res, p=p, seed=5, offset=9)
    want = torch.autograd.grad((y * dy).sum() + (h * dh).sum(), (res, x, w, b))
    with torch.no_grad():
        got = ref.layer_norm_bwd(h, dy, w, dh, p=p, seed=5, offset=9)
    for a, c in zip(got, want):
        assert torch.allclose(a, c, rtol=1e-10, atol=1e-12)

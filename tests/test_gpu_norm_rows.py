"""The layer norm and dropout of very many rows: what the first and the last rows
hold, where an index that wraps would show.  Bounds as in
tests/test_gpu_layer_norm.py."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import structured_sparse_state_amd as pk
from tests import block_reference as ref
from tests.test_gpu_layer_norm import DEV, HALF, near, rms, say

pytestmark = pytest.mark.gpu

SEED, OFFSET = 0x1234567890ABCDEF, (5 << 32) + 7


def kept(rows, D, p):
    """Which values of the given rows dropout keeps."""
    units = (D + 7) // 8
    unit, row = np.meshgrid(np.arange(units), np.asarray(rows))
    off = [np.full_like(unit, OFFSET >> s & 0xFFFFFFFF) for s in (0, 32)]
    words = ref.philox([unit, row, *off], [SEED & 0xFFFFFFFF, SEED >> 32])
    halves = np.stack([words & np.uint32(0xFFFF), words >> np.uint32(16)], 1).transpose(2, 3, 0, 1)
    return torch.from_numpy(halves.reshape(len(rows), 8 * units)[:, :D].astype(np.int64)) >= ref.threshold(p)


def test_the_rows_own_bits():
    """(the helper above against the reference's whole tensor)"""
    assert torch.equal(kept(range(3, 9), 20, 0.4), ref.bits(9, 20, SEED, OFFSET)[3:] >= ref.threshold(0.4))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,D", [((1 << 24) + 5, 4), ((1 << 22) + 1, 24), ((1 << 25) + 77, 9)])
def test_first_and_last_rows(dtype, rows, D):
    say(f"[case] {rows} rows of {D}")
    p, scale = 0.3, 65536 / (65536 - ref.threshold(0.3))
    gen = torch.Generator(device=DEV).manual_seed(1)
    x, r, dy = (torch.randn(rows, D, generator=gen, device=DEV).to(dtype) for _ in range(3))
    how = dict(p=p, seed=SEED, offset=OFFSET)
    y, h = pk.layer_norm(x, residual=r, **how)
    dr, dx, _, _ = pk.layer_norm_bwd(h, dy, dh=r, **how)
    d = pk.dropout(x, residual=r, **how)
    torch.cuda.synchronize()
    assert torch.equal(d, h)
    for at in (0, rows // 2, rows - 40):
        cut = slice(at, at + 40)
        keep = kept(range(at, at + 40), D, p)
        want_h = torch.where(keep, x[cut].double().cpu() * scale, 0.0) + r[cut].double().cpu()
        assert ((h[cut].double().cpu() - want_h).abs() <=
                HALF[dtype] * want_h.abs() + 2.0 ** -23 * (want_h.abs() + r[cut].double().cpu().abs())).all()
        spread = lambda t: (t - t.mean(-1, keepdim=True)).square().mean(-1, keepdim=True).add(1e-5).sqrt()  # noqa: E731
        c = want_h - want_h.mean(-1, keepdim=True)
        ratio = 1 + rms(want_h) / spread(want_h)
        near(y[cut], c / spread(want_h), ratio * ratio, "y")
        hd, dyd = h[cut].double().cpu(), dy[cut].double().cpu()
        want, _, _, _ = ref.layer_norm_bwd(hd, dyd, dh=r[cut])
        ratio = 1 + rms(hd) / spread(hd)
        size = ratio * ratio * rms(dyd) / spread(hd) * (1 + (hd - hd.mean(-1, keepdim=True)).abs() / spread(hd)) + \
            r[cut].double().cpu().abs()
        near(dr[cut], want, size, "dr")
        near(dx[cut], torch.where(keep, want * scale, 0.0), size * scale, "dx")


def test_more_than_2_to_the_32_units():
    """2^21 rows and some of 2048 units, in place (69 GB)."""
    rows, D = (1 << 21) + 3, 16384
    say("[case] 2^32 units")
    x = torch.ones(rows, D, dtype=torch.bfloat16, device=DEV)
    pk.dropout(x, 0.5, SEED, OFFSET, out=x)
    torch.cuda.synchronize()
    for at in (0, 1 << 20, rows - 4):
        assert torch.equal(x[at:at + 4].cpu() != 0, kept(range(at, at + 4), D, 0.5))
        assert ((x[at:at + 4] == 0) | (x[at:at + 4] == 2)).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("D", [5, 1000, 16384])
def test_rows_of_large_values(dtype, D):
    """Values of up to 1e17, whose squares fp32 still holds the sum of."""
    gen = torch.Generator().manual_seed(3)
    x = (1e17 * (2 * torch.rand(7, D, generator=gen) - 1)).to(DEV, dtype)
    x[0, 0], x[0, 1:] = 1e17, -1e17
    dy = torch.randn(7, D, generator=gen).to(DEV, dtype)
    say(f"[case] values of 1e17, D={D}")
    y, _ = pk.layer_norm(x)
    dr, _, _, _ = pk.layer_norm_bwd(x, dy)
    torch.cuda.synchronize()
    want, h = ref.layer_norm(x)
    spread = (h - h.mean(-1, keepdim=True)).square().mean(-1, keepdim=True).sqrt()
    ratio = 1 + rms(h) / spread
    near(y, want, ratio * ratio, "y")
    want = ref.layer_norm_bwd(x, dy)[0]
    size = ratio * ratio * rms(dy.double().cpu()) / spread * (1 + (h - h.mean(-1, keepdim=True)).abs() / spread)
    near(dr, want, size, "dr")

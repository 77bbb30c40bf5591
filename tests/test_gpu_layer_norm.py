"""The layer norm with residual and dropout, its gradients, and dropout alone on
the GPU against the 64-bit reference.

Tolerances, fixed beforehand.  fp32: a row's sums are of at most 32 values in a
lane, then by halves over at most 1024 lanes, 32 + 10 roundings of 2^-24 of
partial sums no larger than the sum of sizes; with the few operations of a value
the error is below 64 * 2^-24 = 4e-6 of the row's size: y and the gradients are
held to 4e-6 of (|value| + the row's root mean square), times the ratio of
|h| to its spread, which cancels bits of c = h - mean.  dw and db sum rows one
after another in a lane and then by workgroups: 4e-6 + rows * 2^-24 of the sum
of sizes.  A bf16 result is that rounded once: half a step is at most 2^-8 of the value (2^-9 of
its binade's upper end).  h = residual + x * scale has two roundings: 2^-23."""
from __future__ import annotations

import pytest
import torch

import structured_sparse_state_amd as pk
from tests import block_reference as ref

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
TOL = 4e-6
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def say(msg):
    print(msg, flush=True)


def near(got, want, size, name):
    """Every value within one rounding of itself and TOL of its row's size."""
    assert got.shape == want.shape and torch.isfinite(got).all(), name
    e = (got.double().cpu() - want).abs()
    bound = HALF[got.dtype] * want.abs() + TOL * (want.abs() + size)
    worst = float((e / bound.clamp_min(1e-300)).max()) if e.numel() else 0.0
    say(f"  {name} {worst:.2f} of its bound")
    assert (e <= bound).all(), name


def rms(t):
    return t.square().mean(-1, keepdim=True).sqrt()


def inputs(seed, shape, dtype, residual=True, affine=True, offset=0.0):
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=gen)  # noqa: E731
    x = {n: (r(*shape) * s + m).to(dtype).to(DEV) for n, s, m in
         (("x", 1.0, 0.0), ("residual", 1.5, offset), ("dy", 1.0, 0.0), ("dh", 1.0, 0.0))}
    if not residual:
        x["residual"] = x["dh"] = None
    D = shape[-1]
    x["w"], x["b"] = ((1 + 0.3 * r(D)).to(DEV), r(D).to(DEV)) if affine else (None, None)
    return x


def check(x, label, p=0.0, seed=0, offset=0, eps=1e-5):
    say(f"[case] {label} p={p}")
    how = dict(eps=eps, p=p, seed=seed, offset=offset)
    y, h = pk.layer_norm(x["x"], x["w"], x["b"], residual=x["residual"], **how)
    torch.cuda.synchronize()
    want_y, want_h = ref.layer_norm(x["x"], x["w"], x["b"], x["residual"], **how)
    e = (h.double().cpu() - want_h).abs()
    terms = want_h.abs() + (x["residual"].double().cpu().abs() if x["residual"] is not None else 0)
    assert (e <= HALF[h.dtype] * want_h.abs() + 2.0 ** -23 * terms).all()
    spread = (want_h - want_h.mean(-1, keepdim=True)).square().mean(-1, keepdim=True).add(eps).sqrt()
    cancels = (1 + rms(want_h) / spread) * (x["w"].double().cpu().abs().max() if x["w"] is not None else 1)
    near(y, want_y, cancels * (1 + rms(want_h) / spread), "y")

    affine = x["w"] is not None
    dr, dx, dw, db = pk.layer_norm_bwd(h, x["dy"], x["w"], dh=x["dh"], want_db=affine, **how)
    torch.cuda.synchronize()
    want = ref.layer_norm_bwd(h, x["dy"], x["w"], x["dh"], **how)
    hd, dyd = h.double().cpu(), x["dy"].double().cpu()
    spread = (hd - hd.mean(-1, keepdim=True)).square().mean(-1, keepdim=True).add(eps).sqrt()
    ratio = 1 + rms(hd) / spread
    e = dyd * (x["w"].double().cpu() if affine else 1)
    size = ratio * ratio * rms(e) / spread * (1 + (hd - hd.mean(-1, keepdim=True)).abs() / spread) + \
        (x["dh"].double().cpu().abs() if x["dh"] is not None else 0)
    near(dr, want[0], size, "dr")
    near(dx, want[1], size * 65536 / (65536 - ref.threshold(p)), "dx")
    assert (dx is dr) == (ref.threshold(p) == 0)
    if affine:
        rows = hd[..., 0].numel()
        flat = lambda t: t.reshape(-1, t.shape[-1]).abs().sum(0)  # noqa: E731
        unit = (hd - hd.mean(-1, keepdim=True)) / spread
        for name, a, b, terms in (("dw", dw, want[2], flat(dyd * (unit.abs() + ratio)) * float(ratio.max())),
                                  ("db", db, want[3], flat(dyd))):
            assert a.dtype == torch.float32 and torch.isfinite(a).all()
            assert ((a.double().cpu() - b).abs() <= (TOL + rows * 2.0 ** -24) * terms).all(), name
    else:
        assert dw is None and db is None
    return y, h, dr, dx, dw, db


WIDTHS = [1, 2, 7, 8, 9, 64, 127, 128, 129, 136, 500, 512, 520, 1000, 1024, 1025, 2048, 2049, 4096, 4100, 8192, 8200,
          16384]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("D", WIDTHS)
def test_widths(dtype, D):
    check(inputs(D, (2, 3, D), TYPES[dtype]), f"D={D}", p=0.3, seed=D, offset=1 << 40)
    check(inputs(D, (5, D), TYPES[dtype], residual=False, affine=False), f"D={D} plain")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,D", [(1, 2048), (2500, 72), (4099, 256), (9001, 40), (3001, 1000), (700, 4096), (40, 16000)])
def test_row_counts(dtype, rows, D):
    check(inputs(rows, (rows, D), TYPES[dtype]), f"rows={rows} D={D}", p=0.1, seed=3)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("offset", [100.0, 3000.0])
def test_a_mean_far_from_zero(dtype, offset):
    check(inputs(5, (8, 1024), TYPES[dtype], offset=offset), f"mean {offset}")


def test_rows_of_one_value():
    """Rows whose variance is zero, and rows of zeros."""
    for value in (0.0, 2.5):
        x = torch.full((3, 200), value, device=DEV)
        w, b = torch.randn(200, device=DEV), torch.randn(200, device=DEV)
        y, h = pk.layer_norm(x, w, b)
        torch.cuda.synchronize()
        assert h is x and torch.equal(y, b.expand(3, 200))


@pytest.mark.parametrize("dtype", TYPES)
def test_strides(dtype):
    """Rows apart, in another order, and off every 16-byte boundary."""
    t = TYPES[dtype]
    x = inputs(6, (2, 3, 5, 72), t)
    want = check(x, "contiguous", p=0.4, seed=1 << 63, offset=3)
    wide = lambda v, o: torch.full((2, 5, 3, 80), 7.0, dtype=t, device=DEV)[..., o:o + 72].permute(0, 2, 1, 3).copy_(v)  # noqa: E731
    for o in (0, 1, 8):
        y = {n: wide(v, o) if v is not None and v.dim() > 1 else v for n, v in x.items()}
        out, h = wide(x["x"], o), wide(x["x"], o)
        how = dict(p=0.4, seed=1 << 63, offset=3)
        pk.layer_norm(y["x"], y["w"], y["b"], residual=y["residual"], out=out, h=h, **how)
        grads = (wide(x["x"], o), wide(x["x"], o))
        got = pk.layer_norm_bwd(h, y["dy"], y["w"], dh=y["dh"], want_db=True, out=grads, **how)
        drop, dropped = pk.dropout(y["x"], 0.4, 1 << 63, 3, residual=y["residual"]), wide(x["x"], o)
        pk.dropout(y["x"], 0.4, 1 << 63, 3, residual=y["residual"], out=dropped)
        torch.cuda.synchronize()
        for a, b in zip((out, h, *got, drop, dropped), (*want, want[1], want[1])):
            assert torch.equal(a, b)
        for base in (out, h, *grads, dropped):      # nothing beside the rows
            whole = base.permute(0, 2, 1, 3)
            whole = whole.as_strided((2, 5, 3, 80), whole.stride(), whole.storage_offset() - o)
            assert (whole[..., :o] == 7.0).all() and (whole[..., o + 72:] == 7.0).all()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("p", [0.0, 2.0 ** -18, 2.0 ** -17, 0.1, 0.5, 0.999, 1 - 2.0 ** -18])
@pytest.mark.parametrize("shape,residual", [((3, 7, 40), False), ((1001, 331), True), ((5,), True), ((2, 3, 4, 8), False)])
def test_dropout(dtype, p, shape, residual):
    """Masks bit for bit, kept values within two roundings."""
    x = inputs(9, shape, TYPES[dtype], residual=residual)
    say(f"[case] dropout {shape} p={p}")
    seed, offset = 0x9E3779B97F4A7C15, (1 << 64) - 5
    y = pk.dropout(x["x"], p, seed, offset, residual=x["residual"])
    torch.cuda.synchronize()
    want = ref.dropped(x["x"], p, seed, offset)
    dropped = want == 0
    if residual:
        want = want + x["residual"].double().cpu()
    bound = HALF[y.dtype] * want.abs() + 2.0 ** -23 * (want.abs() + (x["residual"].double().cpu().abs() if residual else 0))
    assert ((y.double().cpu() - want).abs() <= bound).all()
    if not residual:
        assert torch.equal(y.cpu() == 0, dropped)
    if p < 2.0 ** -17:
        assert torch.equal(y, x["x"] if not residual else (x["x"].float() + x["residual"].float()).to(y.dtype))


def test_the_generators_first_block():
    """Counter and key of zero: the published first answer, half by half."""
    halves = [w >> s & 0xFFFF for w in (0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8) for s in (0, 16)]
    x = torch.ones(1, 8, device=DEV)
    for n, bits in enumerate(halves):
        for T, kept in ((bits, True), (bits + 1, False)):
            y = pk.dropout(x, T / 65536, 0)
            assert bool(y[0, n] != 0) is kept


def test_values_that_are_dropped_do_not_matter():
    """NaN and infinities in dropped places leave no trace."""
    x = inputs(10, (40, 300), torch.float32)
    how = dict(p=0.5, seed=4)
    mask = ref.bits(40, 300, 4, 0).view(40, 300) < ref.threshold(0.5)
    bad = torch.where(mask.to(DEV), torch.tensor([float("nan"), float("inf"), -float("inf")], device=DEV).repeat(100), x["x"])
    for a, b in zip(pk.layer_norm(bad, residual=x["residual"], **how), pk.layer_norm(x["x"], residual=x["residual"], **how)):
        assert torch.equal(a, b)
    assert torch.equal(pk.dropout(bad, 0.5, 4), pk.dropout(x["x"], 0.5, 4))


def test_what_is_not_finite_stays_in_its_row():
    x = inputs(11, (7, 5, 200), torch.bfloat16)
    y, h = pk.layer_norm(x["x"], x["w"], x["b"], residual=x["residual"])
    bad = x["x"].clone()
    bad[3, 2, 17] = float("inf")
    y2, h2 = pk.layer_norm(bad, x["w"], x["b"], residual=x["residual"])
    rest = torch.ones(7, 5, dtype=torch.bool, device=DEV)
    rest[3, 2] = False
    assert torch.equal(y2[rest], y[rest]) and torch.equal(h2[rest], h[rest]) and not torch.isfinite(y2[3, 2]).any()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("D", [72, 1000, 2048, 4096])
def test_in_place(dtype, D):
    """Results over inputs, as the documentation allows."""
    x = inputs(12, (300, D), TYPES[dtype])
    how = dict(p=0.2, seed=8)
    y, h = pk.layer_norm(x["x"], x["w"], x["b"], residual=x["residual"], **how)
    dr, dx, dw, db = pk.layer_norm_bwd(h, x["dy"], x["w"], dh=x["dh"], want_db=True, **how)
    d = pk.dropout(x["x"], 0.2, 8, residual=x["residual"])
    a, r = x["x"].clone(), x["residual"].clone()
    pk.layer_norm(a, x["w"], x["b"], residual=r, out=a, h=r, **how)
    dy, dh = x["dy"].clone(), x["dh"].clone()
    _, _, dw2, db2 = pk.layer_norm_bwd(h, dy, x["w"], dh=dh, want_db=True, out=(dh, dy), **how)
    b, e = x["x"].clone(), x["residual"].clone()
    pk.dropout(b, 0.2, 8, residual=e, out=b)
    pk.dropout(x["x"], 0.2, 8, residual=e, out=e)
    torch.cuda.synchronize()
    for got, want in ((a, y), (r, h), (dh, dr), (dy, dx), (dw2, dw), (db2, db), (b, d), (e, d)):
        assert torch.equal(got, want)


def test_empty_shapes():
    for shape in ((0, 8), (3, 0, 8), (0, 2, 5, 8)):
        x = torch.zeros(shape, device=DEV)
        w = torch.ones(8, device=DEV)
        y, h = pk.layer_norm(x, w, w, residual=x, p=0.5, seed=1)
        dr, dx, dw, db = pk.layer_norm_bwd(x, x, w, want_db=True, p=0.5, seed=1)
        assert y.shape == h.shape == dr.shape == dx.shape == x.shape == pk.dropout(x, 0.5, 1).shape
        assert torch.equal(dw, torch.zeros_like(w)) and torch.equal(db, torch.zeros_like(w))


def test_results_are_reproducible_whatever_the_workspace_holds():
    x = inputs(13, (2000, 520), torch.bfloat16)
    ws = pk.pdssm_layer_norm_bwd_workspace_bytes(1, 1, 2000, 520)
    results = [pk.layer_norm_bwd(x["x"], x["dy"], x["w"], want_db=True,
                                 workspace=torch.full((ws,), fill, dtype=torch.uint8, device=DEV)) for fill in (0, 255)]
    for a, b in zip(*results):
        assert torch.equal(a, b)


def test_a_seed_in_device_memory():
    x = inputs(14, (64, 256), torch.bfloat16)
    rng = torch.tensor([5, 9], dtype=torch.int64, device=DEV)
    for a, b in zip(pk.layer_norm(x["x"], p=0.3, seed=rng), pk.layer_norm(x["x"], p=0.3, seed=5, offset=9)):
        assert torch.equal(a, b)
    assert torch.equal(pk.dropout(x["x"], 0.3, rng), pk.dropout(x["x"], 0.3, 5, 9))
    for a, b in zip(pk.layer_norm_bwd(x["x"], x["dy"], p=0.3, seed=rng)[:2], pk.layer_norm_bwd(x["x"], x["dy"], p=0.3, seed=5, offset=9)):
        assert torch.equal(a, b)


def test_graph_replays_draw_anew():
    """Forward, backward and dropout captured; the seed in device memory changes between replays."""
    x = inputs(15, (700, 264), torch.bfloat16)
    rng = torch.tensor([5, 0], dtype=torch.int64, device=DEV)
    ws = torch.empty(pk.pdssm_layer_norm_bwd_workspace_bytes(1, 1, 700, 264), dtype=torch.uint8, device=DEV)

    def call(seed, offset=0):
        y, h = pk.layer_norm(x["x"], x["w"], x["b"], residual=x["residual"], p=0.3, seed=seed, offset=offset)
        grads = pk.layer_norm_bwd(h, x["dy"], x["w"], dh=x["dh"], want_db=True, p=0.3, seed=seed, offset=offset, workspace=ws)
        return [y, h, *grads, pk.dropout(x["x"], 0.3, seed, offset)]

    call(rng)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = call(rng)
    for n in range(3):
        rng[1] = n
        x["x"].copy_(torch.randn(700, 264, device=DEV))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, call(5, n)):
            assert torch.equal(a, b)


def test_gradient_against_differences():
    x = inputs(16, (4, 40), torch.float32)
    how = dict(p=0.25, seed=77, offset=1)
    y, h = pk.layer_norm(x["x"], x["w"], x["b"], residual=x["residual"], **how)
    grads = dict(zip(("residual", "x", "w", "b"), pk.layer_norm_bwd(h, x["dy"], x["w"], dh=x["dh"], want_db=True, **how)))
    z = {n: t.double().cpu() for n, t in x.items()}

    def loss(z):
        y, h = ref.layer_norm(z["x"], z["w"], z["b"], z["residual"], **how)
        return (y * z["dy"]).sum() + (h * z["dh"]).sum()

    gen = torch.Generator().manual_seed(1)
    for name, grad in grads.items():
        d = torch.randn(z[name].shape, generator=gen, dtype=torch.float64)
        diff = (loss({**z, name: z[name] + 1e-6 * d}) - loss({**z, name: z[name] - 1e-6 * d})) / 2e-6
        along = (grad.double().cpu() * d).sum()
        assert abs(diff - along) <= 1e-4 * float(grad.double().norm()) * d.numel() ** 0.5, name


def test_more_rows_than_a_grid_dimension():
    """2^24 rows and some of few values."""
    rows = (1 << 24) + 5
    x = torch.randn(rows, 4, device=DEV)
    say("[case] 2^24 rows")
    y, _ = pk.layer_norm(x)
    dr, _, _, _ = pk.layer_norm_bwd(x, y)
    d = pk.dropout(x, 0.5, 3)
    torch.cuda.synchronize()
    for at in (0, rows - 40):
        want, _ = ref.layer_norm(x[at:at + 40])
        assert ((y[at:at + 40].double().cpu() - want).abs() <= 1e-3).all()
    assert torch.isfinite(dr).all()
    bits = torch.stack([ref.bits(1, 4, 3, 0)[0] for _ in range(1)])
    assert torch.equal((d[:1] != 0).cpu(), bits >= 32768)

"""The query/key norm with rotation on the GPU against the 64-bit reference.

Tolerances, fixed beforehand: fp32 results are a dozen fp32 operations and a
sum of at most 256 squares: 32 * 2^-24 = 2e-6 of the norm, for dx, which is a
difference, of its terms' norm (a row of one value has none but rounding left);
bf16 results add their rounding, at most 2^-8 (8 bits, to nearest).  Weight gradients are fp32 sums over all rows,
in tree order: 1e-5 of the norm of the sum of the terms' sizes over its root."""
from __future__ import annotations

import sys

import pytest
import torch

import structured_sparse_state_amd as pk
from tests import layers_reference as ref

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
TOL = {"bf16": 2.0 ** -8 + 1e-5, "f32": 2e-6}


def off(got, want, terms=None):
    got = got.double().cpu()
    assert got.shape == want.shape and torch.isfinite(got).all()
    n = want.norm() if terms is None else terms.norm()
    return float((got - want).norm() / n) if n > 0 else float(got.norm())


def inputs(seed, B, Hq, Hk, L, D, R, dtype, weights=True, pos=True, order="packed", table=None):
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=gen)  # noqa: E731
    table = table or 2 * L + 3
    x = r(B, L, Hq + Hk, D).to(dtype)
    if order == "packed":       # slices of one projection
        x = x.to(DEV)
        q, k = x[:, :, :Hq].transpose(1, 2), x[:, :, Hq:].transpose(1, 2)
    elif order == "head":
        q, k = (t.transpose(1, 2).contiguous().to(DEV) for t in (x[:, :, :Hq], x[:, :, Hq:]))
    else:                       # rows off every 16-byte boundary
        base = torch.full((B, Hq + Hk, L + 1, D + 3), float("nan"), dtype=dtype, device=DEV)
        base[:, :, 1:, 1:D + 1] = x.transpose(1, 2).to(DEV)
        q, k = base[:, :Hq, 1:, 1:D + 1], base[:, Hq:, 1:, 1:D + 1]
    angle = r(table, R // 2)
    c = {"q": q, "k": k, "wq": r(D).to(DEV) if weights else None, "wk": r(D).to(DEV) if weights else None,
         "cos": angle.cos().to(DEV) if R else None, "sin": angle.sin().to(DEV) if R else None,
         "pos": torch.randint(0, table, (B, L), generator=gen).int().to(DEV) if pos and R else None}
    return c, r(B, Hq, L, D).to(dtype).to(DEV), r(B, Hk, L, D).to(dtype).to(DEV)


def check(c, dq_out, dk_out, kind, pairs, dtype, eps=1e-6):
    how = dict(kind=kind, pairs=pairs, eps=eps)
    got = pk.qk_norm_rope(**c, **how)
    grads = pk.qk_norm_rope_bwd(c["q"], c["k"], dq_out, dk_out, c["wq"], c["wk"], c["cos"], c["sin"], c["pos"], **how)
    torch.cuda.synchronize()
    rest = (c["cos"], c["sin"], c["pos"], kind, pairs, eps)
    for n, (name, dy) in enumerate((("q", dq_out), ("k", dk_out))):
        x, w = c[name], c["w" + name]
        want = ref.norm(x, w, *rest)
        dx, dw = ref.norm_bwd(x, dy, w, *rest)
        r = 1 / torch.sqrt(x.double().cpu().square().sum(-1, keepdim=True) / (x.shape[-1] if kind == "rms" else 1) + eps)
        e = ref.rotate(dy.double().cpu(), c["cos"], c["sin"], c["pos"], pairs, True)
        errors = [off(got[n], want), off(grads[n], dx, r * e * (1 if w is None else w.double().cpu()))]
        print(f"  {name}: {errors[0]:.2e}, d{name} {errors[1]:.2e}", flush=True)
        assert max(errors) <= TOL[dtype], name
        if w is None:
            assert grads[2 + n] is None
        else:
            terms = (ref.rotate(dy.double().cpu(), c["cos"], c["sin"], c["pos"], pairs, True)
                     * ref.norm(x, None, None, None, None, kind, pairs, eps)).square().sum((0, 1, 2)).sqrt()
            assert float((grads[2 + n].double().cpu() - dw).norm()) <= 1e-5 * float(terms.norm() + dw.norm())
    return got, grads


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("kind", ["rms", "l2"])
@pytest.mark.parametrize("pairs", ["half", "adjacent"])
@pytest.mark.parametrize("D,R", [(1, 0), (2, 2), (7, 4), (8, 8), (64, 64), (64, 0), (72, 20), (72, 16), (100, 48), (128, 128),
                                 (128, 64), (128, 30), (129, 128), (200, 160), (256, 256), (255, 254)])
def test_head_sizes(dtype, kind, pairs, D, R):
    print(f"[case] D={D} R={R} {kind} {pairs} {dtype}", flush=True)
    sys.stdout.flush()
    c, dq, dk = inputs(D + R, 2, 3, 1, 5, D, R, TYPES[dtype])
    check(c, dq, dk, kind, pairs, dtype)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("B,Hq,Hk,L", [(1, 1, 1, 1), (5, 16, 4, 1), (1, 9, 5, 130), (2, 32, 8, 300), (3, 4, 4, 1500), (1, 70, 6, 900)])
def test_shapes(dtype, B, Hq, Hk, L):
    """Few and many rows (a lane takes one head or four), heads in incomplete fours."""
    print(f"[case] B={B} Hq={Hq} Hk={Hk} L={L} {dtype}", flush=True)
    c, dq, dk = inputs(L, B, Hq, Hk, L, 64, 32, TYPES[dtype])
    check(c, dq, dk, "rms", "half", dtype)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("order", ["head", "apart"])
@pytest.mark.parametrize("pairs", ["half", "adjacent"])
def test_memory_orders(dtype, order, pairs):
    c, dq, dk = inputs(3, 2, 4, 2, 50, 64, 32, TYPES[dtype], order=order)
    got, _ = check(c, dq, dk, "rms", pairs, dtype)
    if order == "head":
        assert got[0].is_contiguous()


def test_order_of_results_and_given_places():
    c, dq, dk = inputs(4, 2, 4, 2, 20, 64, 64, torch.bfloat16)
    q, k = pk.qk_norm_rope(**c)
    assert q.stride(3) == 1 and q.stride(1) < q.stride(2)       # token by token, as the projection
    base = torch.full((2, 5, 21, 67), 3.0, dtype=torch.bfloat16, device=DEV)
    out = base[:, :4, 1:, 2:66]
    pk.qk_norm_rope(**c, out=(out, k))
    assert torch.equal(out, q)
    base[:, :4, 1:, 2:66] = 3.0
    assert (base == 3.0).all()
    # in place, both directions
    want = pk.qk_norm_rope_bwd(c["q"], c["k"], dq, dk, c["wq"], c["wk"], c["cos"], c["sin"], c["pos"])
    got = pk.qk_norm_rope_bwd(c["q"], c["k"], dq, dk, c["wq"], c["wk"], c["cos"], c["sin"], c["pos"], out=(dq, dk))
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    pk.qk_norm_rope(**c, out=(c["q"], c["k"]))
    assert torch.equal(c["q"], q) and torch.equal(c["k"], k)


def test_positions():
    """No positions: the place in the sequence; positions outside the table: its ends."""
    c, dq, dk = inputs(5, 2, 2, 1, 12, 64, 64, torch.float32, pos=False, table=12)
    check(c, dq, dk, "rms", "half", "f32")
    c["pos"] = torch.tensor([[-5, 0, 3, 11, 12, 100, -2147483648, 2147483647, 1, 2, 3, 4]] * 2, dtype=torch.int32, device=DEV)
    check(c, dq, dk, "rms", "adjacent", "f32")
    short = {**c, "cos": c["cos"][:5].contiguous(), "sin": c["sin"][:5].contiguous(), "pos": None}   # a table shorter than the sequence
    check(short, dq, dk, "l2", "half", "f32")


@pytest.mark.parametrize("dtype", TYPES)
def test_values_at_the_edges(dtype):
    """Rows of zeros, of one value, very large and very small ones."""
    c, dq, dk = inputs(6, 1, 4, 4, 8, 64, 64, TYPES[dtype])
    c["q"][:, 0] = 0
    c["q"][:, 1] *= 1e15
    c["q"][:, 2] *= 1e-15
    c["k"][:, 0, :, 1:] = 0
    for kind in ("rms", "l2"):
        check(c, dq, dk, kind, "half", dtype, eps=1e-5)
    # a NaN stays in its row
    want = pk.qk_norm_rope(**c)[0]
    c["q"][0, 3, 4, 7] = float("nan")
    got = pk.qk_norm_rope(**c)[0]
    assert torch.isnan(got[0, 3, 4]).all()
    got[0, 3, 4] = want[0, 3, 4]
    assert torch.equal(got, want)


@pytest.mark.parametrize("B,Hq,Hk,L", [(0, 2, 1, 4), (2, 0, 3, 4), (2, 3, 0, 4), (2, 2, 1, 0), (1, 0, 0, 3)])
def test_empty_shapes(B, Hq, Hk, L):
    c, dq, dk = inputs(7, B, Hq, Hk, L, 64, 32, torch.bfloat16, table=9)
    got, grads = check(c, dq, dk, "rms", "half", "bf16")
    if B * L * Hq == 0:
        assert (grads[2] == 0).all()


def test_reproducible_on_any_stream_and_in_a_graph():
    c, dq, dk = inputs(8, 2, 8, 2, 700, 128, 128, torch.bfloat16)
    args = (c["q"], c["k"], dq, dk, c["wq"], c["wk"], c["cos"], c["sin"], c["pos"])
    want = [*pk.qk_norm_rope(**c), *pk.qk_norm_rope_bwd(*args)]
    torch.cuda.synchronize()
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        got = [*pk.qk_norm_rope(**c), *pk.qk_norm_rope_bwd(*args)]
    stream.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    ws = torch.empty(pk.pdssm_qk_norm_rope_bwd_workspace_bytes(2, 8, 2, 700, 128), dtype=torch.uint8, device=DEV)
    with torch.cuda.graph(graph):
        held = [*pk.qk_norm_rope(**c), *pk.qk_norm_rope_bwd(*args, workspace=ws)]
    for n in range(3):
        c["q"].copy_(torch.randn(c["q"].shape, device=DEV))
        ws.fill_(255)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        eager = [*pk.qk_norm_rope(**c), *pk.qk_norm_rope_bwd(*args)]
        torch.cuda.synchronize()
        for a, b in zip(held, eager):
            assert torch.equal(a, b)


def test_gradient_against_differences():
    c, dq, dk = inputs(9, 1, 2, 1, 6, 24, 8, torch.float32)
    how = (c["cos"], c["sin"], c["pos"], "rms", "half", 1e-6)
    got = pk.qk_norm_rope_bwd(c["q"], c["k"], dq, dk, c["wq"], c["wk"], c["cos"], c["sin"], c["pos"])
    x, w, dy = c["q"].double().cpu(), c["wq"].double().cpu(), dq.double().cpu()
    loss = lambda x, w: (ref.norm(x, w, *how) * dy).sum()  # noqa: E731
    gen = torch.Generator().manual_seed(2)
    h = 1e-6
    d, e = (torch.randn(t.shape, generator=gen, dtype=torch.float64) for t in (x, w))
    for grad, diff, along in ((got[0], loss(x + h * d, w) - loss(x - h * d, w), d),
                              (got[2], loss(x, w + h * e) - loss(x, w - h * e), e)):
        exact = (grad.double().cpu() * along).sum()
        assert abs(diff / (2 * h) - exact) <= 1e-5 * float(grad.double().norm()) * along.numel() ** 0.5

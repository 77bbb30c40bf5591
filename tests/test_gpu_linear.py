"""Linear attention with decays on the GPU (forward, gradients, single step)
against the 64-bit step-by-step reference.

Tolerances, fixed beforehand.  Every product is held to 2^-24 and summed in fp32
over at most Dk + 64 = 192 terms in a chunk; the partial sums are of the size of
the result, so its error is at most 192 * 2^-24 = 1.2e-5 of its norm, and one
rounding of 2^-24 more for each chunk that the state passes: 2e-5 up to 130
chunks.  A bf16 result is that rounded once, half a step or 2^-9 of 1 to 2, at
most 2^-8 / 2 * 2 = 2^-8 of a value: 2^-8 + 2e-5.  dg is <S, dS>, both known to
2e-5 of their norms, as a sum over pairs of steps that may cancel among
themselves by the root of 64: 16 * 2e-5 of |S| |dS| (twice the root of 64).  A
value that is not a normal fp32 number has no 24 bits: any may also be off by the
smallest normal one, 2^-126."""
from __future__ import annotations

import pytest
import torch

import structured_sparse_state_amd as pk
from tests import block_reference as ref

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
TOL_F32, TOL_BF16 = 2e-5, 2.0 ** -8 + 2e-5
TINY = 2.0 ** -126
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
STEPS = ("q", "k", "v", "g")


def say(msg):
    print(msg, flush=True)


def off(got, want):
    got, want = got.double().cpu(), want.double().cpu()
    assert got.shape == want.shape and torch.isfinite(got).all()
    n = want.norm()
    return float((got - want).norm() / n) if n > 0 else float(got.norm())


def place(t, order):
    """The same values held in another way."""
    if t is None or order == "head":
        return t if t is None else t.contiguous()
    if order == "token":
        return t.transpose(1, 2).contiguous().transpose(1, 2)
    # "apart": rows off every 16-byte boundary, gaps between all of them
    base = torch.full([n + 3 for n in t.shape], float("nan"), dtype=t.dtype, device=t.device)
    cut = base[tuple(slice(1, n + 1) for n in t.shape)]
    cut.copy_(t)
    return cut


def inputs(seed, B, Hk, Hv, L, Dk, Dv, dtype, s0=True, order="head", gates="plain"):
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=gen)  # noqa: E731
    q, k = 0.5 * r(B, Hk, L, Dk), 0.5 * (r(B, Hk, L, Dk) + 0.5 * r(B, Hk, 1, Dk))
    v, do = r(B, Hv, L, Dv), r(B, Hv, L, Dv)
    g = -0.2 * r(B, Hv, L).abs()
    if gates == "none":
        g = None
    elif gates == "heads":
        g = -torch.exp2(-torch.linspace(1, 8, Hv))
    elif gates == "strong":
        g = 60 * g
    elif gates == "growing":
        g = 0.02 * r(B, Hv, L)
    elif gates == "empty":      # steps that empty the state, the first and the last among them
        g = torch.where(torch.rand(g.shape, generator=gen) < 0.06, -float("inf"), g)
        g[..., 0] = g[..., -1] = -float("inf")
    x = {"q": q.to(dtype), "k": k.to(dtype), "v": v.to(dtype), "do": do.to(dtype), "g": g}
    x = {n: t if t is None else place(t.to(DEV), order if t.dim() > 2 else "head") for n, t in x.items()}
    x["s0"], x["ds"] = (0.3 * r(B, Hv, Dk, Dv).to(DEV) if s0 else None for _ in range(2))
    return x


def check_fwd(x, label, **kw):
    say(f"[case] forward {label}")
    want_o, want_s, _ = ref.linear(*(x[n] for n in STEPS), x["s0"], **kw)
    o, s = pk.linear_attention(*(x[n] for n in STEPS), x["s0"], **kw)
    torch.cuda.synchronize()
    eo, es = off(o, want_o), off(s, want_s)
    say(f"  o {eo:.2e} s {es:.2e}")
    assert eo <= (TOL_F32 if o.dtype == torch.float32 else TOL_BF16) and es <= TOL_F32
    return o, s


def check_dg(dg, want, size, g):
    assert torch.isfinite(dg).all()
    if g.dim() == 1:
        want, size = want.sum((0, 2)), size.sum((0, 2))
    e = ((dg.double().cpu() - want).abs() - TINY) / size.clamp_min(1e-300)
    say(f"  dg {float(e.max()):.2e}")
    assert (e <= 16 * TOL_F32).all()


def check_bwd(x, label, **kw):
    say(f"[case] backward {label}")
    args = [x[n] for n in STEPS]
    want, size = ref.linear_bwd(*args, x["do"], x["s0"], x["ds"], **kw)
    got = pk.linear_attention_bwd(*args, x["do"], x["s0"], x["ds"], **kw)
    plain = pk.linear_attention_bwd(*args, x["do"], x["s0"], x["ds"], want_dg=False, **kw)
    torch.cuda.synchronize()
    f32 = x["q"].dtype == torch.float32
    for name, n in (("dq", 0), ("dk", 1), ("dv", 2), ("ds0", 4)):
        assert torch.equal(got[n], plain[n]), name
        e = float((got[n].double().cpu() - want[n]).norm())
        say(f"  {name} {e / float(want[n].norm() + 1e-300):.2e}")
        assert torch.isfinite(got[n]).all()
        assert e <= (TOL_F32 if f32 or n == 4 else TOL_BF16) * float(want[n].norm()) + TINY * want[n].numel() ** 0.5, name
    assert plain[3] is None
    if x["g"] is None:
        assert got[3] is None
    else:
        check_dg(got[3], want[3], size, x["g"])
    return got


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("L", [1, 2, 15, 17, 63, 64, 65, 129, 200])
def test_lengths(dtype, L):
    x = inputs(L, 2, 1, 2, L, 48, 40, TYPES[dtype])
    check_fwd(x, f"L={L}")
    check_bwd(x, f"L={L}")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("Dk,Dv", [(1, 1), (8, 8), (3, 128), (128, 5), (64, 64), (65, 33), (96, 72), (128, 128)])
def test_head_sizes(dtype, Dk, Dv):
    x = inputs(Dk + Dv, 1, 1, 2, 140, Dk, Dv, TYPES[dtype])
    check_fwd(x, f"Dk={Dk} Dv={Dv}")
    check_bwd(x, f"Dk={Dk} Dv={Dv}")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("Hk,Hv", [(1, 1), (2, 4), (1, 3), (3, 3)])
@pytest.mark.parametrize("gates", ["plain", "heads"])
def test_shared_heads(dtype, Hk, Hv, gates):
    """Gradients of a query and key head that several value heads share, and of
    a decay that all sequences and steps share."""
    x = inputs(Hk * 10 + Hv, 2, Hk, Hv, 90, 64, 64, TYPES[dtype], s0=False, gates=gates)
    check_fwd(x, f"Hk={Hk} Hv={Hv} {gates}")
    check_bwd(x, f"Hk={Hk} Hv={Hv} {gates}")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("Dk,Dv", [(64, 32), (128, 100)])
@pytest.mark.parametrize("gates", ["none", "heads", "strong", "growing", "empty"])
def test_gates(dtype, gates, Dk, Dv):
    x = inputs(7, 1, 2, 2, 150, Dk, Dv, TYPES[dtype], gates=gates)
    check_fwd(x, gates)
    dg = check_bwd(x, gates)[3]
    if gates == "empty":
        assert (dg[torch.isinf(x["g"])] == 0).all()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("order", ["token", "apart"])
def test_memory_orders(dtype, order):
    x = inputs(3, 2, 2, 4, 77, 64, 48, TYPES[dtype], order=order)
    o, _ = check_fwd(x, order)
    if order == "token":
        assert o.stride() == x["v"].stride()
    check_bwd(x, order)

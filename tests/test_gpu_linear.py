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


def test_outputs_in_given_places():
    """Outputs with strides of their own, s_final over s0 and ds0 over
    ds_final, and nothing written beside them."""
    x = inputs(4, 2, 1, 2, 70, 40, 24, torch.bfloat16)
    args = [x[n] for n in STEPS]
    want_o, want_s = pk.linear_attention(*args, x["s0"])
    grads = pk.linear_attention_bwd(*args, x["do"], x["s0"], x["ds"])
    base = torch.full((2, 73, 5, 29), 7.0, dtype=torch.bfloat16, device=DEV)
    o = base[:, 2:72, 1:3, 3:27].transpose(1, 2)
    s = x["s0"].clone()
    pk.linear_attention(*args, s, o=o, s_final=s)
    torch.cuda.synchronize()
    assert torch.equal(o, want_o) and torch.equal(s, want_s)
    out = [torch.empty_like(x[n]) for n in ("q", "k")] + [o, torch.empty_like(x["g"])]
    ds = x["ds"].clone()
    pk.linear_attention_bwd(*args, x["do"], x["s0"], ds, out=(*out, ds))
    torch.cuda.synchronize()
    for a, b in zip((*out, ds), grads):
        assert torch.equal(a, b)
    base[:, 2:72, 1:3, 3:27] = 7.0
    assert (base == 7.0).all()


@pytest.mark.parametrize("dtype", TYPES)
def test_broadcast_inputs(dtype):
    """One query row for all steps, one key head for all batches, one gate for
    all steps (strides of 0), and a decay of every head against the same one
    written out for every step."""
    x = inputs(5, 2, 1, 2, 80, 64, 32, TYPES[dtype], gates="heads")
    x["q"] = x["q"][:, :, :1].expand(2, 1, 80, 64)
    x["k"] = x["k"][:1].expand(2, 1, 80, 64)
    x["do"] = x["do"][:, :, :1].expand(2, 2, 80, 32)
    heads = x["g"]
    o, s = check_fwd(x, "broadcast")
    out = [torch.empty(t.shape, dtype=t.dtype, device=DEV) for t in (x["q"], x["k"], x["v"], heads, x["s0"])]
    args = [x[n] for n in STEPS]
    pk.linear_attention_bwd(*args, x["do"], x["s0"], x["ds"], out=out)
    x["g"] = heads[None, :, None].expand(2, 2, 80)
    o2, s2 = pk.linear_attention(*(x[n] for n in STEPS), x["s0"])
    out2 = [torch.empty_like(t) for t in out[:3]] + [torch.empty(2, 2, 80, device=DEV), torch.empty_like(out[4])]
    pk.linear_attention_bwd(*(x[n] for n in STEPS), x["do"], x["s0"], x["ds"], out=out2)
    written = x["g"].contiguous()
    o3, s3 = pk.linear_attention(x["q"], x["k"], x["v"], written, x["s0"])
    torch.cuda.synchronize()
    assert torch.equal(o, o2) and torch.equal(s, s2) and torch.equal(o, o3) and torch.equal(s, s3)
    for n in (0, 1, 2, 4):
        assert torch.equal(out[n], out2[n])
    want, size = ref.linear_bwd(*args, x["do"], x["s0"], x["ds"])
    for n, a in enumerate(out[:3]):
        assert off(a.float(), want[n]) <= (TOL_BF16 if dtype == "bf16" else TOL_F32)
    check_dg(out[3], want[3], size, heads)
    check_dg(out2[3], want[3], size, written)


def cut(B, Hk, Hv, L, Dk, Dv, flags=1):
    """Whether the forward of these sizes is walked in segments."""
    return pk.pdssm_linear_workspace_bytes(B, Hk, Hv, L, Dk, Dv, flags) > 256


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("B,Hk,Hv,L,Dk,Dv,order,gates,s0", [
    (1, 1, 2, 64 * 40 + 5, 64, 64, "token", "plain", True),
    (1, 1, 2, 64 * 40 + 5, 128, 128, "head", "heads", True),
    (1, 1, 1, 64 * 16, 128, 128, "head", "plain", False),       # the fewest chunks
    (2, 1, 3, 64 * 33 + 1, 64, 32, "token", "plain", True),     # shared heads, one step in the last chunk
    (1, 1, 2, 64 * 41, 64, 128, "token", "empty", True),        # a last segment of one chunk; empty states in all
    (1, 2, 2, 64 * 37 + 5, 128, 96, "head", "empty", False),
    (2, 1, 2, 64 * 20 + 9, 50, 70, "apart", "none", True),      # rows read value by value
    (3, 1, 1, 64 * 18, 72, 8, "apart", "strong", True),
    (1, 1, 1, 64 * 130, 16, 16, "head", "heads", True),
])
def test_cut_sequences(dtype, B, Hk, Hv, L, Dk, Dv, order, gates, s0):
    x = inputs(L, B, Hk, Hv, L, Dk, Dv, TYPES[dtype], order=order, gates=gates, s0=s0)
    assert cut(B, Hk, Hv, L, Dk, Dv, int(dtype == "bf16"))
    check_fwd(x, f"cut L={L} Dk={Dk} Dv={Dv} {order} {gates}")
    check_bwd(x, f"cut L={L} Dk={Dk} Dv={Dv} {order} {gates}")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("B,Hk,Hv,L,Dk,Dv,order,gates,s0", [
    (1, 1, 1, 64 * 2, 64, 64, "token", "plain", True),          # two chunks: a segment each, where that pays
    (1, 1, 2, 64 * 3 + 1, 100, 40, "head", "heads", True),      # segments of one chunk, one step in the last
    (2, 1, 2, 64 * 4, 128, 128, "token", "empty", True),
    (1, 2, 4, 64 * 6, 128, 72, "apart", "strong", True),        # the fewest chunks of a bf16 forward that are cut
    (1, 2, 2, 64 * 7 + 9, 64, 128, "head", "none", False),
    (2, 40, 80, 130, 24, 72, "token", "plain", True),           # so many heads that a workgroup takes 128 columns
    (2, 64, 64, 64, 8, 128, "head", "heads", False),            # and just not
    (1, 100, 100, 64 * 16 + 1, 16, 16, "token", "plain", True), # two segments
])
def test_columns_and_segments_of_short_sequences(dtype, B, Hk, Hv, L, Dk, Dv, order, gates, s0):
    x = inputs(L + Dv, B, Hk, Hv, L, Dk, Dv, TYPES[dtype], order=order, gates=gates, s0=s0)
    check_fwd(x, f"short L={L} Hv={Hv} Dk={Dk} Dv={Dv} {order} {gates}")
    check_bwd(x, f"short L={L} Hv={Hv} Dk={Dk} Dv={Dv} {order} {gates}")


@pytest.mark.parametrize("Dk,Dv", [(64, 64), (128, 128), (40, 72)])
def test_states_in_place_of_cut_sequences(Dk, Dv):
    """s_final over s0 and ds0 over ds_final, bit for bit as elsewhere."""
    x = inputs(Dk + 1, 1, 1, 2, 2565, Dk, Dv, torch.bfloat16, order="token")
    assert cut(1, 1, 2, 2565, Dk, Dv)
    args = [x[n] for n in STEPS]
    want = [*pk.linear_attention(*args, x["s0"]), *pk.linear_attention_bwd(*args, x["do"], x["s0"], x["ds"])]
    s, ds = x["s0"].clone(), x["ds"].clone()
    o, _ = pk.linear_attention(*args, s, s_final=s)
    out = [torch.empty_like(t) for t in want[2:6]]
    pk.linear_attention_bwd(*args, x["do"], x["s0"], ds, out=(*out, ds))
    torch.cuda.synchronize()
    for a, b in zip((o, s, *out, ds), want):
        assert torch.equal(a, b)


LOWEST = torch.finfo(torch.float32).min


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("at", [(0,), (10,), (63, 64), (10, 11, 100), (149,)])
@pytest.mark.parametrize("gate", [-103.0, -105.0, -1e4, -1e30, LOWEST])
def test_large_negative_gates(dtype, at, gate):
    """A mask's value among ordinary gates: at the first and the last step, in
    and at the ends of a chunk, once and several times."""
    x = inputs(21, 1, 1, 2, 150, 32, 32, TYPES[dtype])
    x["g"][:, :, list(at)] = gate
    check_fwd(x, f"gate {gate:.3g} at {at}")
    dg = check_bwd(x, f"gate {gate:.3g} at {at}")[3]
    if gate < -104:
        assert (dg[:, :, list(at)] == 0).all()


@pytest.mark.parametrize("gate", [-105.0, LOWEST, -float("inf")])
def test_heads_that_forget_everything(gate):
    """A fixed decay that empties the state before every step: o_t = scale (q_t . k_t) v_t."""
    x = inputs(23, 2, 1, 3, 200, 64, 64, torch.float32, gates="heads")
    x["g"][1] = gate
    check_fwd(x, f"heads, {gate:.3g}")
    dg = check_bwd(x, f"heads, {gate:.3g}")[3]
    assert dg[1] == 0


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("Dk,Dv,Hk", [(48, 40, 2), (128, 128, 1), (64, 100, 1)])
@pytest.mark.parametrize("gates", [-0.2, -2.0, -10.0, -20.0, "mixed"])
def test_every_gradient_of_a_gate(dtype, gates, Dk, Dv, Hk):
    """dg step by step under decays that make it small (the bound of check_dg is
    relative to |S| |dS| of the step)."""
    x = inputs(71, 1, Hk, 2, 150, Dk, Dv, TYPES[dtype])
    noise = x["g"]      # -0.2 |normal|
    x["g"] = noise + gates if gates != "mixed" else torch.where(noise < -0.2, 100 * noise, noise)
    check_bwd(x, f"dg, gates {gates}, Dk={Dk} Dv={Dv}")


@pytest.mark.parametrize("Dk,Dv", [(64, 64), (128, 128), (40, 72)])
def test_bf16_results_are_rounded_once(Dk, Dv):
    """Results of fp32 accuracy rounded to bf16 differ from the reference
    rounded to bf16 only where a value lies next to the middle of two: an error
    of d moves a value by an ulp in d / ulp of the cases, so the norm of the
    difference is about the root of |d| |ulp|, for the 2e-5 of fp32 results
    and 2^-7 the root of 1.6e-7: 4e-4, below 2^-11."""
    x = inputs(61, 2, 2, 4, 200, Dk, Dv, torch.bfloat16)
    args = [x[n] for n in STEPS]
    want_o, _, _ = ref.linear(*args, x["s0"])
    grads, _ = ref.linear_bwd(*args, x["do"], x["s0"], x["ds"])
    got = [pk.linear_attention(*args, x["s0"])[0], *pk.linear_attention_bwd(*args, x["do"], x["s0"], x["ds"])[:3]]
    torch.cuda.synchronize()
    for name, a, b in zip(("o", "dq", "dk", "dv"), got, (want_o, *grads)):
        apart = float((a.double().cpu() - b.to(torch.bfloat16).double()).norm() / b.norm())
        say(f"  {name} {apart:.2e}")
        assert apart <= 2.0 ** -11, name


def test_gradient_against_differences():
    """The GPU's gradients along random directions against central differences
    of the 64-bit reference's loss."""
    for gates in ("plain", "heads"):
        x = inputs(11, 1, 1, 2, 40, 16, 16, torch.float32, gates=gates)
        got = pk.linear_attention_bwd(*(x[n] for n in STEPS), x["do"], x["s0"], x["ds"])
        y = {n: t.double().cpu() for n, t in x.items()}
        loss = lambda z: sum((a * b).sum() for a, b in zip(ref.linear(*(z[n] for n in STEPS), z["s0"])[:2], (y["do"], y["ds"])))  # noqa: E731
        gen = torch.Generator().manual_seed(1)
        for name, grad in zip((*STEPS, "s0"), got):
            d = torch.randn(y[name].shape, generator=gen, dtype=torch.float64)
            diff = (loss({**y, name: y[name] + 1e-6 * d}) - loss({**y, name: y[name] - 1e-6 * d})) / 2e-6
            along = (grad.double().cpu() * d).sum()
            assert abs(diff - along) <= 1e-4 * float(grad.double().norm()) * (d.numel() ** 0.5), name


def test_scale_and_no_state():
    x = inputs(12, 1, 1, 1, 30, 32, 32, torch.float32, s0=False)
    args = [x[n] for n in STEPS]
    o, s = pk.linear_attention(*args, scale=2.5, want_state=False)
    assert s is None and off(o, ref.linear(*args, scale=2.5)[0]) <= TOL_F32
    got = pk.linear_attention_bwd(*args, x["do"], scale=2.5, want_ds0=False)
    assert got[4] is None
    for a, b in zip(got[:3], ref.linear_bwd(*args, x["do"], scale=2.5)[0]):
        assert off(a, b) <= TOL_F32


def test_empty_shapes():
    for B, Hv, L in ((0, 2, 5), (2, 0, 5), (2, 2, 0), (0, 0, 0)):
        q = torch.zeros(B, Hv, L, 8, device=DEV)
        s0 = torch.randn(B, Hv, 8, 8, device=DEV)
        for g in (torch.zeros(B, Hv, L, device=DEV), torch.full((Hv,), -0.1, device=DEV), None):
            o, s = pk.linear_attention(q, q, q, g, s0)
            assert o.shape == q.shape and torch.equal(s, s0)
            assert torch.equal(pk.linear_attention(q, q, q, g)[1], torch.zeros_like(s0))
            dq, dk, dv, dg, ds0 = pk.linear_attention_bwd(q, q, q, g, q, s0, s0)
            assert torch.equal(ds0, s0) and dq.shape == dk.shape == dv.shape == q.shape
            if g is not None:
                assert dg.shape == g.shape and (dg == 0).all()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("L", [150, 64 * 40])
def test_results_are_reproducible_whatever_the_workspace_holds(L, dtype):
    x = inputs(13, 1, 1, 2, L, 64, 100, TYPES[dtype])
    args = [x[n] for n in STEPS]
    results = []
    for fill in (0, 255):       # 255: NaN in every word
        fwd, bwd = (torch.full((f(1, 1, 2, L, 64, 100, int(dtype == "bf16")),), fill, dtype=torch.uint8, device=DEV)
                    for f in (pk.pdssm_linear_workspace_bytes, pk.pdssm_linear_bwd_workspace_bytes))
        results.append([*pk.linear_attention(*args, x["s0"], workspace=fwd),
                        *pk.linear_attention_bwd(*args, x["do"], x["s0"], x["ds"], workspace=bwd)])
    torch.cuda.synchronize()
    for a, b in zip(*results):
        assert torch.equal(a, b)


NAN, INF = float("nan"), float("inf")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("name,value", [("q", NAN), ("q", INF), ("k", NAN), ("k", INF), ("v", NAN), ("v", -INF), ("g", NAN),
                                        ("g", INF)])
@pytest.mark.parametrize("L,at,Dk,Dv", [(150, 0, 64, 64), (150, 5, 40, 72), (150, 63, 64, 64), (150, 100, 128, 128),
                                        (150, 149, 64, 33), (2565, 1000, 128, 64), (2565, 2564, 64, 64)])
def test_what_is_not_finite_leaves_the_steps_before_alone(dtype, name, value, L, at, Dk, Dv):
    """In the state's rows and columns that it reaches, from its step on, and
    nowhere else."""
    x = inputs(81, 2, 1, 2, L, Dk, Dv, TYPES[dtype])
    say(f"[case] {name} = {value} at {at} of {L}, Dk={Dk} Dv={Dv} {dtype}")
    o, s = pk.linear_attention(*(x[n] for n in STEPS), x["s0"])
    y = x[name].clone()
    y[(1, 0, at) if name == "g" else (1, 0, at, 3)] = value
    bad, bad_s = pk.linear_attention(*({**x, name: y}[n] for n in STEPS), x["s0"])
    torch.cuda.synchronize()
    reached = torch.zeros_like(o, dtype=torch.bool)     # both value heads share the query and key head
    if name == "q":
        reached[1, :, at] = True
    elif name == "v":
        reached[1, 0, at:, 3] = True
    else:
        reached[1, :2 if name == "k" else 1, at:] = True
    assert torch.equal(bad[~reached], o[~reached])
    assert not torch.isfinite(bad[reached]).any()
    state = torch.zeros_like(s, dtype=torch.bool)
    if name == "k":             # S += k v^T: a value of k has one row of the state
        state[1, :, 3] = True
    elif name != "q":
        state[:] = reached[:, :, -1, None, :].expand_as(s)
    assert torch.equal(bad_s[~state], s[~state]) and not torch.isfinite(bad_s[state]).any()


def test_what_is_not_finite_stays_in_its_sequence_of_the_gradients():
    x = inputs(82, 3, 1, 2, 150, 64, 64, torch.bfloat16)
    want = pk.linear_attention_bwd(*(x[n] for n in STEPS), x["do"], x["s0"], x["ds"])
    for name in ("q", "k", "v", "do"):
        y = {**x, name: x[name].clone()}
        y[name][1, 0, 70, 5] = NAN
        got = pk.linear_attention_bwd(*(y[n] for n in STEPS), y["do"], y["s0"], y["ds"])
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a[0], b[0]) and torch.equal(a[2], b[2]), name


def test_another_stream():
    x = inputs(15, 1, 2, 2, 300, 64, 64, torch.bfloat16)
    args = [x[n] for n in STEPS]
    want = [*pk.linear_attention(*args, x["s0"]), *pk.linear_attention_bwd(*args, x["do"], x["s0"], x["ds"])]
    torch.cuda.synchronize()
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        got = list(pk.linear_attention(*args, x["s0"]))
    ws = torch.empty(pk.pdssm_linear_bwd_workspace_bytes(1, 2, 2, 300, 64, 64, 1), dtype=torch.uint8, device=DEV)
    out = [torch.empty_like(t) for t in want[2:]]
    torch.cuda.synchronize()
    got += list(pk.linear_attention_bwd(*args, x["do"], x["s0"], x["ds"], out=out, workspace=ws, stream=stream))
    stream.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("L", [100, 64 * 20])
def test_graph_replays(L):
    """A captured forward, backward and step, replayed with other inputs in between."""
    x = inputs(16, 2, 1, 2, L, 64, 64, torch.bfloat16)
    fwd = torch.empty(pk.pdssm_linear_workspace_bytes(2, 1, 2, L, 64, 64, 1), dtype=torch.uint8, device=DEV)
    bwd = torch.empty(pk.pdssm_linear_bwd_workspace_bytes(2, 1, 2, L, 64, 64, 1), dtype=torch.uint8, device=DEV)
    o, s = torch.empty_like(x["v"]), torch.empty_like(x["s0"])
    grads = [torch.empty_like(x[n]) for n in (*STEPS, "s0")]
    first = [x[n][:, :, 0].contiguous() for n in STEPS]
    so, state, ds = torch.empty_like(first[2]), x["s0"].clone(), x["ds"].clone()
    args = [x[n] for n in STEPS]

    def call():
        pk.linear_attention(*args, x["s0"], o=o, s_final=s, workspace=fwd)
        pk.linear_attention_bwd(*args, x["do"], x["s0"], ds, out=grads, workspace=bwd)
        pk.linear_attention_step(*first, state, o=so)

    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for n in range(3):
        x["v"].copy_(torch.randn(x["v"].shape, device=DEV))
        state.copy_(x["s0"])
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        eager = [*pk.linear_attention(*args, x["s0"]), *pk.linear_attention_bwd(*args, x["do"], x["s0"], ds)]
        stepped = x["s0"].clone()
        eager_o = pk.linear_attention_step(*first, stepped)
        torch.cuda.synchronize()
        for a, b in zip((o, s, *grads, so, state), (*eager, eager_o, stepped)):
            assert torch.equal(a, b)


def test_offsets_beyond_32_bits():
    """A batch stride of more than 2^32 bytes."""
    far = (1 << 31) + 64
    base = torch.empty(far + 64 * 70, dtype=torch.bfloat16, device=DEV)
    x = inputs(17, 2, 1, 1, 70, 64, 64, torch.bfloat16)
    v = base.as_strided((2, 1, 70, 64), (far, 70 * 64, 64, 1))
    v.copy_(x["v"])
    o = torch.empty(2, 1, 70, 64, dtype=torch.bfloat16, device=DEV)
    want, _ = pk.linear_attention(*(x[n] for n in STEPS), x["s0"])
    pk.linear_attention(x["q"], x["k"], v, x["g"], x["s0"], o=o)
    torch.cuda.synchronize()
    assert torch.equal(o, want)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("gates", ["empty", "heads", "none"])
@pytest.mark.parametrize("B,Hk,Hv,Dk,Dv", [(1, 1, 1, 1, 1), (3, 2, 4, 64, 64), (2, 1, 3, 128, 128), (1, 2, 2, 65, 33),
                                           (2, 2, 2, 7, 128), (300, 1, 1, 16, 20)])
def test_step(dtype, gates, B, Hk, Hv, Dk, Dv):
    x = inputs(B + Dk, B, Hk, Hv, 3, Dk, Dv, TYPES[dtype], gates=gates)
    say(f"[case] step B={B} Hk={Hk} Hv={Hv} Dk={Dk} Dv={Dv} {gates}")
    want_o, _, states = ref.linear(*(x[n] for n in STEPS), x["s0"])
    s = x["s0"].clone()
    for t in range(3):
        args = [x[n][:, :, t] for n in ("q", "k", "v")]     # views with the sequence's strides
        args.append(x["g"][:, :, t] if gates == "empty" else x["g"])
        before, apart = s.clone(), torch.full_like(s, float("nan"))
        o = pk.linear_attention_step(*args, s)
        o2 = pk.linear_attention_step(*args, before, s_out=apart)
        torch.cuda.synchronize()
        assert torch.equal(o, o2) and torch.equal(s, apart)
        assert off(o.float(), want_o[:, :, t]) <= (TOL_F32 if dtype == "f32" else TOL_BF16)
        assert off(s, states[t + 1]) <= TOL_F32


def test_steps_continue_a_sequence():
    """A prompt through the forward, then steps, against one long forward."""
    x = inputs(20, 2, 2, 4, 90, 64, 64, torch.bfloat16)
    o, s = pk.linear_attention(*(x[n] for n in STEPS), x["s0"])
    first, state = pk.linear_attention(*(x[n][:, :, :70] for n in STEPS), x["s0"])
    rest = [pk.linear_attention_step(*(x[n][:, :, t] for n in STEPS), state) for t in range(70, 90)]
    got = torch.cat([first, torch.stack(rest, 2)], 2)
    torch.cuda.synchronize()
    assert off(got.float(), o.float()) <= 2 * TOL_BF16 and off(state, s) <= 2 * TOL_F32


def test_more_heads_than_one_grid_dimension_holds():
    """2^24 sequences and some: more than 2^32 threads in one row of workgroups."""
    B = (1 << 24) + 70
    gen = torch.Generator(device=DEV).manual_seed(51)
    r = lambda *s: torch.randn(s, generator=gen, device=DEV)  # noqa: E731
    q, k, v, s, g = r(B, 1, 1), r(B, 1, 1), r(B, 1, 1), r(B, 1, 1, 1), -r(B, 1).abs()
    say("[case] 2^24 states")
    S = s.double() * g.double().exp()[..., None, None] + k.double()[..., None] * v.double()[..., None, :]
    want = q.double() * S[..., 0]
    o, s2 = pk.linear_attention(*(x[:, :, None] for x in (q, k, v, g)), s)
    assert off(s2, S) <= TOL_F32 and off(o[:, :, 0], want) <= TOL_F32
    del o, s2
    o = pk.linear_attention_step(q, k, v, g, s)
    torch.cuda.synchronize()
    assert off(s, S) <= TOL_F32 and off(o, want) <= TOL_F32

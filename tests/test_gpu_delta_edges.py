"""The gated delta rule on the GPU at the edges of its range: gates that empty
the state, whatever value says so; long sequences of few heads, which are cut
into segments; gates whose gradient strong decays make small; values that are
not finite; more states than one grid dimension holds.  Inputs and tolerances
are those of test_gpu_delta; a result that is not a normal fp32 number has no
24 bits, so every value may also be off by the smallest normal one, 2^-126."""
from __future__ import annotations

import pytest
import torch

import structured_sparse_state_amd as pk
from tests import layers_reference as ref
from tests.test_gpu_delta import TOL_F32, TOL_KEYS, TOL_OUT, TYPES, inputs, off, say

pytestmark = pytest.mark.gpu

LOWEST = torch.finfo(torch.float32).min
STEPS = ("q", "k", "v", "g", "beta")


def check(x, label):
    """Forward and gradients against the reference; returns the gradients."""
    say(f"[case] {label}")
    args = [x[n] for n in STEPS]
    want_o, want_s, _ = ref.delta(*args, x["s0"])
    grads, terms = ref.delta_bwd(*args, x["do"], x["s0"], x["ds"])
    got = [*pk.delta_rule(*args, x["s0"]), *pk.delta_rule_bwd(*args, x["do"], x["s0"], x["ds"])]
    torch.cuda.synchronize()
    f32 = x["q"].dtype == torch.float32
    tols = [TOL_F32] * 8 if f32 else [TOL_OUT, TOL_F32, TOL_KEYS, TOL_KEYS, TOL_OUT, TOL_F32, TOL_F32, TOL_F32]
    for name, a, b, tol in zip(("o", "s", "dq", "dk", "dv", "dg", "dbeta", "ds0"), got, (want_o, want_s, *grads), tols):
        assert a.shape == b.shape and torch.isfinite(a).all(), name
        size = b.norm() + (8 * terms.norm() if name == "dg" else 0)
        e = float((a.double().cpu() - b).norm())
        say(f"  {name} {e:.2e} of {size:.2e}")
        assert e <= tol * size + 2.0 ** -126 * b.numel() ** 0.5, name
    return got[2:]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("at", [(0,), (10,), (63, 64), (10, 11, 100), (149,)])
@pytest.mark.parametrize("gate", [-103.0, -105.0, -1e4, -1e12, -1e30, LOWEST])
def test_large_negative_gates(dtype, at, gate):
    """A mask's value among ordinary gates: at the first and the last step, in
    and at the ends of a chunk, once and several times."""
    x = inputs(21, 1, 1, 2, 150, 32, 32, TYPES[dtype])
    x["g"][:, :, list(at)] = gate
    dg = check(x, f"{dtype} gate {gate:.3g} at {at}")[3]
    if gate < -104:
        assert (dg[:, :, list(at)] == 0).all()


@pytest.mark.parametrize("gate", [-1e4, -1e15, LOWEST, -float("inf")])
def test_whole_sequences_and_steps_agree_on_gates(gate):
    x = inputs(22, 2, 1, 2, 70, 64, 64, torch.bfloat16)
    x["g"][:, 0, ::7] = gate
    x["g"][:, 1, 33:] = gate
    say(f"[case] forward against steps, gate {gate:.3g}")
    o, s = pk.delta_rule(*(x[n] for n in STEPS), x["s0"])
    state = x["s0"].clone()
    steps = [pk.delta_step(*(x[n][:, :, t] for n in STEPS), state) for t in range(70)]
    torch.cuda.synchronize()
    assert off(o.float(), torch.stack(steps, 2).float().cpu()) <= 2 * TOL_OUT and off(s, state.cpu()) <= 2 * TOL_F32


def cut(B, Hk, Hv, L, Dk, Dv):
    """Whether a bf16 sequence of these sizes is walked in segments."""
    chunks = B * Hv * ((L + 63) // 64)
    return pk.pdssm_delta_workspace_bytes(B, Hk, Hv, L, Dk, Dv, 1) > chunks * (2 * 2560 + 512) * 4


@pytest.mark.parametrize("Dk,Dv", [(64, 64), (128, 128), (40, 72)])
def test_states_in_place_of_cut_sequences(Dk, Dv):
    """s_final over s0 and ds0 over ds_final, bit for bit as elsewhere."""
    x = inputs(Dk + 1, 1, 1, 2, 2565, Dk, Dv, torch.bfloat16, order="token")
    assert cut(1, 1, 2, 2565, Dk, Dv)
    args = [x[n] for n in STEPS]
    say(f"[case] in place, cut, Dk={Dk} Dv={Dv}")
    want = [*pk.delta_rule(*args, x["s0"]), *pk.delta_rule_bwd(*args, x["do"], x["s0"], x["ds"])]
    s, ds = x["s0"].clone(), x["ds"].clone()
    o, _ = pk.delta_rule(*args, s, s_final=s)
    out = [torch.empty_like(t) for t in want[2:7]]
    pk.delta_rule_bwd(*args, x["do"], x["s0"], ds, out=(*out, ds))
    torch.cuda.synchronize()
    for a, b in zip((o, s, *out, ds), want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("B,Hk,Hv,L,Dk,Dv,order,gates,s0", [
    (1, 1, 1, 64 * 16, 128, 128, "head", "plain", False),       # the fewest chunks
    (2, 1, 3, 64 * 33 + 1, 64, 32, "token", "plain", True),     # shared heads, one step in the last chunk
    (1, 1, 2, 64 * 41, 64, 64, "token", "empty", True),         # a last segment of one chunk; empty states in all
    (1, 2, 2, 64 * 37 + 5, 128, 96, "head", "empty", False),
    (2, 1, 2, 64 * 20 + 9, 50, 70, "apart", "plain", True),     # rows read value by value
    (3, 1, 1, 64 * 18, 72, 8, "apart", "strong", True),
])
def test_cut_sequences(B, Hk, Hv, L, Dk, Dv, order, gates, s0):
    x = inputs(L, B, Hk, Hv, L, Dk, Dv, torch.bfloat16, order=order, gates=gates, s0=s0)
    assert cut(B, Hk, Hv, L, Dk, Dv)
    check(x, f"cut B={B} Hk={Hk} Hv={Hv} L={L} Dk={Dk} Dv={Dv} {order} {gates}")


def test_step_of_more_heads_than_one_grid_dimension_holds():
    """2^24 states and some, more than 2^32 threads in one row of workgroups."""
    B = (1 << 24) + 70
    gen = torch.Generator(device="cuda:0").manual_seed(51)
    r = lambda *s: torch.randn(s, generator=gen, device="cuda:0")  # noqa: E731
    q, k, v, s = r(B, 1, 1), r(B, 1, 1), r(B, 1, 1), r(B, 1, 1, 1)
    g, beta = -r(B, 1).abs(), torch.sigmoid(r(B, 1))
    say("[case] step, 2^24 states")
    S = s.double() * g.double().exp()[..., None, None]
    S = S + (k * beta[..., None]).double()[..., None] * (v.double() - k.double() * S[..., 0])[..., None]
    o = pk.delta_step(q, k, v, g, beta, s)
    torch.cuda.synchronize()
    assert off(s, S.cpu()) <= TOL_F32 and off(o, (q.double() * S[..., 0]).cpu()) <= TOL_F32


@pytest.mark.parametrize("Dk,Dv", [(64, 64), (128, 128), (40, 72)])
def test_bf16_results_are_rounded_once(Dk, Dv):
    """Results of fp32 accuracy rounded to bf16 differ from the reference
    rounded to bf16 only where a value lies next to the middle of two: an error
    of d moves a value by an ulp in d / ulp of the cases, so the norm of the
    difference is about the root of |d| |ulp|, for the 2e-5 of fp32 results
    and 2^-7 the root of 1.6e-7: 4e-4, below 2^-11."""
    x = inputs(61, 2, 2, 4, 200, Dk, Dv, torch.bfloat16)
    say(f"[case] rounded once, Dk={Dk} Dv={Dv}")
    args = [x[n] for n in STEPS]
    want_o, _, _ = ref.delta(*args, x["s0"])
    grads, _ = ref.delta_bwd(*args, x["do"], x["s0"], x["ds"])
    got = [pk.delta_rule(*args, x["s0"])[0], *pk.delta_rule_bwd(*args, x["do"], x["s0"], x["ds"])[:3]]
    torch.cuda.synchronize()
    for name, a, b in zip(("o", "dq", "dk", "dv"), got, (want_o, *grads)):
        apart = float((a.double().cpu() - b.to(torch.bfloat16).double()).norm() / b.norm())
        say(f"  {name} {apart:.2e}")
        assert apart <= 2.0 ** -11, name


def sizes_of_dg(x):
    """|S| |dS| around every step's decay, whose product dg is, in 64 bits."""
    group = x["v"].shape[1] // x["q"].shape[1]
    _, _, states = ref.delta(*(x[n] for n in STEPS), x["s0"])
    q, k = (x[n].double().cpu().repeat_interleave(group, 1) for n in "qk")
    g, beta, do = (x[n].double().cpu() for n in ("g", "beta", "do"))
    dS = torch.zeros_like(states[0]) if x["ds"] is None else x["ds"].double().cpu()
    out = torch.zeros_like(g)
    for t in reversed(range(q.shape[2])):
        a, kt = g[:, :, t].exp()[..., None, None], k[:, :, t, :, None]
        dS = dS + q.shape[-1] ** -0.5 * q[:, :, t, :, None] * do[:, :, t, None, :]
        dS = dS - kt * (beta[:, :, t, None] * (kt * dS).sum(-2))[..., None, :]
        out[:, :, t] = (states[t] * a).norm(dim=(-2, -1)) * dS.norm(dim=(-2, -1))
        dS = dS * a
    return out


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("Dk,Dv,Hk", [(48, 40, 2), (128, 128, 1), (64, 100, 1)])
@pytest.mark.parametrize("gates", [-0.2, -2.0, -10.0, -20.0, "mixed"])
def test_every_gradient_of_a_gate(dtype, gates, Dk, Dv, Hk):
    """dg step by step.  It is <S, dS>, both known to TOL_F32 of their norms, as
    a sum over pairs of steps that may cancel among themselves by the root of
    64: 16 * TOL_F32 of |S| |dS|, which strong decays make small.  (Parts below
    fp32's normal numbers again have no 24 bits.)"""
    x = inputs(71, 1, Hk, 2, 150, Dk, Dv, TYPES[dtype])
    noise = x["g"]      # -0.2 |normal|
    x["g"] = noise + gates if gates != "mixed" else torch.where(noise < -0.2, 100 * noise, noise)
    say(f"[case] dg, {dtype}, gates {gates}, Dk={Dk} Dv={Dv}")
    args = [x[n] for n in STEPS]
    want = ref.delta_bwd(*args, x["do"], x["s0"], x["ds"])[0][3]
    got = pk.delta_rule_bwd(*args, x["do"], x["s0"], x["ds"])[3].double().cpu()
    size = sizes_of_dg(x)
    torch.cuda.synchronize()
    e = ((got - want).abs() - 2.0 ** -126) / size
    say(f"  worst {float(e.max()):.2e} median {float(((got - want).abs() / want.abs()).median()):.2e}")
    assert (want.abs() <= size * (1 + 1e-9)).all() and (e <= 16 * TOL_F32).all()


NAN, INF = float("nan"), float("inf")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("name,value", [("q", NAN), ("q", INF), ("k", NAN), ("k", INF), ("v", NAN), ("v", -INF), ("g", NAN),
                                        ("g", INF), ("beta", NAN), ("beta", INF)])
@pytest.mark.parametrize("L,at,Dk,Dv", [(150, 0, 64, 64), (150, 5, 40, 72), (150, 63, 64, 64), (150, 100, 128, 128),
                                        (150, 149, 64, 33), (2565, 1000, 128, 64), (2565, 2564, 64, 64)])
def test_what_is_not_finite_leaves_the_steps_before_alone(dtype, name, value, L, at, Dk, Dv):
    """In the state's columns that it reaches, from its step on, and nowhere else."""
    x = inputs(81, 2, 1, 2, L, Dk, Dv, TYPES[dtype])
    say(f"[case] {name} = {value} at {at} of {L}, Dk={Dk} Dv={Dv} {dtype}")
    o, s = pk.delta_rule(*(x[n] for n in STEPS), x["s0"])
    y = x[name].clone()
    y[(1, 0, at) if name in ("g", "beta") else (1, 0, at, 3)] = value
    bad, bad_s = pk.delta_rule(*({**x, name: y}[n] for n in STEPS), x["s0"])
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
    if name != "q":
        state[:] = reached[:, :, -1, None, :].expand_as(s)
    assert torch.equal(bad_s[~state], s[~state]) and not torch.isfinite(bad_s[state]).any()

"""Linear attention whose state grows by more than fp32 holds while it, or what it
is read with, is zero or tiny: finite inputs with finite results.

Bounds, fixed beforehand, step by step, for sizes differ by many powers of ten.
A product's terms are summed in fp32 over at most 192 of them, and a state takes
one rounding a step and two of its decay (e^g to 2^-23 of itself): over the at
most 200 steps that a state lives here, (192 + 3 * 200) * 2^-24 = 4.8e-5 of the
product of the sizes of what is multiplied: TOL = 5e-5.  o: scale |q_t| |S_t|.
dq, dk, dv likewise with the state and its gradient, dg: |S| |dS| of the step
and, as a sum over pairs of steps, 16 times that.  A bf16 result is rounded once,
2^-8 of itself at most.  Any value may be off by the smallest normal one."""
from __future__ import annotations

import pytest
import torch

import structured_sparse_state_amd as pk
from tests import block_reference as ref
from tests.test_gpu_linear import DEV, STEPS, TINY, TYPES, inputs, say

pytestmark = pytest.mark.gpu

TOL = 5e-5
NONE = -float("inf")


def near(got, want, size, name, tol=TOL):
    """Every value within its rounding and `tol` of `size` (of its row)."""
    assert got.shape == want.shape
    half = 2.0 ** -8 if got.dtype == torch.bfloat16 else 0.0
    assert torch.isfinite(want).all() and torch.isfinite(got).all(), name
    e = (got.double().cpu() - want).abs()
    bound = half * want.abs() + tol * size + TINY
    say(f"  {name} {float((e / bound).max()):.2f} of its bound")
    assert (e <= bound).all(), name


def length(x):
    return x.double().cpu().norm(dim=-1, keepdim=True)


def heads(x, group):
    return x.repeat_interleave(group, 1)


def check(x, label, backward=True):
    say(f"[case] {label}")
    args, group = [x[n] for n in STEPS], x["v"].shape[1] // x["q"].shape[1]
    scale = x["q"].shape[-1] ** -0.5
    want_o, want_s, states = ref.linear(*args, x["s0"])
    o, s = pk.linear_attention(*args, x["s0"])
    torch.cuda.synchronize()
    after = torch.stack([S.norm(dim=(-2, -1)) for S in states[1:]], 2)[..., None]
    near(o, want_o, scale * heads(length(x["q"]), group) * after, "o")
    near(s, want_s, after[:, :, -1, None], "s")
    if not backward:
        return
    want, size = ref.linear_bwd(*args, x["do"], x["s0"], x["ds"])
    dq, dk, dv, dg, ds0 = pk.linear_attention_bwd(*args, x["do"], x["s0"], x["ds"])
    plain = pk.linear_attention_bwd(*args, x["do"], x["s0"], x["ds"], want_dg=False)
    torch.cuda.synchronize()
    for a, b in zip((dq, dk, dv, ds0), (*plain[:3], plain[4])):
        assert torch.equal(a, b)
    # |dS| of every step, from which dk and dv are read
    g = ref.gates(x["g"], *x["v"].shape[:3])
    dS = torch.zeros_like(states[0]) if x["ds"] is None else x["ds"].double().cpu()
    sizes = []
    for t in reversed(range(g.shape[2])):
        dS = dS + scale * heads(x["q"], group)[:, :, t, :, None].double().cpu() * x["do"][:, :, t, None, :].double().cpu()
        sizes.append(dS.norm(dim=(-2, -1)))
        dS = dS * g[:, :, t].exp()[..., None, None]
    grown = torch.stack(sizes[::-1], 2)[..., None]
    sums = lambda t: t.unflatten(1, (-1, group)).sum(2)  # noqa: E731
    near(dq, want[0], sums(scale * length(x["do"]) * after), "dq")
    near(dk, want[1], sums(length(x["v"]) * grown), "dk")
    near(dv, want[2], heads(length(x["k"]), group) * grown, "dv")
    near(ds0, want[4], dS.norm(dim=(-2, -1), keepdim=True), "ds0")
    dg_size, dg_want = size, want[3]
    if x["g"].dim() == 1:
        dg_size, dg_want = size.sum((0, 2)), dg_want.sum((0, 2))
    near(dg, dg_want, dg_size, "dg", 16 * TOL)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("Dk,Dv,L", [(64, 64, 2), (64, 64, 150), (128, 128, 65), (40, 72, 64), (33, 100, 100)])
def test_two_growing_steps_from_an_empty_state(dtype, Dk, Dv, L):
    """e^60 twice: the first has nothing to grow."""
    x = inputs(1, 2, 1, 2, L, Dk, Dv, TYPES[dtype], s0=False)
    x["g"][:, :, :2] = 60.0
    # (the gradient before the first step is e^120 of itself and more than fp32
    # holds: a decay of the first step that empties the state takes it away)
    check(x, f"first two of {L}, forward", backward=False)
    x["g"][:, :, 0] = NONE
    x["g"][:, :, 1] = 70.0
    check(x, f"one of e^70, {L}")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("Dk,Dv", [(64, 64), (128, 100)])
@pytest.mark.parametrize("gate,first,last", [(3.0, 10, 60), (60.0, 70, 73), (1.5, 5, 140), (100.0, 20, 21), (600.0, 64, 66),
                                             (0.5, 1, 149)])
def test_growth_where_nothing_is_kept(dtype, Dk, Dv, gate, first, last):
    """Steps first .. last grow a state that is empty and whose keys and gradients
    are zero, while queries and values go on as ever."""
    x = inputs(2, 1, 1, 2, 150, Dk, Dv, TYPES[dtype])
    x["g"][:, :, first:last + 1] = gate
    x["g"][:, :, first] = NONE
    if last + 1 < 150:
        x["g"][:, :, last + 1] = NONE
    else:
        x["ds"] = torch.zeros_like(x["ds"])
    for name in ("k", "do"):
        x[name][:, :, first:last + 1] = 0
    check(x, f"gates {gate} at {first} to {last}")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("Dk,Dv", [(64, 64), (128, 128)])
def test_values_and_keys_that_meet_zeros(dtype, Dk, Dv):
    """Values without keys and keys without values before e^120, and after it
    the first that are both there."""
    x = inputs(3, 1, 1, 2, 130, Dk, Dv, TYPES[dtype], s0=False)
    x["g"][:, :, :40] = 3.0
    x["k"][:, :, 0:40:2] = 0
    x["v"][:, :, 1:40:2] = 0
    check(x, "keys and values in turn", backward=False)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("Dk,Dv", [(64, 64), (128, 128)])
def test_a_tiny_state(dtype, Dk, Dv):
    """1e-30 times e^120."""
    x = inputs(4, 1, 1, 2, 130, Dk, Dv, TYPES[dtype])
    x["s0"] *= 1e-30
    x["g"][:, :, :2] = 60.0
    x["k"][:, :, :2] = 0
    check(x, "a state of 1e-30", backward=False)


@pytest.mark.parametrize("dtype", TYPES)
def test_heads_that_grow(dtype):
    """A fixed growth of every step, 0.9 over 80 steps and 1 over 70, and beside it a
    decay."""
    for L, g in ((80, 0.9), (70, 1.0)):
        x = inputs(5, 2, 1, 2, L, 64, 48, TYPES[dtype], s0=False, gates="heads")
        x["g"] = torch.tensor([g, -0.1], device=DEV)
        check(x, f"heads that grow by {g}")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("gate", [0.3, 3.0])
@pytest.mark.parametrize("Dk,Dv", [(64, 64), (128, 128)])
def test_growth_over_segments(dtype, gate, Dk, Dv):
    """Many chunks of a cut sequence that grow an empty state: 0.3 a step is e^19
    a chunk and e^190 together, 3 a step e^192 in each chunk."""
    L = 64 * 24 + 5
    x = inputs(6, 1, 1, 1, L, Dk, Dv, TYPES[dtype])
    assert pk.pdssm_linear_workspace_bytes(1, 1, 1, L, Dk, Dv, int(dtype == "bf16")) > 256
    first, last = 64 * 7 + 9, 64 * 17 + 30
    x["g"] = x["g"] - 0.05
    x["g"][:, :, first:last + 1] = gate
    x["g"][:, :, first] = x["g"][:, :, last + 1] = NONE
    for name in ("k", "do"):
        x[name][:, :, first:last + 1] = 0
    check(x, f"gates {gate} over segments")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("L,spread", [(150, 0.5), (150, 1.0), (150, 2.0), (150, 3.0), (1541, 0.5), (1541, 1.0), (1541, 2.0)])
def test_gates_of_both_signs(dtype, spread, L):
    """Positive gates of a chunk add up to about 13, 25, 50 and 75 and the negative
    ones to as much; a drift down keeps the longer sequence where it is.  (Of 3.0
    over 1541 steps |S| |dS| reaches 3.5e39, which dg needs below 3.4e38.)"""
    x = inputs(10, 1, 1, 2, L, 64, 40, TYPES[dtype])
    gen = torch.Generator().manual_seed(11)
    x["g"] = (spread * torch.randn(1, 2, L, generator=gen) - (0.0 if L < 200 else 0.1)).to(DEV)
    check(x, f"gates of {spread} and both signs, {L}")


@pytest.mark.parametrize("dtype", TYPES)
def test_growth_over_the_chunks_of_a_segment(dtype):
    """Segments of many chunks (there are many heads), each chunk of e^19 and the
    segment above what fp32 holds."""
    L, H = 64 * 40, 40
    x = inputs(9, 1, H, H, L, 16, 8, TYPES[dtype])
    assert pk.pdssm_linear_workspace_bytes(1, H, H, L, 16, 8, int(dtype == "bf16")) > 256
    first, last = 64 * 3 + 9, 64 * 36 + 30
    x["g"] = x["g"] - 0.05
    x["g"][:, :, first:last + 1] = 0.3
    x["g"][:, :, first] = x["g"][:, :, last + 1] = NONE
    for name in ("k", "do"):
        x[name][:, :, first:last + 1] = 0
    check(x, "gates 0.3 over many chunks")


@pytest.mark.parametrize("dtype", TYPES)
def test_gates_of_both_signs_over_segments(dtype):
    """Segments of many chunks of which some grow, with states that live on: the
    segments' decays as products of both."""
    L, H = 64 * 40, 40
    x = inputs(12, 1, H, H, L, 16, 24, TYPES[dtype])
    assert pk.pdssm_linear_workspace_bytes(1, H, H, L, 16, 24, int(dtype == "bf16")) > 256
    gen = torch.Generator().manual_seed(13)
    g = 3.0 * torch.randn(1, H, L, generator=gen) - 1.2
    assert (g.clamp_min(0).unflatten(2, (-1, 64)).sum(-1) > 60).float().mean() > 0.02
    x["g"] = g.to(DEV)
    check(x, "gates of both signs over segments")


@pytest.mark.parametrize("dtype", TYPES)
def test_growing_steps(dtype):
    """Single steps: e^100 of nothing, of 1e-20, and e^1000 of nothing."""
    x = inputs(7, 3, 1, 2, 1, 128, 100, TYPES[dtype])
    x["s0"][0] = x["s0"][2] = 0
    x["s0"][1] *= 1e-20
    x["g"][0], x["g"][1], x["g"][2] = 100.0, 100.0, 1000.0
    y = {**x, "g": x["g"].clone()}
    y["g"][2] = 0.0                     # (64 bits do not hold e^1000 either)
    want_o, want_s, _ = ref.linear(*(y[n] for n in STEPS), y["s0"])
    s = x["s0"].clone()
    o = pk.linear_attention_step(*(x[n][:, :, 0] for n in STEPS), s)
    o2, s2 = pk.linear_attention(*(x[n] for n in STEPS), x["s0"])
    torch.cuda.synchronize()
    size = want_s.norm(dim=(-2, -1))
    for name, got, state in (("step", o, s), ("forward", o2[:, :, 0], s2)):
        near(got, want_o[:, :, 0], 128 ** -0.5 * heads(length(x["q"]), 2)[:, :, 0] * size[..., None], name)
        near(state, want_s, size[..., None, None], name + "'s state")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("name,value", [("q", float("nan")), ("k", float("nan")), ("v", float("inf")), ("g", float("nan")),
                                        ("g", float("inf"))])
@pytest.mark.parametrize("L,at", [(200, 5), (200, 130), (64 * 24 + 5, 700)])
def test_what_is_not_finite_beside_growth(dtype, name, value, L, at):
    """In walks that are done step by step: from its step on, in the rows and
    columns of the state that it reaches, and nowhere else."""
    x = inputs(14, 2, 1, 2, L, 64, 48, TYPES[dtype])
    x["g"][:, :, 80:84] = 40.0
    x["g"][:, :, 80] = x["g"][:, :, 84] = NONE
    x["k"][:, :, 80:84] = 0
    say(f"[case] {name} = {value} at {at} of {L}")
    o, s = pk.linear_attention(*(x[n] for n in STEPS), x["s0"])
    y = x[name].clone()
    y[(1, 0, at) if name == "g" else (1, 0, at, 3)] = value
    bad, bad_s = pk.linear_attention(*({**x, name: y}[n] for n in STEPS), x["s0"])
    torch.cuda.synchronize()
    assert torch.isfinite(o).all() and torch.isfinite(s).all()
    reached, state = torch.zeros_like(o, dtype=torch.bool), torch.zeros_like(s, dtype=torch.bool)
    if name == "q":
        reached[1, :, at] = True
    elif name == "v":
        reached[1, 0, at:, 3] = state[1, 0, :, 3] = True
    else:
        both = slice(0, 2 if name == "k" else 1)
        reached[1, both, at:] = True
        state[1, both, 3 if name == "k" else slice(None)] = True
    assert torch.equal(bad[~reached], o[~reached]) and not torch.isfinite(bad[reached]).any()
    assert torch.equal(bad_s[~state], s[~state]) and not torch.isfinite(bad_s[state]).any()


def test_growth_in_place_reproducible_and_on_a_stream():
    """Growth with states in place, from whatever the workspace holds, on a given
    stream, captured and replayed: the same bits."""
    L = 64 * 24
    x = inputs(8, 1, 1, 2, L, 128, 128, torch.bfloat16)
    x["g"][:, :, 700:900] = 2.0
    x["g"][:, :, 700] = x["g"][:, :, 900] = NONE
    x["k"][:, :, 700:900] = 0
    x["do"][:, :, 700:900] = 0
    args = [x[n] for n in STEPS]
    want = [*pk.linear_attention(*args, x["s0"]), *pk.linear_attention_bwd(*args, x["do"], x["s0"], x["ds"])]
    torch.cuda.synchronize()
    assert all(torch.isfinite(t).all() for t in want)
    side = torch.cuda.Stream()
    fwd, bwd = (torch.full((f(1, 1, 2, L, 128, 128, 1),), 255, dtype=torch.uint8, device=DEV)
                for f in (pk.pdssm_linear_workspace_bytes, pk.pdssm_linear_bwd_workspace_bytes))
    o, s, ds = torch.empty_like(want[0]), x["s0"].clone(), x["ds"].clone()
    out = [torch.empty_like(t) for t in want[2:6]]

    def call(**kw):
        pk.linear_attention(*args, s, o=o, s_final=s, workspace=fwd, **kw)
        pk.linear_attention_bwd(*args, x["do"], x["s0"], ds, out=(*out, ds), workspace=bwd, **kw)

    torch.cuda.synchronize()
    call(stream=side)
    side.synchronize()
    for a, b in zip((o, s, *out, ds), want):
        assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for _ in range(3):
        s.copy_(x["s0"])
        ds.copy_(x["ds"])
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip((o, s, *out, ds), want):
            assert torch.equal(a, b)

"""The gated delta rule on the GPU (forward, gradients, single step) against
the 64-bit step-by-step reference.

Tolerances, fixed beforehand.  fp32 results: every product is held to 2^-24
and summed over at most Dk + 64 = 192 terms in fp32 inside a chunk, and the
errors of earlier chunks do not grow (keys of unit length): 192 * 2^-24 =
1.2e-5 in the worst case, 2e-5 of the result's norm.  bf16 results: the
rounding is at most 2^-8 of a value (8 bits, rounded to nearest); o and dv add
terms of 16 bits (2^-16), dq and dk one more rounding of 2^-8 inside the chunk:
2^-8 + 1e-4 and 2^-7 of the norm.  dg is a sum of up to 64 differences q . dq - v . dv, so its error is
measured against its own norm plus sqrt(64) times that of the terms."""
from __future__ import annotations

import sys

import pytest
import torch

import structured_sparse_state_amd as pk
from tests import layers_reference as ref

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
TOL_F32, TOL_OUT, TOL_KEYS = 2e-5, 2.0 ** -8 + 1e-4, 2.0 ** -7


def say(msg):
    print(msg, flush=True)
    sys.stdout.flush()


def off(got, want):
    got, want = got.double().cpu(), want.double()
    assert got.shape == want.shape and torch.isfinite(got).all()
    n = want.norm()
    return float((got - want).norm() / n) if n > 0 else float(got.norm())


def inputs(seed, B, Hk, Hv, L, Dk, Dv, dtype, s0=True, order="head", gates="plain"):
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=gen)  # noqa: E731
    unit = lambda x: x / x.norm(dim=-1, keepdim=True).clamp_min(1e-6)  # noqa: E731
    q, k = unit(r(B, Hk, L, Dk)), unit(r(B, Hk, L, Dk) + 0.5 * r(B, Hk, 1, Dk))
    v, do = r(B, Hv, L, Dv), r(B, Hv, L, Dv)
    g, beta = -0.2 * r(B, Hv, L).abs(), torch.sigmoid(r(B, Hv, L))
    if gates == "none":
        g = torch.zeros_like(g)
    elif gates == "strong":
        g = 60 * g
    elif gates == "growing":
        g = 0.02 * r(B, Hv, L)
    elif gates == "edges":      # beta of 0, 1, 2 and below 0
        beta = torch.tensor([0.0, 1.0, 2.0, -0.5])[torch.randint(0, 4, beta.shape, generator=gen)]
    elif gates == "empty":      # steps that empty the state, the first and the last among them
        g = torch.where(torch.rand(g.shape, generator=gen) < 0.06, -float("inf"), g)
        g[..., 0] = g[..., -1] = -float("inf")
    x = {"q": q.to(dtype), "k": k.to(dtype), "v": v.to(dtype), "do": do.to(dtype), "g": g, "beta": beta,
         "s0": 0.3 * r(B, Hv, Dk, Dv) if s0 else None, "ds": 0.3 * r(B, Hv, Dk, Dv) if s0 else None}
    return {n: t if t is None else place(t.to(DEV), order if n not in ("s0", "ds") else "head") for n, t in x.items()}


def place(t, order):
    """The same values held in another way."""
    if order == "head":
        return t.contiguous()
    if order == "token":
        return t.transpose(1, 2).contiguous().transpose(1, 2)
    if order == "apart":        # rows off every 16-byte boundary, gaps between all of them
        wide = [n + 3 for n in t.shape]
        base = torch.full(wide, float("nan"), dtype=t.dtype, device=t.device)
        cut = base[tuple(slice(1, n + 1) for n in t.shape)]
        cut.copy_(t)
        return cut
    raise ValueError(order)


def check_fwd(x, label, **kw):
    say(f"[case] forward {label}")
    want_o, want_s, _ = ref.delta(x["q"], x["k"], x["v"], x["g"], x["beta"], x["s0"], **kw)
    o, s = pk.delta_rule(x["q"], x["k"], x["v"], x["g"], x["beta"], x["s0"], **kw)
    torch.cuda.synchronize()
    f32 = o.dtype == torch.float32
    eo, es = off(o, want_o), off(s, want_s)
    say(f"  o {eo:.2e} s {es:.2e}")
    assert eo <= (TOL_F32 if f32 else TOL_OUT) and es <= TOL_F32
    return o, s


def check_bwd(x, label, **kw):
    say(f"[case] backward {label}")
    want, terms = ref.delta_bwd(x["q"], x["k"], x["v"], x["g"], x["beta"], x["do"], x["s0"], x["ds"], **kw)
    got = pk.delta_rule_bwd(x["q"], x["k"], x["v"], x["g"], x["beta"], x["do"], x["s0"], x["ds"], **kw)
    torch.cuda.synchronize()
    f32 = x["q"].dtype == torch.float32
    tols = [TOL_F32] * 6 if f32 else [TOL_KEYS, TOL_KEYS, TOL_OUT, TOL_F32, TOL_F32, TOL_F32]
    for name, a, b, tol in zip(("dq", "dk", "dv", "dg", "dbeta", "ds0"), got, want, tols):
        if name == "dg":
            assert torch.isfinite(a).all()
            e = float((a.double().cpu() - b).norm() / (b.norm() + 8 * terms.norm() + 1e-30))
        else:
            e = off(a, b)
        say(f"  {name} {e:.2e}")
        assert e <= tol, name
    return got


TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("L", [1, 2, 15, 17, 63, 64, 65, 129, 200])
def test_lengths(dtype, L):
    x = inputs(L, 2, 1, 2, L, 48, 40, TYPES[dtype])
    check_fwd(x, f"L={L}")
    check_bwd(x, f"L={L}")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("Dk,Dv", [(1, 1), (8, 8), (3, 128), (128, 5), (64, 64), (65, 33), (96, 72), (128, 128)])
def test_head_sizes(dtype, Dk, Dv):
    x = inputs(Dk + Dv, 1, 1, 2, 70, Dk, Dv, TYPES[dtype])
    check_fwd(x, f"Dk={Dk} Dv={Dv}")
    check_bwd(x, f"Dk={Dk} Dv={Dv}")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("Hk,Hv", [(1, 1), (2, 4), (1, 3), (3, 3)])
def test_shared_heads(dtype, Hk, Hv):
    """Gradients of a query and key head that several value heads share."""
    x = inputs(Hk * 10 + Hv, 2, Hk, Hv, 90, 64, 64, TYPES[dtype], s0=False)
    check_fwd(x, f"Hk={Hk} Hv={Hv}")
    check_bwd(x, f"Hk={Hk} Hv={Hv}")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("gates", ["none", "strong", "growing", "edges", "empty"])
def test_gates(dtype, gates):
    x = inputs(7, 1, 2, 2, 150, 64, 32, TYPES[dtype], gates=gates)
    check_fwd(x, gates)
    _, _, _, dg, _, _ = check_bwd(x, gates)
    if gates == "empty":
        assert (dg[torch.isinf(x["g"])] == 0).all()


def test_a_step_that_empties_the_state_starts_anew():
    """Two documents in one sequence give what each gives alone."""
    x = inputs(9, 1, 1, 2, 100, 64, 64, torch.bfloat16, s0=False)
    x["g"][:, :, 37] = -float("inf")
    o, s = pk.delta_rule(x["q"], x["k"], x["v"], x["g"], x["beta"])
    second = [x[n][:, :, 37:].contiguous() for n in ("q", "k", "v", "g", "beta")]
    o2, s2 = pk.delta_rule(*second)
    torch.cuda.synchronize()
    assert off(o[:, :, 37:].float(), o2.float().cpu()) <= 2 * TOL_OUT and off(s, s2.cpu()) <= TOL_F32


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
    want, _, _ = ref.delta(x["q"], x["k"], x["v"], x["g"], x["beta"], x["s0"])
    grads, _ = ref.delta_bwd(x["q"], x["k"], x["v"], x["g"], x["beta"], x["do"], x["s0"], x["ds"])
    base = torch.full((2, 73, 5, 29), 7.0, dtype=torch.bfloat16, device=DEV)
    o = base[:, 2:72, 1:3, 3:27].transpose(1, 2)
    s = x["s0"].clone()
    pk.delta_rule(x["q"], x["k"], x["v"], x["g"], x["beta"], s, o=o, s_final=s)
    out = [torch.empty_like(x[n]) for n in ("q", "k")] + [o] + [torch.empty_like(x[n]) for n in ("g", "beta")]
    torch.cuda.synchronize()
    assert off(o.float(), want) <= TOL_OUT
    ds = x["ds"].clone()
    pk.delta_rule_bwd(x["q"], x["k"], x["v"], x["g"], x["beta"], x["do"], x["s0"], ds, out=(*out, ds))
    torch.cuda.synchronize()
    assert off(o.float(), grads[2]) <= TOL_OUT and off(ds, grads[5]) <= TOL_F32
    base[:, 2:72, 1:3, 3:27] = 7.0
    assert (base == 7.0).all()


@pytest.mark.parametrize("dtype", TYPES)
def test_broadcast_inputs(dtype):
    """One query row for all steps, one key head for all batches (strides of 0)."""
    x = inputs(5, 2, 1, 2, 80, 64, 32, TYPES[dtype])
    x["q"] = x["q"][:, :, :1].expand(2, 1, 80, 64)
    x["k"] = x["k"][:1].expand(2, 1, 80, 64)
    x["do"] = x["do"][:, :, :1].expand(2, 2, 80, 32)
    check_fwd(x, "broadcast")
    out = [torch.empty(t.shape, dtype=t.dtype, device=DEV) for t in (x["q"], x["k"], x["v"], x["g"], x["beta"], x["s0"])]
    pk.delta_rule_bwd(x["q"], x["k"], x["v"], x["g"], x["beta"], x["do"], x["s0"], x["ds"], out=out)
    want, _ = ref.delta_bwd(x["q"], x["k"], x["v"], x["g"], x["beta"], x["do"], x["s0"], x["ds"])
    torch.cuda.synchronize()
    for a, b, tol in zip(out[:3], want, (TOL_KEYS, TOL_KEYS, TOL_OUT)):
        assert off(a.float(), b) <= (tol if dtype == "bf16" else TOL_F32)


@pytest.mark.parametrize("Dk,Dv", [(64, 64), (128, 128), (40, 72)])
def test_long_sequences_of_few_heads(Dk, Dv):
    """Sequences long enough to be walked in segments, in both directions."""
    x = inputs(Dk, 1, 1, 2, 64 * 40 + 5, Dk, Dv, torch.bfloat16, order="token")
    assert pk.pdssm_delta_workspace_bytes(1, 1, 2, 2565, Dk, Dv, 1) > 41 * 2 * 22528     # it has segments
    check_fwd(x, f"long Dk={Dk}")
    check_bwd(x, f"long Dk={Dk}")


def test_gradient_against_differences():
    """The GPU's gradients along random directions against central differences
    of the 64-bit reference's loss."""
    x = inputs(11, 1, 1, 2, 40, 16, 16, torch.float32)
    got = pk.delta_rule_bwd(x["q"], x["k"], x["v"], x["g"], x["beta"], x["do"], x["s0"], x["ds"])
    y = {n: t.double().cpu() for n, t in x.items()}
    loss = lambda z: sum((a * b).sum() for a, b in zip(  # noqa: E731
        ref.delta(z["q"], z["k"], z["v"], z["g"], z["beta"], z["s0"])[:2], (y["do"], y["ds"])))
    gen = torch.Generator().manual_seed(1)
    for name, grad in zip(("q", "k", "v", "g", "beta", "s0"), got):
        d = torch.randn(y[name].shape, generator=gen, dtype=torch.float64)
        h = 1e-6
        diff = (loss({**y, name: y[name] + h * d}) - loss({**y, name: y[name] - h * d})) / (2 * h)
        along = (grad.double().cpu() * d).sum()
        assert abs(diff - along) <= 1e-4 * float(grad.double().norm()) * (d.numel() ** 0.5), name


def test_scale_and_no_state():
    x = inputs(12, 1, 1, 1, 30, 32, 32, torch.float32, s0=False)
    o, s = pk.delta_rule(x["q"], x["k"], x["v"], x["g"], x["beta"], scale=2.5, want_state=False)
    want, _, _ = ref.delta(x["q"], x["k"], x["v"], x["g"], x["beta"], scale=2.5)
    assert s is None and off(o, want) <= TOL_F32
    got = pk.delta_rule_bwd(x["q"], x["k"], x["v"], x["g"], x["beta"], x["do"], scale=2.5, want_ds0=False)
    want, _ = ref.delta_bwd(x["q"], x["k"], x["v"], x["g"], x["beta"], x["do"], scale=2.5)
    assert got[5] is None
    for a, b in zip(got[:3], want):
        assert off(a, b) <= TOL_F32


def test_empty_shapes():
    for B, Hv, L in ((0, 2, 5), (2, 0, 5), (2, 2, 0)):
        q = torch.zeros(B, Hv, L, 8, device=DEV)
        g = torch.zeros(B, Hv, L, device=DEV)
        s0 = torch.randn(B, Hv, 8, 8, device=DEV)
        o, s = pk.delta_rule(q, q, q, g, g, s0)
        assert o.shape == q.shape and torch.equal(s, s0)
        assert torch.equal(pk.delta_rule(q, q, q, g, g)[1], torch.zeros_like(s0))
        grads = pk.delta_rule_bwd(q, q, q, g, g, q, s0, s0)
        assert torch.equal(grads[5], s0)


@pytest.mark.parametrize("L", [150, 64 * 40])
def test_results_are_reproducible_whatever_the_workspace_holds(L):
    x = inputs(13, 1, 1, 2, L, 64, 64, torch.bfloat16)
    need = pk.pdssm_delta_bwd_workspace_bytes(1, 1, 2, L, 64, 64, 1)
    results = []
    for fill in (0, 255):       # 255: NaN in every word
        ws = torch.full((need,), fill, dtype=torch.uint8, device=DEV)
        results.append(list(pk.delta_rule(x["q"], x["k"], x["v"], x["g"], x["beta"], x["s0"], workspace=ws))
                       + list(pk.delta_rule_bwd(x["q"], x["k"], x["v"], x["g"], x["beta"], x["do"], x["s0"], x["ds"],
                                                workspace=ws)))
    torch.cuda.synchronize()
    for a, b in zip(*results):
        assert torch.equal(a, b)


def test_not_a_number_stays_in_its_sequence_and_behind_its_chunk():
    x = inputs(14, 2, 1, 2, 200, 64, 64, torch.bfloat16)
    o, s = pk.delta_rule(x["q"], x["k"], x["v"], x["g"], x["beta"], x["s0"])
    for name in ("v", "k", "beta"):
        y = {**x, name: x[name].clone()}
        y[name][0, 0, 130] = float("nan") if name != "v" else float("inf")
        bad, bad_s = pk.delta_rule(y["q"], y["k"], y["v"], y["g"], y["beta"], y["s0"])
        torch.cuda.synchronize()
        assert torch.equal(bad[0, :, :128], o[0, :, :128]) and torch.equal(bad[1], o[1]), name
        assert torch.equal(bad_s[1], s[1]) and not torch.isfinite(bad_s[0, 0]).all(), name


def test_another_stream():
    x = inputs(15, 1, 2, 2, 300, 64, 64, torch.bfloat16)
    want = list(pk.delta_rule(x["q"], x["k"], x["v"], x["g"], x["beta"], x["s0"]))
    want += list(pk.delta_rule_bwd(x["q"], x["k"], x["v"], x["g"], x["beta"], x["do"], x["s0"], x["ds"]))
    torch.cuda.synchronize()
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        got = list(pk.delta_rule(x["q"], x["k"], x["v"], x["g"], x["beta"], x["s0"]))
    ws = torch.empty(pk.pdssm_delta_bwd_workspace_bytes(1, 2, 2, 300, 64, 64, 1), dtype=torch.uint8, device=DEV)
    out = [torch.empty_like(t) for t in (x["q"], x["k"], x["v"], x["g"], x["beta"], x["s0"])]
    torch.cuda.synchronize()
    got += list(pk.delta_rule_bwd(x["q"], x["k"], x["v"], x["g"], x["beta"], x["do"], x["s0"], x["ds"], out=out,
                                  workspace=ws, stream=stream))
    stream.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_graph_replays():
    """A captured forward and step, replayed with other inputs in between."""
    x = inputs(16, 2, 2, 2, 100, 64, 64, torch.bfloat16)
    ws = torch.empty(pk.pdssm_delta_workspace_bytes(2, 2, 2, 100, 64, 64, 1), dtype=torch.uint8, device=DEV)
    o, s = torch.empty_like(x["v"]), torch.empty_like(x["s0"])
    first = [x[n][:, :, 0].contiguous() for n in ("q", "k", "v", "g", "beta")]
    so = torch.empty_like(first[2])
    state = x["s0"].clone()
    call = lambda: pk.delta_rule(x["q"], x["k"], x["v"], x["g"], x["beta"], x["s0"], o=o, s_final=s, workspace=ws)  # noqa: E731
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
        pk.delta_step(*first, state, o=so)
    for n in range(3):
        x["v"].copy_(torch.randn(x["v"].shape, device=DEV))
        state.copy_(x["s0"])
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        eager = pk.delta_rule(x["q"], x["k"], x["v"], x["g"], x["beta"], x["s0"])
        stepped = x["s0"].clone()
        eager_o = pk.delta_step(*first, stepped)
        torch.cuda.synchronize()
        assert torch.equal(o, eager[0]) and torch.equal(s, eager[1])
        assert torch.equal(so, eager_o) and torch.equal(state, stepped)


def test_offsets_beyond_32_bits():
    """A batch stride of more than 2^32 bytes."""
    far = (1 << 31) + 64
    base = torch.empty(far + 64 * 70, dtype=torch.bfloat16, device=DEV)
    x = inputs(17, 2, 1, 1, 70, 64, 64, torch.bfloat16)
    v = base.as_strided((2, 1, 70, 64), (far, 70 * 64, 64, 1))
    v.copy_(x["v"])
    x["v"] = v
    o = torch.empty(2, 1, 70, 64, dtype=torch.bfloat16, device=DEV)
    want, _, _ = ref.delta(x["q"], x["k"], v, x["g"], x["beta"], x["s0"])
    pk.delta_rule(x["q"], x["k"], v, x["g"], x["beta"], x["s0"], o=o)
    torch.cuda.synchronize()
    assert off(o.float(), want) <= TOL_OUT


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("B,Hk,Hv,Dk,Dv", [(1, 1, 1, 1, 1), (3, 2, 4, 64, 64), (2, 1, 3, 128, 128), (1, 2, 2, 65, 33),
                                           (2, 2, 2, 7, 128), (300, 1, 1, 16, 20)])
def test_step(dtype, B, Hk, Hv, Dk, Dv):
    x = inputs(B + Dk, B, Hk, Hv, 3, Dk, Dv, TYPES[dtype], gates="empty")
    say(f"[case] step B={B} Hk={Hk} Hv={Hv} Dk={Dk} Dv={Dv}")
    want_o, want_s, states = ref.delta(x["q"], x["k"], x["v"], x["g"], x["beta"], x["s0"])
    s = x["s0"].clone()
    for t in range(3):
        args = [x[n][:, :, t] for n in ("q", "k", "v", "g", "beta")]     # views with the sequence's strides
        before = s.clone()
        apart = torch.full_like(s, float("nan"))
        o = pk.delta_step(*args, s)
        o2 = pk.delta_step(*args, before, s_out=apart)
        torch.cuda.synchronize()
        assert torch.equal(o, o2) and torch.equal(s, apart)
        assert off(o.float(), want_o[:, :, t]) <= (TOL_F32 if dtype == "f32" else TOL_OUT)
        assert off(s, states[t + 1]) <= TOL_F32


def test_steps_continue_a_sequence():
    """A prompt through the forward, then steps, against one long forward."""
    x = inputs(20, 2, 2, 4, 90, 64, 64, torch.bfloat16)
    o, s = pk.delta_rule(x["q"], x["k"], x["v"], x["g"], x["beta"], x["s0"])
    cut = {n: x[n][:, :, :70] for n in ("q", "k", "v", "g", "beta")}
    first, state = pk.delta_rule(*cut.values(), x["s0"])
    rest = [pk.delta_step(*(x[n][:, :, t] for n in ("q", "k", "v", "g", "beta")), state) for t in range(70, 90)]
    got = torch.cat([first, torch.stack(rest, 2)], 2)
    torch.cuda.synchronize()
    assert off(got.float(), o.float().cpu()) <= 2 * TOL_OUT and off(state, s.cpu()) <= 2 * TOL_F32

"""The layer operators on a stream given to the call, without any buffer from
the caller: memory that the call takes for itself is not handed to other
streams' work before the kernels have run."""
from __future__ import annotations

import pytest
import torch

import structured_sparse_state_amd as pk

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


def calls():
    gen = torch.Generator().manual_seed(31)
    r = lambda *s: torch.randn(s, generator=gen).to(DEV)  # noqa: E731
    B, Hk, Hv, L, D = 2, 2, 4, 300, 64
    q, k, v, do = (r(B, h, L, D).to(torch.bfloat16) / 8 for h in (Hk, Hk, Hv, Hv))
    g, beta, s0 = -r(B, Hv, L).abs(), torch.sigmoid(r(B, Hv, L)), r(B, Hv, D, D)
    first, after = [x[:, :, 0] for x in (q, k, v, g, beta)], torch.empty_like(s0)
    w, cos, sin = r(D), r(L, D // 2).cos(), r(L, D // 2).sin()
    flat = lambda x: [t for t in (x if isinstance(x, tuple) else (x,)) if t is not None]  # noqa: E731
    return {
        "delta_rule": lambda **kw: flat(pk.delta_rule(q, k, v, g, beta, s0, **kw)),
        "delta_rule_bwd": lambda **kw: flat(pk.delta_rule_bwd(q, k, v, g, beta, do, s0, s0, **kw)),
        "delta_step": lambda **kw: flat(pk.delta_step(*first, s0, s_out=after, **kw)),
        "qk_norm_rope": lambda **kw: flat(pk.qk_norm_rope(q, v, w, w, cos, sin, **kw)),
        "qk_norm_rope_bwd": lambda **kw: flat(pk.qk_norm_rope_bwd(q, v, q, do, w, w, cos, sin, **kw)),
    }


@pytest.mark.parametrize("handle", [False, True])
@pytest.mark.parametrize("name", ["delta_rule", "delta_rule_bwd", "delta_step", "qk_norm_rope", "qk_norm_rope_bwd"])
def test_memory_of_a_given_stream(name, handle):
    print(f"[case] {name} handle={handle}", flush=True)
    call = calls()[name]
    want = call()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.cuda._sleep(10_000_000)           # the call's kernels wait behind this
    got = call(stream=side.cuda_stream if handle else side)
    # Meanwhile the current stream takes and overwrites memory of every size.
    held = [torch.full((1 << n,), float("nan"), device=DEV) for n in range(8, 24) for _ in range(4)]
    side.synchronize()
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    for t in held:
        assert torch.isnan(t).all()


def test_the_default_stream_by_its_handle():
    call = calls()["delta_rule"]
    want, got = call(), call(stream=0)
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_given_buffers_and_a_stream():
    """With every buffer given a call allocates nothing, on any stream."""
    gen = torch.Generator().manual_seed(32)
    r = lambda *s: torch.randn(s, generator=gen).to(DEV)  # noqa: E731
    q, k, v = (r(1, 2, 90, 32) / 6 for _ in range(3))
    g, beta, s0 = -r(1, 2, 90).abs(), torch.sigmoid(r(1, 2, 90)), r(1, 2, 32, 32)
    first = [x[:, :, 0].contiguous() for x in (q, k, v, g, beta)]
    ws = torch.empty(pk.pdssm_delta_bwd_workspace_bytes(1, 2, 2, 90, 32, 32, 0), dtype=torch.uint8, device=DEV)
    o, s, x = torch.empty_like(v), torch.empty_like(s0), torch.empty_like(first[2])
    grads = tuple(torch.empty_like(t) for t in (q, k, v, g, beta, s0))
    nq, nk = torch.empty_like(q), torch.empty_like(k)
    calls = [lambda **kw: pk.delta_rule(q, k, v, g, beta, s0, o=o, s_final=s, workspace=ws, **kw),
             lambda **kw: pk.delta_rule_bwd(q, k, v, g, beta, v, s0, s0, out=grads, workspace=ws, **kw),
             lambda **kw: pk.delta_step(*first, s0, s_out=s, o=x, **kw),
             lambda **kw: pk.qk_norm_rope(q, k, out=(nq, nk), **kw),
             lambda **kw: pk.qk_norm_rope_bwd(q, k, v, v, out=(nq, nk), **kw)]
    side = torch.cuda.Stream()
    for call in calls:
        want = [t.clone() for t in call() if t is not None]
        torch.cuda.synchronize()
        before = torch.cuda.memory_stats()["allocation.all.allocated"]
        got = call(stream=side)
        assert torch.cuda.memory_stats()["allocation.all.allocated"] == before
        side.synchronize()
        for a, b in zip((t for t in got if t is not None), want):
            assert torch.equal(a, b)

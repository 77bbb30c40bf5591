"""The block's operators together as a layer uses them: the example block runs
and serves, its gradients are those of a 64-bit model of the block, and the
operators take part in calls on a given stream and in a stack of blocks."""
from __future__ import annotations

import importlib.util
import os

import pytest
import torch

import structured_sparse_state_amd as pk
from tests import block_reference as ref

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("linear_layer", os.path.join(ROOT, "examples", "linear_layer.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def test_runs_and_serves(example):
    losses, apart = example.main(B=2, L=100, steps=10)
    print(f"loss {losses[0]:.3f} -> {losses[-1]:.3f}, served {apart:.1e}", flush=True)
    assert len(losses) == 10 and all(x == x and x < 1e6 for x in losses)
    # the state keeps 24 bits; a bf16 output may round the other way (2^-8)
    assert apart < 2 * 2.0 ** -8


def test_gradients_of_the_block(example):
    """Through norm, projections, attention, dropout, residual and norm in fp32
    against autograd through the 64-bit definitions."""
    torch.manual_seed(1)
    B, L, W, Hk, Hv, D, p, seed = 2, 70, 48, 1, 2, 16, 0.25, 11
    r = lambda *s: torch.randn(s, device=DEV)  # noqa: E731
    x, w1, b1, w2, b2 = r(B, L, W), 1 + 0.1 * r(W), r(W), 1 + 0.1 * r(W), r(W)
    proj, out, rate = 0.2 * r((2 * Hk + Hv) * D, W), 0.2 * r(W, Hv * D), -0.1 - r(Hv).abs()
    dy = r(B, L, W)
    leaves = [x, w1, b1, w2, b2, proj, out, rate]
    for t in leaves:
        t.requires_grad_()
    y, h = example.AddNorm.apply(x, torch.zeros_like(x), w1, b1, 0.0, 0)
    heads = (y @ proj.T).unflatten(2, (2 * Hk + Hv, D)).transpose(1, 2)
    o = example.LinearAttention.apply(heads[:, :Hk], heads[:, Hk:2 * Hk], heads[:, 2 * Hk:], rate)
    z, _ = example.AddNorm.apply(o.transpose(1, 2).flatten(2) @ out.T, h, w2, b2, p, seed)
    got = torch.autograd.grad((z * dy).sum(), leaves)
    torch.cuda.synchronize()

    copies = [t.detach().cpu().double().requires_grad_() for t in leaves]
    x, w1, b1, w2, b2, proj, out, rate = copies
    y, h = ref.layer_norm(x, w1, b1)
    heads = (y @ proj.T).unflatten(2, (2 * Hk + Hv, D)).transpose(1, 2)
    o, _, _ = ref.linear(heads[:, :Hk], heads[:, Hk:2 * Hk], heads[:, 2 * Hk:], rate)
    z, _ = ref.layer_norm(o.transpose(1, 2).flatten(2) @ out.T, w2, b2, h, p=p, seed=seed)
    want = torch.autograd.grad((z * dy.cpu().double()).sum(), copies)
    # every stage is fp32 to at most 2e-5 of its norm (torch's products too), about
    # ten of them one behind the other
    for a, b in zip(got, want):
        assert (a.double().cpu() - b).norm() <= 2e-4 * b.norm()


def functions(example):
    gen = torch.Generator().manual_seed(41)
    r = lambda *s: torch.randn(s, generator=gen).to(DEV)  # noqa: E731
    need = lambda *ts: [t.requires_grad_() for t in ts]  # noqa: E731
    attention = need(*((r(2, 2, 70, 32) / 6).to(torch.bfloat16) for _ in range(3)), -r(2, 2, 70).abs())
    norm = need(r(2, 70, 32), r(2, 70, 32), r(32), r(32))
    return {"attention": (lambda: example.LinearAttention.apply(*attention), attention),
            "norm": (lambda: example.AddNorm.apply(*norm, 0.2, 3), norm)}


@pytest.mark.parametrize("name", ["attention", "norm"])
def test_the_gradient_of_a_sum(example, name):
    call, leaves = functions(example)[name]
    outs = call()
    outs = outs if isinstance(outs, tuple) else (outs,)
    want = torch.autograd.grad(outs, leaves, [torch.ones_like(o) for o in outs], retain_graph=True)
    got = torch.autograd.grad(sum(o.sum() for o in outs), leaves)
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_one_output_of_the_norm_unused(example):
    """Either output alone has a gradient (the other's is zero)."""
    call, leaves = functions(example)["norm"]
    y, h = call()
    only_h = torch.autograd.grad(h.sum(), leaves, retain_graph=True)
    only_y = torch.autograd.grad(y.square().sum(), leaves)
    assert torch.equal(only_h[1], torch.ones_like(only_h[1])) and (only_h[2] == 0).all()
    assert all(torch.isfinite(t).all() for t in only_y)


@pytest.mark.parametrize("name", ["attention", "norm"])
def test_no_second_gradient(example, name):
    call, leaves = functions(example)[name]
    outs = call()
    first = torch.autograd.grad(sum(o.float().square().sum() for o in (outs if isinstance(outs, tuple) else (outs,))),
                                leaves, create_graph=True)
    with pytest.raises(RuntimeError):
        first[0].float().square().sum().backward()
    torch.cuda.synchronize()


def calls():
    gen = torch.Generator().manual_seed(31)
    r = lambda *s: torch.randn(s, generator=gen).to(DEV)  # noqa: E731
    q, k = ((r(2, 2, 300, 64) / 8).to(torch.bfloat16) for _ in range(2))
    v, do = ((r(2, 4, 300, 64)).to(torch.bfloat16) for _ in range(2))
    g, s0 = -r(2, 4, 300).abs(), r(2, 4, 64, 64)
    long = [t[:1, :, :1].expand(1, -1, 64 * 20, -1).contiguous() for t in (q, k, v)]
    first, after = [t[:, :, 0] for t in (q, k, v, g)], torch.empty_like(s0)
    x, w = r(600, 264), r(264)
    flat = lambda x: [t for t in (x if isinstance(x, tuple) else (x,)) if t is not None]  # noqa: E731
    return {
        "linear_attention": lambda **kw: flat(pk.linear_attention(q, k, v, g, s0, **kw)),
        "linear_attention, cut": lambda **kw: flat(pk.linear_attention(*long, None, **kw)),
        "linear_attention_bwd": lambda **kw: flat(pk.linear_attention_bwd(q, k, v, g, do, s0, s0, **kw)),
        "linear_attention_step": lambda **kw: flat(pk.linear_attention_step(*first, s0, s_out=after, **kw)),
        "layer_norm": lambda **kw: flat(pk.layer_norm(x, w, w, residual=x, p=0.3, seed=2, **kw)),
        "layer_norm_bwd": lambda **kw: flat(pk.layer_norm_bwd(x, x, w, dh=x, want_db=True, p=0.3, seed=2, **kw)),
        "dropout": lambda **kw: flat(pk.dropout(x, 0.3, 2, **kw)),
    }


@pytest.mark.parametrize("handle", [False, True])
@pytest.mark.parametrize("name", ["linear_attention", "linear_attention, cut", "linear_attention_bwd", "linear_attention_step",
                                  "layer_norm", "layer_norm_bwd", "dropout"])
def test_memory_of_a_given_stream(name, handle):
    """Memory that a call takes for itself is not handed to other streams' work
    before its kernels have run."""
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


def test_two_calls_at_once():
    """The same operators on two streams side by side, each with memory of its own."""
    streams = [torch.cuda.Stream() for _ in range(2)]
    for name, call in calls().items():
        if name == "linear_attention_step":     # (its results are one buffer)
            continue
        want = call()
        torch.cuda.synchronize()
        got = []
        for s in streams:
            with torch.cuda.stream(s):
                got += [call() for _ in range(3)]
        torch.cuda.synchronize()
        for one in got:
            for a, b in zip(one, want):
                assert torch.equal(a, b), name


def test_a_stack_of_blocks():
    """Two blocks forward in bf16, the residual stream and every mask from one
    seed and offsets of their own, against the 64-bit definitions fed with the
    same rounded inputs stage by stage."""
    torch.manual_seed(5)
    B, L, W, H, D = 2, 130, 128, 2, 64
    x = torch.randn(B, L, W, device=DEV).to(torch.bfloat16)
    stream, branch = x, torch.zeros_like(x)
    decay = torch.tensor([-0.01, -0.3], device=DEV)
    for n in range(2):
        w, b = 1 + 0.1 * torch.randn(W, device=DEV), torch.randn(W, device=DEV)
        y, new = pk.layer_norm(branch, w, b, residual=stream, p=0.1, seed=9, offset=n)
        want_y, want_h = ref.layer_norm(branch, w, b, stream, p=0.1, seed=9, offset=n)
        torch.cuda.synchronize()
        assert ((new.double().cpu() - want_h).abs() <= 2.0 ** -8 * want_h.abs() + 1e-6).all()
        assert ((y.double().cpu() - want_y).abs() <= 2.0 ** -8 * want_y.abs() + 1e-4).all()
        heads = y.unflatten(2, (H, D)).transpose(1, 2)
        o, _ = pk.linear_attention(heads, heads, heads, decay)
        want_o, _, _ = ref.linear(heads, heads, heads, decay)
        torch.cuda.synchronize()
        assert float((o.double().cpu() - want_o).norm() / want_o.norm()) <= 2.0 ** -8 + 2e-5
        stream, branch = new, pk.dropout(o.transpose(1, 2).flatten(2), 0.2, 9, 100 + n)

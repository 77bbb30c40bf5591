"""Linear attention with workgroups of 128 columns of the state over cut
sequences, as few large heads of long bf16 sequences take them, and without cuts.

The sizes are checked against the library's rule on the CPU: `rule` says it in
Python, and the workspace's bytes, which follow from columns and segments, have to
agree.  Values are held to the tolerances of tests/test_gpu_linear.py for the
value heads of one query and key head, whose 64-bit reference takes a few
seconds; the states live over at most 71 chunks."""
from __future__ import annotations

import pytest
import torch

import structured_sparse_state_amd as pk
from tests import block_reference as ref
from tests.test_gpu_linear import DEV, STEPS, TINY, TOL_BF16, TOL_F32, check_dg, inputs, off, say

BF16 = torch.bfloat16
NAN = float("nan")


def rule(B, Hk, Hv, L, Dk, Dv, bwd, dg="steps"):
    """(columns, segments of each walk, workspace bytes) of a bf16 call."""
    heads, NC, up = B * Hv, -(-L // 64), lambda n, to: -(-n // to)  # noqa: E731
    padded = lambda D: 64 if D <= 64 else 128  # noqa: E731

    def columns(D, walks):
        return 64 if D <= 64 or walks * max(1, NC // 4) <= 256 else 128

    def cut(walks):
        segs = min(256 // walks, NC if bwd else NC // 2)
        if segs > 1:
            chunks = up(NC, segs)
            if 3 * chunks + 2 * (1 if bwd else 3) <= 2 * NC:
                return up(NC, chunks)
        return 1

    if bwd:
        SL = columns(max(Dk, Dv), heads * (up(Dk, 64) + up(Dv, 64)))
        segs = [cut(heads * (up(Dk, SL) + up(Dv, SL)))] * 2 + [cut(heads * up(Dk, 64))]
    else:
        SL = columns(Dv, heads * up(Dv, 64))
        segs = [cut(heads * up(Dv, SL))]
    rows = max(padded(Dk), padded(Dv))
    groups = (rows if bwd else padded(Dv)) // 16
    takes = [256]
    for n in segs:
        if n > 1:
            takes += [(n + 1) * heads * groups * rows * 64, n * heads * 8]
    if bwd:
        takes.append(heads * Dk * Dv * 4)
        if dg:
            takes += [NC * heads * groups * rows * 64, NC * heads * groups * 64 * 4]
            if Dk > 64 or dg == "heads":
                takes.append(heads * up(Dk, 64) * L * 4)
        if Hv > Hk:
            takes += 2 * [heads * L * up(Dk, 4) * 4 * 4]
    return SL, segs, sum(up(n, 256) * 256 for n in takes)


LONG = 64 * 70 + 5
CASES = {   # B, Hk, Hv, L, Dk, Dv, order, gates, s0; the value heads that are looked at
    "document": ((1, 4, 8, LONG, 128, 128, "token", "plain", True), (0, 3)),
    "document, rows apart, empty states": ((1, 4, 8, LONG, 100, 72, "apart", "empty", True), (0, 0)),
    "document, fixed decays": ((1, 4, 8, 64 * 70, 72, 128, "head", "heads", False), (0, 2)),
    "few keys": ((1, 2, 8, 64 * 70, 40, 128, "token", "strong", True), (0, 1)),
    "many heads": ((2, 8, 32, 64 * 12 + 1, 128, 128, "token", "plain", True), (1, 5)),
    "many heads, no gates": ((2, 16, 32, 64 * 13, 96, 120, "head", "none", True), (1, 15)),
}
WHOLE = {   # not cut
    "a filled device": ((8, 16, 32, 130, 128, 128, "token", "plain", True), (7, 15)),
    "a filled device, rows apart": ((8, 16, 32, 65, 65, 100, "apart", "empty", True), (0, 3)),
}


def test_sizes_take_128_columns_and_segments():
    for cases, is_cut in ((CASES, True), (WHOLE, False)):
        for name, ((B, Hk, Hv, L, Dk, Dv, _, gates, _), _) in cases.items():
            dg = {"none": None, "heads": "heads"}.get(gates, "steps")
            flags = {None: pk.PDSSM_NO_DG, "heads": pk.PDSSM_DG_HEADS, "steps": 0}[dg] | 1
            SL, segs, total = rule(B, Hk, Hv, L, Dk, Dv, False)
            assert SL == 128 and (segs[0] > 1) == is_cut, name
            assert total == pk.pdssm_linear_workspace_bytes(B, Hk, Hv, L, Dk, Dv, 1), name
            SL, segs, total = rule(B, Hk, Hv, L, Dk, Dv, True, dg)
            assert SL == 128 and (segs[0] > 1) == is_cut, name
            assert total == pk.pdssm_linear_bwd_workspace_bytes(B, Hk, Hv, L, Dk, Dv, flags), name
            _, _, total = rule(B, Hk, Hv, L, Dk, Dv, True, None)
            assert total == pk.pdssm_linear_bwd_workspace_bytes(B, Hk, Hv, L, Dk, Dv, 1 | pk.PDSSM_NO_DG), name


def part(x, b, hk, group):
    """What one query and key head of one sequence has to do with."""
    keys, values = (slice(b, b + 1), slice(hk, hk + 1)), (slice(b, b + 1), slice(hk * group, (hk + 1) * group))
    y = {n: x[n][keys] for n in ("q", "k")}
    for n in ("v", "do", "s0", "ds", "g"):
        t = x[n]
        y[n] = t if t is None else t[values[1]] if t.dim() == 1 else t[values]
    return y, keys, values


def check(x, b, hk):
    args = [x[n] for n in STEPS]
    o, s = pk.linear_attention(*args, x["s0"])
    got = pk.linear_attention_bwd(*args, x["do"], x["s0"], x["ds"])
    plain = pk.linear_attention_bwd(*args, x["do"], x["s0"], x["ds"], want_dg=False)
    torch.cuda.synchronize()
    for n in (0, 1, 2, 4):
        assert torch.isfinite(got[n]).all() and torch.equal(got[n], plain[n])
    assert torch.isfinite(o).all() and torch.isfinite(s).all()
    y, keys, values = part(x, b, hk, x["v"].shape[1] // x["q"].shape[1])
    args = [y[n] for n in STEPS]
    want_o, want_s, _ = ref.linear(*args, y["s0"])
    e = off(o[values], want_o), off(s[values], want_s)
    say(f"  o {e[0]:.2e} s {e[1]:.2e}")
    assert e[0] <= TOL_BF16 and e[1] <= TOL_F32
    want, size = ref.linear_bwd(*args, y["do"], y["s0"], y["ds"])
    for label, n, at in (("dq", 0, keys), ("dk", 1, keys), ("dv", 2, values), ("ds0", 4, values)):
        e = float((got[n][at].double().cpu() - want[n]).norm())
        say(f"  {label} {e / float(want[n].norm() + 1e-300):.2e}")
        assert e <= (TOL_F32 if n == 4 else TOL_BF16) * float(want[n].norm()) + TINY * want[n].numel() ** 0.5, label
    if y["g"] is not None:
        check_dg(got[3][values[1] if y["g"].dim() == 1 else values], want[3], size, y["g"])


@pytest.mark.gpu
@pytest.mark.parametrize("name", [*CASES, *WHOLE])
def test_against_the_definition(name):
    (B, Hk, Hv, L, Dk, Dv, order, gates, s0), (b, hk) = {**CASES, **WHOLE}[name]
    say(f"[case] {name}")
    check(inputs(L + Dk, B, Hk, Hv, L, Dk, Dv, BF16, order=order, gates=gates, s0=s0), b, hk)


@pytest.mark.gpu
@pytest.mark.parametrize("gate", [0.3, 3.0])
@pytest.mark.parametrize("name", ["document", "many heads", "a filled device"])
def test_growth_where_nothing_is_kept(name, gate):
    """Steps of the sequence's middle that grow an empty state whose keys and
    gradients are zero by more than fp32 holds."""
    (B, Hk, Hv, L, Dk, Dv, order, _, _), (b, hk) = {**CASES, **WHOLE}[name]
    say(f"[case] {name}, gates {gate}")
    x = inputs(L + 1, B, Hk, Hv, L, Dk, Dv, BF16, order=order)
    first, last = L // 4, L - L // 4
    x["g"][:, :, first:last] = gate
    x["g"][:, :, first] = x["g"][:, :, last] = -float("inf")
    for n in ("k", "do"):
        x[n][:, :, first:last] = 0
    check(x, b, hk)


@pytest.mark.gpu
def test_states_in_place():
    """s_final over s0 and ds0 over ds_final, bit for bit as elsewhere, whatever
    the workspace holds."""
    (B, Hk, Hv, L, Dk, Dv, order, gates, _), _ = CASES["document"]
    x = inputs(3, B, Hk, Hv, L, Dk, Dv, BF16, order=order, gates=gates)
    args = [x[n] for n in STEPS]
    want = [*pk.linear_attention(*args, x["s0"]), *pk.linear_attention_bwd(*args, x["do"], x["s0"], x["ds"])]
    for fill in (0, 255):
        fwd, bwd = (torch.full((f(B, Hk, Hv, L, Dk, Dv, 1),), fill, dtype=torch.uint8, device=DEV)
                    for f in (pk.pdssm_linear_workspace_bytes, pk.pdssm_linear_bwd_workspace_bytes))
        s, ds = x["s0"].clone(), x["ds"].clone()
        o, _ = pk.linear_attention(*args, s, s_final=s, workspace=fwd)
        out = [torch.empty_like(t) for t in want[2:6]]
        pk.linear_attention_bwd(*args, x["do"], x["s0"], ds, out=(*out, ds), workspace=bwd)
        torch.cuda.synchronize()
        for a, b in zip((o, s, *out, ds), want):
            assert torch.equal(a, b)


@pytest.mark.gpu
@pytest.mark.parametrize("at", [0, 2000, LONG - 1])
@pytest.mark.parametrize("name", ["q", "k", "v"])
def test_what_is_not_finite(name, at):
    """In a segment in the middle, the first and the last step: what is before
    it and beside it keeps its bits."""
    (B, Hk, Hv, L, Dk, Dv, order, gates, _), _ = CASES["document"]
    x = inputs(4, B, Hk, Hv, L, Dk, Dv, BF16, order=order, gates=gates)
    o, s = pk.linear_attention(*(x[n] for n in STEPS), x["s0"])
    y = {**x, name: x[name].clone()}
    y[name][0, 1, at, 70] = NAN
    bad, bad_s = pk.linear_attention(*(y[n] for n in STEPS), y["s0"])
    torch.cuda.synchronize()
    reached, state = torch.zeros_like(o, dtype=torch.bool), torch.zeros_like(s, dtype=torch.bool)
    if name == "q":
        reached[0, 2:4, at] = True
    elif name == "v":
        reached[0, 1, at:, 70] = state[0, 1, :, 70] = True
    else:
        reached[0, 2:4, at:] = state[0, 2:4, 70] = True
    assert torch.equal(bad[~reached], o[~reached]) and not torch.isfinite(bad[reached]).any()
    assert torch.equal(bad_s[~state], s[~state]) and not torch.isfinite(bad_s[state]).any()

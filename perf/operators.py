"""Measured cases of the gated delta rule and of the query/key norm with rotation.

Two operators of sequence layers that stand beside the PD-SSM scan:

* the gated delta rule.  Every value head holds a state S [Dk, Dv]; a step is
      S <- exp(g) S;  u = beta (v - S^T k);  S <- S + k u^T;  o = scale S^T q
  as the chunked forward of a whole sequence, its gradients, and the single
  recurrent step of decoding.  Hv value heads share Hk query/key heads in
  groups of Hv / Hk.
* the norm of every query and key head (RMS with a weight, or unit length)
  followed by the rotation of the first R dimensions by the angles of the
  token's position, and its gradients.

``run`` computes a pass in plain torch operations in 32 bits, or, with
``own``, through the package's entry points.
"""
import math
import random

import torch

own = False

DEV = "cuda"
DTYPE = {"bf16": torch.bfloat16, "f32": torch.float32}
CHUNK = 64


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # One user decoding: a single layer's states, where the call itself costs most.
        {"name": "step, one sequence", "op": "step", "B": 1, "Hk": 8, "Hv": 16, "Dk": 128, "Dv": 128,
         "type": "bf16"},
        # A serving batch decoding in step: every state read and written once.
        {"name": "step, batch of 128", "op": "step", "B": 128, "Hk": 16, "Hv": 32, "Dk": 128,
         "Dv": 128, "type": "bf16"},
        # A short prompt of ragged length at a small head size.
        {"name": "forward, short prompt", "op": "fwd", "B": 1, "Hk": 4, "Hv": 4, "L": 77, "Dk": 64,
         "Dv": 64, "type": "bf16", "order": "token", "s0": False},
        # The layer of the scan's main benchmark: 256 sequences of 4096 steps, heads of 64.
        {"name": "forward, LM layer", "op": "fwd", "B": 8, "Hk": 32, "Hv": 32, "L": 4096, "Dk": 64,
         "Dv": 64, "type": "bf16", "order": "head", "s0": False},
        # A long document continued from a state: few sequences, many steps, grouped heads.
        {"name": "forward, long document", "op": "fwd", "B": 1, "Hk": 4, "Hv": 8, "L": 18000,
         "Dk": 128, "Dv": 128, "type": "bf16", "order": "token", "s0": True},
        # A training step's backward, grouped heads of 128.
        {"name": "backward, LM layer", "op": "bwd", "B": 4, "Hk": 8, "Hv": 16, "L": 4096, "Dk": 128,
         "Dv": 128, "type": "bf16", "order": "token", "s0": False},
        # A gradient in 32 bits at odd sizes: time series, small heads of unlike width.
        {"name": "backward, odd sizes", "op": "bwd", "B": 3, "Hk": 2, "Hv": 2, "L": 333, "Dk": 40,
         "Dv": 72, "type": "f32", "order": "head", "s0": True},
        # One token per sequence of a serving batch, positions of its own for each.
        {"name": "norm, one token", "op": "norm", "B": 32, "Hq": 16, "Hk": 4, "L": 1, "D": 128, "R": 128,
         "type": "bf16", "kind": "rms", "pairs": "half", "pos": True},
        # Prefill or training forward of one layer, queries and keys as one projection gives them.
        {"name": "norm, LM layer", "op": "norm", "B": 8, "Hq": 32, "Hk": 8, "L": 4096, "D": 128,
         "R": 128, "type": "bf16", "kind": "rms", "pairs": "half", "pos": False},
        # Unit-length queries and keys for the delta rule in 32 bits, odd length and head size.
        {"name": "norm, odd sizes", "op": "norm", "B": 2, "Hq": 6, "Hk": 3, "L": 1001, "D": 72, "R": 20,
         "type": "f32", "kind": "l2", "pairs": "adjacent", "pos": True},
        # Backward of the layer, half of each head rotated in adjacent pairs.
        {"name": "norm backward, LM layer", "op": "norm_bwd", "B": 8, "Hq": 32, "Hk": 8, "L": 4096,
         "D": 128, "R": 64, "type": "bf16", "kind": "rms", "pairs": "adjacent", "pos": False},
        # Backward of a small batch of ragged length.
        {"name": "norm backward, ragged", "op": "norm_bwd", "B": 3, "Hq": 8, "Hk": 8, "L": 517, "D": 64,
         "R": 64, "type": "bf16", "kind": "l2", "pairs": "half", "pos": True},
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["step", "fwd", "fwd", "bwd", "bwd", "norm", "norm_bwd"])
    kind = {"op": op, "type": rng.choice(["bf16", "bf16", "bf16", "f32"])}
    if op == "step":
        hk = rng.choice([1, 2, 4, 8, 16])
        return {**kind, "B": _spread(rng, 1, 128), "Hk": hk, "Hv": hk * rng.choice([1, 2]),
                "Dk": rng.choice([64, 128, 128, rng.randint(16, 128)]),
                "Dv": rng.choice([64, 128, 128, rng.randint(16, 128)])}
    if op in ("fwd", "bwd"):
        B, hk, group = _spread(rng, 1, 8), rng.choice([1, 2, 3, 4, 8]), rng.choice([1, 1, 2, 4])
        D = rng.choice([64, 128])
        Dk, Dv = (D, D) if rng.random() < 0.6 else (rng.randint(16, 128), rng.randint(16, 128))
        # no more steps in all than the largest listed case of the direction
        most = (144000 if op == "fwd" else 262144) // (2 if kind["type"] == "f32" else 1)
        return {**kind, "B": B, "Hk": hk, "Hv": hk * group,
                "L": _spread(rng, 1, max(2, min(18000 if op == "fwd" else 4096, most // (B * hk * group)))),
                "Dk": Dk, "Dv": Dv, "order": rng.choice(["token", "head"]), "s0": rng.random() < 0.5}
    hk, D = rng.choice([1, 2, 4, 8]), rng.choice([64, 128, 256, 2 * rng.randint(8, 128)])
    B, hq = _spread(rng, 1, 32), hk * rng.choice([1, 2, 4])
    most = 8 * 40 * 4096 * 128 // (D * (hq + hk) * B * (2 if kind["type"] == "f32" else 1))
    return {**kind, "B": B, "Hq": hq, "Hk": hk, "L": _spread(rng, 1, max(1, min(16384, most))), "D": D,
            "R": rng.choice([0, D, D // 4 * 2, 2 * rng.randint(1, D // 2)]), "kind": rng.choice(["rms", "l2"]),
            "pairs": rng.choice(["half", "adjacent"]), "pos": rng.random() < 0.5}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def _normal(gen, *shape):
    return torch.randn(shape, generator=gen, device=DEV)


def _uniform(gen, lo, hi, *shape):
    return torch.rand(shape, generator=gen, device=DEV) * (hi - lo) + lo


def _ordered(x, order):
    """x [B,H,L,D] as given, or the same values held token by token ([B,L,H,D] in memory)."""
    return x if order == "head" else x.transpose(1, 2).contiguous().transpose(1, 2)


def _gates(gen, B, H, *L):
    """log decays of a head's own rate times a softplus of the step, and beta in (0, 1)."""
    tail = (1,) * len(L)
    rate = _uniform(gen, 1.0, 16.0, 1, H, *tail)
    bias = torch.log(torch.expm1(_uniform(gen, math.log(1e-3), math.log(1e-1), 1, H, *tail).exp()))
    g = -rate * torch.log1p(torch.exp(_normal(gen, B, H, *L) + bias))
    return g, torch.sigmoid(_normal(gen, B, H, *L))


def _keys(gen, dtype, *shape):
    """Unit-length rows with a common part, as learned keys have."""
    x = _normal(gen, *shape) + 0.3 * _normal(gen, *shape[:2], *(1,) * (len(shape) - 3), shape[-1])
    return (x / torch.sqrt((x * x).sum(-1, keepdim=True))).to(dtype)


def prepare(case, seed):
    c, dtype = case, DTYPE[case["type"]]
    gen = torch.Generator(device=DEV).manual_seed(seed)
    s = {"case": c}
    if c["op"] == "step":
        B, Hk, Hv, Dk, Dv = (c[n] for n in ("B", "Hk", "Hv", "Dk", "Dv"))
        s["q"], s["k"] = _keys(gen, dtype, B, Hk, Dk), _keys(gen, dtype, B, Hk, Dk)
        s["v"] = _normal(gen, B, Hv, Dv).to(dtype)
        s["g"], s["beta"] = _gates(gen, B, Hv)
        s["state"] = 0.3 * _normal(gen, B, Hv, Dk, Dv)
        s["state_out"] = torch.empty_like(s["state"])
    elif c["op"] in ("fwd", "bwd"):
        B, Hk, Hv, L, Dk, Dv = (c[n] for n in ("B", "Hk", "Hv", "L", "Dk", "Dv"))
        s["q"], s["k"] = (_ordered(_keys(gen, dtype, B, Hk, L, Dk), c["order"]) for _ in range(2))
        s["v"] = _ordered(_normal(gen, B, Hv, L, Dv).to(dtype), c["order"])
        s["g"], s["beta"] = _gates(gen, B, Hv, L)
        if c["order"] == "token":
            s["g"], s["beta"] = (x.transpose(1, 2).contiguous().transpose(1, 2) for x in (s["g"], s["beta"]))
        s["s0"] = 0.3 * _normal(gen, B, Hv, Dk, Dv) if c["s0"] else None
        if c["op"] == "bwd":
            s["do"] = _ordered(_normal(gen, B, Hv, L, Dv).to(dtype), c["order"])
            s["ds"] = 0.3 * _normal(gen, B, Hv, Dk, Dv) if c["s0"] else None
    else:
        B, Hq, Hk, L, D, R = (c[n] for n in ("B", "Hq", "Hk", "L", "D", "R"))
        qk = (_normal(gen, B, L, Hq + Hk, D) * _uniform(gen, 0.2, 3.0, B, L, 1, 1)).to(dtype)   # one projection
        s["q"], s["k"] = qk[:, :, :Hq].transpose(1, 2), qk[:, :, Hq:].transpose(1, 2)
        rms = c["kind"] == "rms"
        s["wq"], s["wk"] = (1 + 0.2 * _normal(gen, D) if rms else None for _ in range(2))
        table = 4 * L + 64
        if R:
            rates = 10000.0 ** (-torch.arange(R // 2, device=DEV, dtype=torch.float64) * 2 / R)
            angle = torch.arange(table, device=DEV, dtype=torch.float64)[:, None] * rates
            s["cos"], s["sin"] = angle.cos().float(), angle.sin().float()
        else:
            s["cos"] = s["sin"] = None
        first = torch.randint(0, 3 * L + 64, (B, 1), generator=gen, device=DEV)
        s["pos"] = (first + torch.arange(L, device=DEV)).to(torch.int32) if c["pos"] and R else None
        if c["op"] == "norm_bwd":
            s["dq"], s["dk"] = _normal(gen, B, Hq, L, D).to(dtype), _normal(gen, B, Hk, L, D).to(dtype)
    return s


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------

def run(state):
    op = state["case"]["op"]
    if own:
        return _run_own(state, op)
    if op == "step":
        return _step_plain(state)
    if op == "fwd":
        return _delta_plain(state)
    if op == "bwd":
        return _delta_bwd_plain(state)
    if op == "norm":
        return {x: _norm_plain(state, x) for x in ("q", "k")}
    return _norm_bwd_plain(state)


def _run_own(s, op):
    import structured_sparse_state_amd as pk
    c = s["case"]
    if op == "step":
        o = pk.delta_step(s["q"], s["k"], s["v"], s["g"], s["beta"], s["state"], s_out=s["state_out"])
        return {"o": o, "s": s["state_out"]}
    if op == "fwd":
        o, s_final = pk.delta_rule(s["q"], s["k"], s["v"], s["g"], s["beta"], s["s0"])
        return {"o": o, "s": s_final}
    if op == "bwd":
        got = pk.delta_rule_bwd(s["q"], s["k"], s["v"], s["g"], s["beta"], s["do"], s["s0"], s["ds"])
        return dict(zip(("dq", "dk", "dv", "dg", "dbeta", "ds0"), got))
    how = {"kind": c["kind"], "pairs": c["pairs"]}
    if op == "norm":
        q, k = pk.qk_norm_rope(s["q"], s["k"], s["wq"], s["wk"], s["cos"], s["sin"], s["pos"], **how)
        return {"q": q, "k": k}
    got = pk.qk_norm_rope_bwd(s["q"], s["k"], s["dq"], s["dk"], s["wq"], s["wk"], s["cos"], s["sin"],
                              s["pos"], **how)
    return {n: x for n, x in zip(("dq", "dk", "dwq", "dwk"), got) if x is not None}


def _step_plain(s):
    group = s["v"].shape[1] // s["q"].shape[1]
    q, k = (s[n].float().repeat_interleave(group, 1) for n in "qk")
    S = s["state"] * torch.exp(s["g"])[..., None, None]
    u = s["beta"][..., None] * (s["v"].float() - (k[..., None] * S).sum(-2))
    S = S + k[..., None] * u[..., None, :]
    o = (q[..., None] * S).sum(-2) * q.shape[-1] ** -0.5
    return {"o": o.to(s["v"].dtype), "s": S}


def _pad(x, pad):
    """x [B,H,L,...] with zero steps at the end, cut into chunks [B,H,NC,CHUNK,...]."""
    if pad:
        x = torch.cat([x, x.new_zeros(*x.shape[:2], pad, *x.shape[3:])], 2)
    return x.reshape(*x.shape[:2], -1, CHUNK, *x.shape[3:])


def _delta_parts(s):
    """What the chunks have in common in both directions: the data in chunks in
    32 bits, the decays, the products of keys and queries inside a chunk, and
    T = (I + diag(beta) N)^-1 with N[i,j] = exp(G_i - G_j) k_i . k_j, j < i."""
    group = s["v"].shape[1] // s["q"].shape[1]
    pad = -s["q"].shape[2] % CHUNK
    q, k = (_pad(s[n].float().repeat_interleave(group, 1), pad) for n in "qk")
    v, g, beta = (_pad(s[n].float(), pad) for n in ("v", "g", "beta"))
    G = torch.cumsum(g, -1)
    apart = G[..., :, None] - G[..., None, :]
    at = torch.arange(CHUNK, device=q.device)
    lower = at[:, None] >= at[None, :]
    decay = torch.where(lower, torch.exp(torch.where(lower, apart, 0.0)), 0.0)
    N = torch.where(at[:, None] > at[None, :], torch.matmul(k, k.transpose(-1, -2)) * decay, 0.0)
    P = torch.matmul(q, k.transpose(-1, -2)) * decay * q.shape[-1] ** -0.5
    A = beta[..., None] * N
    T = torch.eye(CHUNK, device=q.device).expand_as(A).contiguous()
    for i in range(1, CHUNK):   # row i of the inverse from the rows above it
        T[..., i, :i] = -torch.matmul(A[..., i, None, :i], T[..., :i, :i])[..., 0, :]
    return q, k, v, beta[..., None], G, decay, N, P, T


def _start(s):
    shape = (*s["v"].shape[:2], s["q"].shape[-1], s["v"].shape[-1])
    return s["s0"] if s["s0"] is not None else torch.zeros(shape, device=s["q"].device)


def _join(x, L):
    """Chunks [B,H,NC,CHUNK,...] as steps [B,H,L,...]."""
    return x.reshape(*x.shape[:2], -1, *x.shape[4:])[:, :, :L]


def _delta_plain(s):
    q, k, v, beta, G, decay, N, P, T = _delta_parts(s)
    rise, left, whole = torch.exp(G)[..., None], torch.exp(G[..., -1:] - G)[..., None], torch.exp(G[..., -1])
    scale, S, o = q.shape[-1] ** -0.5, _start(s), torch.empty_like(v)
    for n in range(q.shape[2]):
        u = torch.matmul(T[:, :, n], beta[:, :, n] * (v[:, :, n] - rise[:, :, n] * torch.matmul(k[:, :, n], S)))
        o[:, :, n] = scale * rise[:, :, n] * torch.matmul(q[:, :, n], S) + torch.matmul(P[:, :, n], u)
        S = whole[:, :, n, None, None] * S + torch.matmul(k[:, :, n].transpose(-1, -2), left[:, :, n] * u)
    return {"o": _join(o, s["q"].shape[2]).to(s["v"].dtype), "s": S}


def _shared(x, heads):
    """The sum over the value heads of each group."""
    return x.reshape(x.shape[0], heads, -1, *x.shape[2:]).sum(2)


def _delta_bwd_plain(s):
    q, k, v, beta, G, decay, N, P, T = _delta_parts(s)
    t = lambda x: x.transpose(-1, -2)  # noqa: E731
    dot = lambda x, y: (x * y).sum(-1)  # noqa: E731
    rise, left, whole = torch.exp(G)[..., None], torch.exp(G[..., -1:] - G)[..., None], torch.exp(G[..., -1])
    scale, S, NC = q.shape[-1] ** -0.5, _start(s), q.shape[2]
    below = torch.ones(CHUNK, CHUNK, dtype=torch.bool, device=q.device).tril(-1)
    starts, us = [], torch.empty_like(v)
    for n in range(NC):   # the states before every chunk, and u
        starts.append(S)
        us[:, :, n] = torch.matmul(T[:, :, n], beta[:, :, n] * (v[:, :, n] - rise[:, :, n] * torch.matmul(k[:, :, n], S)))
        S = whole[:, :, n, None, None] * S + torch.matmul(t(k[:, :, n]), left[:, :, n] * us[:, :, n])
    do = _pad(s["do"].float(), -s["q"].shape[2] % CHUNK)
    dS = s["ds"] if s["ds"] is not None else torch.zeros_like(S)
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    dG, dbeta = torch.empty_like(G), torch.empty_like(G)
    for n in reversed(range(NC)):
        K, Q, U, dO, S, b = k[:, :, n], q[:, :, n], us[:, :, n], do[:, :, n], starts[n], beta[:, :, n]
        r, l, w, Nn, Pn = rise[:, :, n], left[:, :, n], whole[:, :, n], N[:, :, n], P[:, :, n]
        carried = l * torch.matmul(K, dS)
        dU = torch.matmul(t(Pn), dO) + carried
        dR = torch.matmul(t(T[:, :, n]), dU)            # gradient of beta (v - e^G K S)
        KS = r * torch.matmul(K, S)
        V = v[:, :, n] - KS
        dV = b * dR
        dP = torch.matmul(dO, t(U))
        dN = -b * torch.matmul(dR, t(U))                # of N, below its diagonal
        X, Y = dP * decay[:, :, n] * scale, torch.where(below, dN * decay[:, :, n], 0.0)
        out = r * scale * torch.matmul(dO, t(S))
        dq[:, :, n] = out + torch.matmul(X, K)
        dk[:, :, n] = (torch.matmul(t(X), Q) + torch.matmul(Y + t(Y), K) + l * torch.matmul(U, t(dS))
                       - r * torch.matmul(dV, t(S)))
        dv[:, :, n] = dV
        dbeta[:, :, n] = dot(dR, V) - dot(dR, torch.matmul(Nn, U))
        pairs = dP * Pn + dN * Nn
        kept = dot(U, carried)
        dG[:, :, n] = dot(Q, out) - dot(dV, KS) + pairs.sum(-1) - pairs.sum(-2) - kept
        dG[:, :, n, -1] += kept.sum(-1) + w * (S * dS).sum((-1, -2))
        dS = w[..., None, None] * dS + torch.matmul(t(Q), scale * r * dO) - torch.matmul(t(K), r * dV)
    dg = dG.flip(-1).cumsum(-1).flip(-1)
    L, Hk, dtype = s["q"].shape[2], s["q"].shape[1], s["v"].dtype
    return {"dq": _shared(_join(dq, L), Hk).to(dtype), "dk": _shared(_join(dk, L), Hk).to(dtype),
            "dv": _join(dv, L).to(dtype), "dg": _join(dg, L), "dbeta": _join(dbeta, L), "ds0": dS}


EPS = 1e-6


def _angles(s, bits):
    """cos and sin of every token's position, [B or 1, 1, L, R/2]."""
    L = s["q"].shape[2]
    at = s["pos"].long() if s["pos"] is not None else torch.arange(L, device=s["q"].device)[None]
    return tuple(s[n][at][:, None].to(bits) for n in ("cos", "sin"))


def _rotate(y, c, pairs, cos, sin):
    """The first 2 * cos.shape[-1] dimensions of y rotated."""
    half = cos.shape[-1]
    if pairs == "half":
        a, b = y[..., :half], y[..., half:2 * half]
        turned = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
    else:
        a, b = y[..., 0:2 * half:2], y[..., 1:2 * half:2]
        turned = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    return torch.cat([turned, y[..., 2 * half:]], -1)


def _norm_plain(s, name):
    c, x, w = s["case"], s[name].float(), s["w" + name]
    ms = (x * x).mean(-1, keepdim=True) if c["kind"] == "rms" else (x * x).sum(-1, keepdim=True)
    y = x * torch.rsqrt(ms + EPS)
    if w is not None:
        y = y * w
    if c["R"]:
        y = _rotate(y, c, c["pairs"], *_angles(s, torch.float32))
    return y.to(s[name].dtype)


def _norm_bwd_plain(s):
    c, got = s["case"], {}
    for name in ("q", "k"):
        x, w, dy = s[name].float(), s["w" + name], s["d" + name].float()
        if c["R"]:
            cos, sin = _angles(s, torch.float32)
            dy = _rotate(dy, c, c["pairs"], cos, -sin)
        count = x.shape[-1] if c["kind"] == "rms" else 1
        r = torch.rsqrt((x * x).sum(-1, keepdim=True) / count + EPS)
        if w is not None:
            got["dw" + name] = (dy * x * r).sum((0, 1, 2))
            dy = dy * w
        dx = r * dy - x * r * r * r * ((dy * x).sum(-1, keepdim=True) / count)
        got["d" + name] = dx.to(s[name].dtype)
    return got


# ---------------------------------------------------------------------------
# Work and exact results
# ---------------------------------------------------------------------------

def work(case):
    c, size = case, 2 if case["type"] == "bf16" else 4
    if c["op"] == "step":
        heads, kv = c["B"] * c["Hv"], c["Dk"] * c["Dv"]
        rows = c["B"] * (2 * c["Hk"] * c["Dk"] + 2 * c["Hv"] * c["Dv"])
        return {"bytes": 8 * heads * kv + size * rows + 8 * heads, "flops": 7 * heads * kv}
    if c["op"] in ("fwd", "bwd"):
        steps, states = c["B"] * c["L"], c["B"] * c["Hv"] * c["Dk"] * c["Dv"] * 4
        keys, values = 2 * c["Hk"] * c["Dk"], 2 * c["Hv"] * c["Dv"]   # q and k; v and o, or v and do
        has = 2 if c["s0"] else 1
        kv = steps * c["Hv"] * c["Dk"] * c["Dv"]
        if c["op"] == "fwd":
            return {"bytes": steps * (size * (keys + values) + 8 * c["Hv"]) + has * states, "flops": 7 * kv}
        return {"bytes": steps * (size * (2 * keys + 1.5 * values) + 16 * c["Hv"]) + (2 * has - 1) * states,
                "flops": 17 * kv}
    count = c["B"] * c["L"] * (c["Hq"] + c["Hk"]) * c["D"]
    table = 4 * c["L"] * c["R"] * (c["B"] if c["pos"] else 1)
    if c["op"] == "norm":
        return {"bytes": 2 * size * count + table, "flops": 8 * count}
    return {"bytes": 3 * size * count + table, "flops": 16 * count}


def exact(case, seed):
    """The definitions step by step in 64 bits."""
    c, s = case, prepare(case, seed)
    if c["op"] in ("norm", "norm_bwd"):
        return _norm_exact(c, s)
    if c["op"] == "step":
        got = _recurrence(*(s[n].double()[:, :, None] for n in ("q", "k", "v", "g", "beta")), s["state"].double())
        return {"o": got["o"][:, :, 0], "s": got["s"]}
    S = _start(s).double()
    ins = [s[n].double() for n in ("q", "k", "v", "g", "beta")]
    if c["op"] == "fwd":
        return _recurrence(*ins, S)
    return _recurrence_bwd(*ins, S, s["do"].double(), None if s["ds"] is None else s["ds"].double())


def _advance(S, k, v, g, beta):
    """The state after one step, and the step's u."""
    S = S * g.exp()[..., None, None]
    u = (v - (k.unsqueeze(-2) @ S).squeeze(-2)) * beta[..., None]
    return torch.addcmul(S, k[..., None], u[..., None, :]), u


def _recurrence(q, k, v, g, beta, S):
    group = v.shape[1] // q.shape[1]
    q, k = q.repeat_interleave(group, 1), k.repeat_interleave(group, 1)
    o = torch.empty_like(v)
    for t in range(q.shape[2]):
        S, _ = _advance(S, k[:, :, t], v[:, :, t], g[:, :, t], beta[:, :, t])
        o[:, :, t] = (q[:, :, t].unsqueeze(-2) @ S).squeeze(-2) / math.sqrt(q.shape[-1])
    return {"o": o, "s": S}


def _recurrence_bwd(q, k, v, g, beta, S, do, dS):
    """Reverse mode of the recurrence, step by step; states are kept for every
    64th step and made again from there."""
    Hk, group, L, every = q.shape[1], v.shape[1] // q.shape[1], q.shape[2], 64
    q, k = q.repeat_interleave(group, 1), k.repeat_interleave(group, 1)
    kept = []
    for t in range(L):
        if t % every == 0:
            kept.append(S)
        S, _ = _advance(S, k[:, :, t], v[:, :, t], g[:, :, t], beta[:, :, t])
    dS = torch.zeros_like(S) if dS is None else dS
    do = do / math.sqrt(q.shape[-1])
    d = {n: torch.empty_like(x) for n, x in (("dq", q), ("dk", k), ("dv", v), ("dg", g), ("dbeta", beta))}
    for first in reversed(range(0, L, every)):
        S, states, us = kept[first // every], [], []
        for t in range(first, min(L, first + every)):
            states.append(S)
            S, u = _advance(S, k[:, :, t], v[:, :, t], g[:, :, t], beta[:, :, t])
            us.append(u)
        states.append(S)
        for t in reversed(range(first, min(L, first + every))):
            K, a, b, u = k[:, :, t], g[:, :, t].exp(), beta[:, :, t, None], us[t - first]
            old, new = states[t - first] * a[..., None, None], states[t - first + 1]
            d["dq"][:, :, t] = (new @ do[:, :, t, :, None])[..., 0]
            dS = dS + q[:, :, t, :, None] * do[:, :, t, None, :]
            du = (K.unsqueeze(-2) @ dS).squeeze(-2)
            d["dv"][:, :, t] = b * du
            d["dbeta"][:, :, t] = (du * (v[:, :, t] - (K.unsqueeze(-2) @ old).squeeze(-2))).sum(-1)
            d["dk"][:, :, t] = (dS @ u[..., None] - old @ (b * du)[..., None])[..., 0]
            dS = dS - K[..., None] * (b * du)[..., None, :]
            d["dg"][:, :, t] = (dS * old).sum((-1, -2))
            dS = dS * a[..., None, None]
    for n in ("dq", "dk"):
        d[n] = d[n].unflatten(1, (Hk, group)).sum(2)
    return {**d, "ds0": dS}


def _norm_exact(c, s):
    got, R = {}, c["R"]
    for name in ("q", "k"):
        x = s[name].double()
        n = torch.linalg.vector_norm(x, dim=-1, keepdim=True) ** 2
        r = (n / (c["D"] if c["kind"] == "rms" else 1) + EPS) ** -0.5
        w = s["w" + name].double() if s["w" + name] is not None else torch.ones(c["D"], device=DEV, dtype=torch.float64)
        # the rotation as one complex factor for each pair
        first = torch.arange(R // 2, device=DEV) * (1 if c["pairs"] == "half" else 2)
        second = first + (R // 2 if c["pairs"] == "half" else 1)
        if R:
            cos, sin = _angles(s, torch.float64)
            turn = torch.complex(cos, sin)
        if c["op"] == "norm":
            y = x * r * w
            if R:
                z = torch.complex(y[..., first], y[..., second]) * turn
                y[..., first], y[..., second] = z.real, z.imag
            got[name] = y
            continue
        dy = s["d" + name].double().clone()
        if R:
            z = torch.complex(dy[..., first], dy[..., second]) * turn.conj()
            dy[..., first], dy[..., second] = z.real, z.imag
        unit = x * r
        if s["w" + name] is not None:
            got["dw" + name] = (dy * unit).sum((0, 1, 2))
        dy = dy * w
        share = (dy * unit).sum(-1, keepdim=True) / (c["D"] if c["kind"] == "rms" else 1)
        got["d" + name] = r * (dy - unit * share)
    return got


if __name__ == "__main__":
    for case in listed() + [draw(random.Random(n)) for n in range(6)]:
        print(case, work(case))

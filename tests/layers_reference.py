"""The gated delta rule and the query/key norm with rotation in 64 bits,
literally from their definitions (include/pdssm_layers.h): step by step, on
the CPU, with no chunks.  Gradients by reverse mode of the same steps."""
from __future__ import annotations

import torch

F64 = torch.float64


def _heads(x, group):
    return x.to("cpu", F64).repeat_interleave(group, 1)


def delta(q, k, v, g, beta, s0=None, scale=None):
    """(o [B,Hv,L,Dv], s_final, the states after every step) in fp64."""
    group = v.shape[1] // q.shape[1]
    scale = q.shape[-1] ** -0.5 if scale is None else scale
    q, k, v, g, beta = _heads(q, group), _heads(k, group), v.to("cpu", F64), g.to("cpu", F64), beta.to("cpu", F64)
    B, H, L, Dk = q.shape
    S = torch.zeros(B, H, Dk, v.shape[-1], dtype=F64) if s0 is None else s0.to("cpu", F64)
    o, states = torch.zeros_like(v), [S]
    for t in range(L):
        S = S * g[:, :, t].exp()[..., None, None]
        u = beta[:, :, t, None] * (v[:, :, t] - torch.einsum("bhk,bhkv->bhv", k[:, :, t], S))
        S = S + k[:, :, t, :, None] * u[:, :, None, :]
        o[:, :, t] = scale * torch.einsum("bhk,bhkv->bhv", q[:, :, t], S)
        states.append(S)
    return o, S, states


def delta_bwd(q, k, v, g, beta, do, s0=None, ds_final=None, scale=None):
    """(dq, dk, dv, dg, dbeta, ds0) in fp64, and the size of the terms whose
    sum dg is, |q . dq| + |v . dv| of every step."""
    Hk = q.shape[1]
    group = v.shape[1] // Hk
    scale = q.shape[-1] ** -0.5 if scale is None else scale
    _, _, states = delta(q, k, v, g, beta, s0, scale)
    q, k, v, g, beta = _heads(q, group), _heads(k, group), v.to("cpu", F64), g.to("cpu", F64), beta.to("cpu", F64)
    do = do.to("cpu", F64)
    dS = torch.zeros_like(states[0]) if ds_final is None else ds_final.to("cpu", F64)
    dq, dk, dv, dg, db = (torch.zeros_like(x) for x in (q, k, v, g, beta))
    for t in reversed(range(q.shape[2])):
        a, kt, bt, new = g[:, :, t].exp(), k[:, :, t], beta[:, :, t, None], states[t + 1]
        old = states[t] * a[..., None, None]        # the state the step reads
        r = v[:, :, t] - torch.einsum("bhk,bhkv->bhv", kt, old)
        dq[:, :, t] = scale * torch.einsum("bhkv,bhv->bhk", new, do[:, :, t])
        dS = dS + scale * q[:, :, t, :, None] * do[:, :, t, None, :]
        du = torch.einsum("bhk,bhkv->bhv", kt, dS)
        dv[:, :, t] = bt * du
        db[:, :, t] = (du * r).sum(-1)
        dk[:, :, t] = torch.einsum("bhkv,bhv->bhk", dS, bt * r) - torch.einsum("bhkv,bhv->bhk", old, bt * du)
        dS = dS - kt[..., None] * (bt * du)[..., None, :]
        dg[:, :, t] = (dS * old).sum((-1, -2))
        dS = dS * a[..., None, None]
    terms = (q * dq).sum(-1).abs() + (v * dv).sum(-1).abs()
    sums = lambda x: x.unflatten(1, (Hk, group)).sum(2)  # noqa: E731
    return (sums(dq), sums(dk), dv, dg, db, dS), terms


def rotate(y, cos, sin, pos, pairs, back=False):
    """The first 2 * cos.shape[1] dimensions of y [B,H,L,D] turned."""
    if cos is None or cos.shape[1] == 0:
        return y
    B, _, L, _ = y.shape
    half = cos.shape[1]
    at = (torch.arange(L)[None].expand(B, L) if pos is None else pos.cpu().long()).clamp(0, cos.shape[0] - 1)
    c, s = cos.to("cpu", F64)[at][:, None], sin.to("cpu", F64)[at][:, None]
    if back:
        s = -s
    i = torch.arange(half)
    a, b = (i, i + half) if pairs == "half" else (2 * i, 2 * i + 1)
    out = y.clone()
    out[..., a] = c * y[..., a] - s * y[..., b]
    out[..., b] = s * y[..., a] + c * y[..., b]
    return out


def norm(x, w, cos, sin, pos, kind, pairs, eps):
    x = x.to("cpu", F64)
    n = x.shape[-1] if kind == "rms" else 1
    y = x / torch.sqrt((x * x).sum(-1, keepdim=True) / n + eps)
    if w is not None:
        y = y * w.to("cpu", F64)
    return rotate(y, cos, sin, pos, pairs)


def norm_bwd(x, dy, w, cos, sin, pos, kind, pairs, eps):
    """(dx, dw) in fp64 (dw whether or not there is a weight)."""
    x, dy = x.to("cpu", F64), dy.to("cpu", F64)
    n = x.shape[-1] if kind == "rms" else 1
    r = 1 / torch.sqrt((x * x).sum(-1, keepdim=True) / n + eps)
    e = rotate(dy, cos, sin, pos, pairs, back=True)
    dw = (e * x * r).sum((0, 1, 2))
    if w is not None:
        e = e * w.to("cpu", F64)
    return r * (e - x * r * (e * x * r).sum(-1, keepdim=True) / n), dw

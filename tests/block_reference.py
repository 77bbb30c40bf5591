"""Linear attention with decays in 64 bits, literally from its definition
(include/pdssm_block.h): step by step, on the CPU, with no chunks.  Gradients
by reverse mode of the same steps."""
from __future__ import annotations

import torch

F64 = torch.float64


def _heads(x, group):
    return x.to("cpu", F64).repeat_interleave(group, 1)


def gates(g, B, Hv, L):
    """The log decays of every sequence, head and step."""
    if g is None:
        return torch.zeros(B, Hv, L, dtype=F64)
    g = g.to("cpu", F64)
    return g[None, :, None].expand(B, Hv, L) if g.dim() == 1 else g


def linear(q, k, v, g, s0=None, scale=None):
    """(o [B,Hv,L,Dv], s_final, the states after every step) in fp64."""
    group = v.shape[1] // q.shape[1]
    scale = q.shape[-1] ** -0.5 if scale is None else scale
    q, k, v = _heads(q, group), _heads(k, group), v.to("cpu", F64)
    B, H, L, Dk = q.shape
    g = gates(g, B, H, L)
    S = torch.zeros(B, H, Dk, v.shape[-1], dtype=F64) if s0 is None else s0.to("cpu", F64)
    o, states = torch.zeros_like(v), [S]
    for t in range(L):
        S = S * g[:, :, t].exp()[..., None, None] + k[:, :, t, :, None] * v[:, :, t, None, :]
        o[:, :, t] = scale * (q[:, :, t, None, :] @ S)[..., 0, :]
        states.append(S)
    return o, S, states


def linear_bwd(q, k, v, g, do, s0=None, ds_final=None, scale=None):
    """(dq, dk, dv, dg [B,Hv,L], ds0) in fp64, and |S| |dS| around every step's
    decay, whose product dg is."""
    Hk = q.shape[1]
    group = v.shape[1] // Hk
    scale = q.shape[-1] ** -0.5 if scale is None else scale
    _, _, states = linear(q, k, v, g, s0, scale)
    q, k, v, do = _heads(q, group), _heads(k, group), v.to("cpu", F64), do.to("cpu", F64)
    g = gates(g, *v.shape[:3])
    dS = torch.zeros_like(states[0]) if ds_final is None else ds_final.to("cpu", F64)
    dq, dk, dv, dg, size = torch.zeros_like(q), torch.zeros_like(q), torch.zeros_like(v), *(torch.zeros(v.shape[:3], dtype=F64) for _ in range(2))
    for t in reversed(range(q.shape[2])):
        a = g[:, :, t].exp()[..., None, None]
        dq[:, :, t] = scale * (states[t + 1] @ do[:, :, t, :, None])[..., 0]
        dS = dS + scale * q[:, :, t, :, None] * do[:, :, t, None, :]
        dk[:, :, t] = (dS @ v[:, :, t, :, None])[..., 0]
        dv[:, :, t] = (k[:, :, t, None, :] @ dS)[..., 0, :]
        old = states[t] * a
        dg[:, :, t] = (dS * old).sum((-1, -2))
        size[:, :, t] = old.norm(dim=(-2, -1)) * dS.norm(dim=(-2, -1))
        dS = dS * a
    sums = lambda x: x.unflatten(1, (Hk, group)).sum(2)  # noqa: E731
    return (sums(dq), sums(dk), dv, dg, dS), size

"""Linear attention with decays, dropout and the layer norm in 64 bits,
literally from their definitions (include/pdssm_block.h), on the CPU: the
recurrence step by step, with no chunks; gradients by reverse mode of the same
steps; random bits from the generator in unsigned arithmetic."""
from __future__ import annotations

import numpy as np
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


def philox(counter, key):
    """Philox 4x32 with ten rounds: counter [4, ...] and key (2 numbers) of 32
    bits to [4, ...] uint32."""
    c = [np.asarray(x, np.uint64) for x in counter]
    k, low = [int(x) for x in key], np.uint64(0xFFFFFFFF)
    for _ in range(10):
        a, b = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(b >> np.uint64(32)) ^ c[1] ^ np.uint64(k[0]), b & low, (a >> np.uint64(32)) ^ c[3] ^ np.uint64(k[1]), a & low]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return np.stack([x.astype(np.uint32) for x in c])


def bits(rows, D, seed, offset):
    """The 16 random bits of every value of [rows, D]."""
    units = (D + 7) // 8
    unit, row = np.meshgrid(np.arange(units), np.arange(rows))
    off = [np.full_like(unit, offset >> s & 0xFFFFFFFF) for s in (0, 32)]
    words = philox([unit, row, *off], [seed & 0xFFFFFFFF, seed >> 32 & 0xFFFFFFFF])
    halves = np.stack([words & np.uint32(0xFFFF), words >> np.uint32(16)], 1)       # [word, half, row, unit]
    return torch.from_numpy(halves.transpose(2, 3, 0, 1).reshape(rows, 8 * units)[:, :D].astype(np.int64))


def threshold(p):
    return min(65535, int(p * 65536 + 0.5))


def dropped(x, p, seed, offset):
    """dropout(x) in fp64."""
    x, T = x.to("cpu", F64), threshold(p)
    keep = bits(x[..., 0].numel(), x.shape[-1], seed, offset).view(x.shape) >= T
    return torch.where(keep, x * (65536 / (65536 - T)), 0.0)


def layer_norm(x, w=None, b=None, residual=None, eps=1e-5, p=0.0, seed=0, offset=0):
    """(y, h) in fp64."""
    h = dropped(x, p, seed, offset)
    if residual is not None:
        h = h + residual.to("cpu", F64)
    c = h - h.mean(-1, keepdim=True)
    y = c / torch.sqrt((c * c).mean(-1, keepdim=True) + eps)
    if w is not None:
        y = y * w.to("cpu", F64)
    if b is not None:
        y = y + b.to("cpu", F64)
    return y, h


def layer_norm_bwd(h, dy, w=None, dh=None, eps=1e-5, p=0.0, seed=0, offset=0):
    """(dr, dx, dw, db) in fp64, from h as stored."""
    h, dy = h.to("cpu", F64), dy.to("cpu", F64)
    c = h - h.mean(-1, keepdim=True)
    r = 1 / torch.sqrt((c * c).mean(-1, keepdim=True) + eps)
    unit, e = c * r, dy if w is None else dy * w.to("cpu", F64)
    dr = r * (e - e.mean(-1, keepdim=True) - unit * (e * unit).mean(-1, keepdim=True))
    if dh is not None:
        dr = dr + dh.to("cpu", F64)
    flat = lambda t: t.reshape(-1, t.shape[-1]).sum(0)  # noqa: E731
    return dr, dropped(dr, p, seed, offset), flat(dy * unit), flat(dy)

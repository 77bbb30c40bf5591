"""A sequence layer of the gated delta rule, trained and then served.

The layer takes queries, keys and values from one projection, normalises every
query and key head and rotates part of it by position (``qk_norm_rope``), runs
the gated delta rule (``delta_rule``) and projects back.  Training uses the
gradients ``delta_rule_bwd`` and ``qk_norm_rope_bwd`` through two
autograd functions; serving runs a prompt through the same forward and then
single tokens with ``delta_step``, the state carried between them.

    python examples/delta_layer.py            # needs an MI355X
"""
from __future__ import annotations

import os
import sys

import torch
import torch.nn.functional as F
from torch.autograd.function import once_differentiable

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import structured_sparse_state_amd as pk  # noqa: E402


def rows(grad):
    """A gradient whose rows lie whole in memory (that of a sum does not)."""
    return grad if grad.stride(-1) == 1 else grad.contiguous()


class QkNormRope(torch.autograd.Function):
    """Unit-length queries and keys, rotated by position."""

    @staticmethod
    def forward(ctx, q, k, wq, wk, cos, sin):
        ctx.save_for_backward(q, k, wq, wk, cos, sin)
        return pk.qk_norm_rope(q, k, wq, wk, cos, sin, kind="l2")

    @staticmethod
    @once_differentiable
    def backward(ctx, dq_out, dk_out):
        q, k, wq, wk, cos, sin = ctx.saved_tensors
        return *pk.qk_norm_rope_bwd(q, k, rows(dq_out), rows(dk_out), wq, wk, cos, sin, kind="l2"), None, None


class DeltaRule(torch.autograd.Function):
    """The gated delta rule over whole sequences from an empty state."""

    @staticmethod
    def forward(ctx, q, k, v, g, beta):
        ctx.save_for_backward(q, k, v, g, beta)
        return pk.delta_rule(q, k, v, g, beta, want_state=False)[0]

    @staticmethod
    @once_differentiable
    def backward(ctx, do):
        return pk.delta_rule_bwd(*ctx.saved_tensors, rows(do), want_ds0=False)[:5]


class DeltaLayer(torch.nn.Module):
    def __init__(self, width: int, key_heads: int, value_heads: int, head: int, positions: int, rotated: int):
        super().__init__()
        self.Hk, self.Hv, self.D = key_heads, value_heads, head
        rows = (2 * key_heads + value_heads) * head + 2 * value_heads
        self.project = torch.nn.Linear(width, rows, bias=False)
        self.out = torch.nn.Linear(value_heads * head, width, bias=False)
        self.wq, self.wk = (torch.nn.Parameter(torch.ones(head)) for _ in range(2))
        self.rate = torch.nn.Parameter(torch.zeros(value_heads))
        angle = torch.arange(positions)[:, None] * 10000.0 ** (-torch.arange(rotated // 2) * 2 / rotated)
        self.register_buffer("cos", angle.cos())
        self.register_buffer("sin", angle.sin())

    def parts(self, x):
        """q, k, v [B,H,L,D] as views of one projection, g and beta [B,Hv,L]."""
        Hk, Hv, D = self.Hk, self.Hv, self.D
        y = self.project(x).to(torch.bfloat16)
        B, L, _ = y.shape
        heads = y[..., :(2 * Hk + Hv) * D].unflatten(2, (2 * Hk + Hv, D)).transpose(1, 2)
        gates = y[..., (2 * Hk + Hv) * D:].float().transpose(1, 2)
        g = -F.softplus(gates[:, :Hv] + self.rate[:, None] - 2.0)
        return heads[:, :Hk], heads[:, Hk:2 * Hk], heads[:, 2 * Hk:], g, torch.sigmoid(gates[:, Hv:])

    def forward(self, x):
        q, k, v, g, beta = self.parts(x)
        q, k = QkNormRope.apply(q, k, self.wq, self.wk, self.cos, self.sin)
        o = DeltaRule.apply(q, k, v, g, beta)
        return self.out(o.transpose(1, 2).flatten(2).to(x.dtype))

    @torch.no_grad()
    def prefill(self, x):
        """The prompt's outputs and the state after it."""
        q, k, v, g, beta = self.parts(x)
        q, k = pk.qk_norm_rope(q, k, self.wq, self.wk, self.cos, self.sin, kind="l2")
        o, state = pk.delta_rule(q, k, v, g, beta)
        return self.out(o.transpose(1, 2).flatten(2).to(x.dtype)), state

    @torch.no_grad()
    def step(self, x, position, state):
        """One token's outputs; the state is updated in place."""
        q, k, v, g, beta = self.parts(x[:, None])
        pos = torch.full((x.shape[0], 1), position, dtype=torch.int32, device=x.device)
        q, k = pk.qk_norm_rope(q, k, self.wq, self.wk, self.cos, self.sin, pos, kind="l2")
        o = pk.delta_step(q[:, :, 0], k[:, :, 0], v[:, :, 0], g[:, :, 0], beta[:, :, 0], state)
        return self.out(o.flatten(1).to(x.dtype))


def main(B: int = 4, L: int = 192, width: int = 128, steps: int = 60, device: str = "cuda:0"):
    """Trains the layer to repeat each token's pair from earlier in the sequence;
    returns the losses and how far decoding is from the full forward."""
    torch.manual_seed(0)
    layer = DeltaLayer(width, key_heads=2, value_heads=4, head=64, positions=L, rotated=16).to(device)
    table = torch.randn(32, width, device=device)
    answers = torch.randn(32, width, device=device)
    optim = torch.optim.AdamW(layer.parameters(), lr=3e-3)
    losses = []
    for _ in range(steps):
        ids = torch.randint(0, 32, (B, L), device=device)
        loss = F.mse_loss(layer(table[ids]), answers[ids])
        optim.zero_grad()
        loss.backward()
        optim.step()
        losses.append(loss.detach())
    losses = torch.stack(losses).tolist()

    x = table[torch.randint(0, 32, (B, L), device=device)]
    with torch.no_grad():
        whole = layer(x)
    cut = L - 16
    first, state = layer.prefill(x[:, :cut])
    rest = [layer.step(x[:, t], t, state) for t in range(cut, L)]
    served = torch.cat([first, torch.stack(rest, 1)], 1)
    apart = float((served - whole).norm() / whole.norm())
    return losses, apart


if __name__ == "__main__":
    losses, apart = main()
    print(f"loss {losses[0]:.4f} -> {losses[-1]:.4f} over {len(losses)} steps; "
          f"prompt and single tokens against one forward: {apart:.1e} of its norm")

"""A residual block of linear attention with decays, trained and then served.

The block normalises the residual stream (``layer_norm``), takes queries, keys,
values and the log decay of every head and step from one projection, runs
``linear_attention``, projects back, and adds the result, with dropout, to the
stream under the next norm (``layer_norm`` with residual and dropout).  Training
uses the library's gradients through two autograd functions; serving runs a
prompt through the same forward and then single tokens with
``linear_attention_step``, the state carried between them.

    python examples/linear_layer.py            # needs an MI355X
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
    return grad if grad is None or grad.stride(-1) == 1 else grad.contiguous()


class AddNorm(torch.autograd.Function):
    """(norm(h), h) of h = residual + dropout(x)."""

    @staticmethod
    def forward(ctx, x, residual, w, b, p, seed):
        y, h = pk.layer_norm(x, w, b, residual=residual, p=p, seed=seed)
        ctx.save_for_backward(h, w)
        ctx.dropout = {"p": p, "seed": seed}
        ctx.set_materialize_grads(False)
        return y, h

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, dh):
        h, w = ctx.saved_tensors
        dy = torch.zeros_like(h) if dy is None else rows(dy)
        dr, dx, dw, db = pk.layer_norm_bwd(h, dy, w, dh=rows(dh), want_db=True, **ctx.dropout)
        return dx, dr, dw, db, None, None


class LinearAttention(torch.autograd.Function):
    """Linear attention over whole sequences from an empty state; g [B,H,L] or [H]."""

    @staticmethod
    def forward(ctx, q, k, v, g):
        ctx.save_for_backward(q, k, v, g)
        return pk.linear_attention(q, k, v, g, want_state=False)[0]

    @staticmethod
    @once_differentiable
    def backward(ctx, do):
        q, k, v, g = ctx.saved_tensors
        return pk.linear_attention_bwd(q, k, v, g, rows(do), want_ds0=False)[:4]


class LinearBlock(torch.nn.Module):
    def __init__(self, width: int, key_heads: int, value_heads: int, head: int, p: float):
        super().__init__()
        self.Hk, self.Hv, self.D, self.p = key_heads, value_heads, head, p
        self.project = torch.nn.Linear(width, (2 * key_heads + value_heads) * head + value_heads, bias=False)
        self.out = torch.nn.Linear(value_heads * head, width, bias=False)
        self.w1, self.w2 = (torch.nn.Parameter(torch.ones(width)) for _ in range(2))
        self.b1, self.b2 = (torch.nn.Parameter(torch.zeros(width)) for _ in range(2))
        self.rate = torch.nn.Parameter(torch.linspace(-4.0, 0.0, value_heads))

    def parts(self, y):
        """q, k, v [B,H,L,D] as views of one projection, g [B,Hv,L]."""
        Hk, Hv, D = self.Hk, self.Hv, self.D
        z = self.project(y).to(torch.bfloat16)
        heads = z[..., :(2 * Hk + Hv) * D].unflatten(2, (2 * Hk + Hv, D)).transpose(1, 2)
        g = -F.softplus(z[..., (2 * Hk + Hv) * D:].float().transpose(1, 2) + self.rate[:, None])
        return heads[:, :Hk], heads[:, Hk:2 * Hk], heads[:, 2 * Hk:], g

    def forward(self, x, seed: int = 0):
        """The normalised stream after the block, and the stream."""
        y, x = AddNorm.apply(x, torch.zeros_like(x), self.w1, self.b1, 0.0, 0)
        o = LinearAttention.apply(*self.parts(y))
        branch = self.out(o.transpose(1, 2).flatten(2).to(x.dtype))
        return AddNorm.apply(branch, x, self.w2, self.b2, self.p if self.training else 0.0, seed)

    @torch.no_grad()
    def prefill(self, x):
        """The prompt's outputs and the state after it."""
        y, _ = pk.layer_norm(x, self.w1, self.b1)
        o, state = pk.linear_attention(*self.parts(y))
        branch = self.out(o.transpose(1, 2).flatten(2).to(x.dtype))
        return pk.layer_norm(branch, self.w2, self.b2, residual=x)[0], state

    @torch.no_grad()
    def step(self, x, state):
        """One token's outputs; the state is updated in place."""
        y, _ = pk.layer_norm(x, self.w1, self.b1)
        q, k, v, g = (t[:, :, 0] for t in self.parts(y[:, None]))
        branch = self.out(pk.linear_attention_step(q, k, v, g, state).flatten(1).to(x.dtype))
        return pk.layer_norm(branch, self.w2, self.b2, residual=x)[0]


def main(B: int = 4, L: int = 192, width: int = 128, steps: int = 40, device: str = "cuda:0"):
    """Trains the block to name the token before; returns the losses and how far
    decoding is from the full forward."""
    torch.manual_seed(0)
    block = LinearBlock(width, key_heads=2, value_heads=4, head=64, p=0.1).to(device)
    table = torch.randn(32, width, device=device)
    answers = torch.randn(32, width, device=device)
    optim = torch.optim.AdamW(block.parameters(), lr=3e-3)
    losses = []
    for n in range(steps):
        ids = torch.randint(0, 32, (B, L), device=device)
        loss = F.mse_loss(block(table[ids], seed=n)[0], answers[ids.roll(1, 1)])
        optim.zero_grad()
        loss.backward()
        optim.step()
        losses.append(loss.detach())
    losses = torch.stack(losses).tolist()

    block.eval()
    x = table[torch.randint(0, 32, (B, L), device=device)]
    with torch.no_grad():
        whole, _ = block(x)
    cut = L - 16
    first, state = block.prefill(x[:, :cut])
    rest = [block.step(x[:, t], state) for t in range(cut, L)]
    served = torch.cat([first, torch.stack(rest, 1)], 1)
    apart = float((served - whole).norm() / whole.norm())
    return losses, apart


if __name__ == "__main__":
    losses, apart = main()
    print(f"loss {losses[0]:.4f} -> {losses[-1]:.4f} over {len(losses)} steps; "
          f"prompt and single tokens against one forward: {apart:.1e} of its norm")

"""A block with decayed linear attention, trained on a sequence and served token by token.

    h = residual + scale * x                      residual_norm: the norm before the block
    q, k, v, z, a = projections of norm(h)        (library products)
    o = decay attention of q, k, v                one decay per head and token, from a
    x = projection of norm(o) * silu(z)           gated_norm, one group per head

``python examples/decay_attention_block.py`` checks on the GPU that a prompt
taken at once, and the same prompt in one piece followed by single tokens, give
the same outputs, and takes a few gradient steps.
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import selective_state_space_10_amd as ssm  # noqa: E402


class Block(torch.nn.Module):
    def __init__(self, width, heads, key_heads, dk, dv, dtype=torch.bfloat16, device="cuda"):
        super().__init__()
        self.sizes = (heads, key_heads, dk, dv)
        self.parts = [key_heads * dk, key_heads * dk, heads * dv, heads * dv, heads]
        self.pad = -sum(self.parts) % 8  # rows of the projection stay 16-byte aligned
        f32 = dict(dtype=torch.float32, device=device)
        self.project = torch.nn.Linear(width, sum(self.parts) + self.pad, bias=False, dtype=dtype, device=device)
        self.out = torch.nn.Linear(heads * dv, width, bias=False, dtype=dtype, device=device)
        self.norm = torch.nn.Parameter(torch.ones(width, **f32))
        self.scale = torch.nn.Parameter(torch.full((width,), 0.5, **f32))
        self.gate_norm = torch.nn.Parameter(torch.ones(heads * dv, **f32))
        self.decay_bias = torch.nn.Parameter(torch.linspace(-6.0, -1.0, heads, **f32))

    def _inputs(self, y):
        H, G, dk, dv = self.sizes
        q, k, v, z, a = self.project(y).split([*self.parts[:4], self.parts[4] + self.pad], -1)
        g = -torch.nn.functional.softplus(a[..., :H].float() + self.decay_bias)
        return q.unflatten(-1, (G, dk)), k.unflatten(-1, (G, dk)), v.unflatten(-1, (H, dv)), z, g

    def forward(self, x, residual, state=None):
        """x, residual (batch, length, width); returns x, the residual stream and the last state."""
        y, h = ssm.residual_norm(x, residual, self.norm, self.scale)
        q, k, v, z, g = self._inputs(y)
        o, state = ssm.decay_attention(q, k, v, g, None, state)
        return self.out(ssm.gated_norm(o.flatten(2), z, self.gate_norm, self.sizes[3])), h, state

    @torch.no_grad()
    def step(self, x, residual, state):
        """One token: x, residual (batch, width); the state is updated in place."""
        y, h, _ = ssm.residual_norm_fwd(x, residual, self.norm, self.scale)
        q, k, v, z, g = self._inputs(y)
        o = ssm.decay_attn_update(state, q, k, v, g.contiguous())
        u, _ = ssm.gated_norm_fwd(o.flatten(1), z, self.gate_norm, self.sizes[3])
        return self.out(u), h


def run(batch=2, length=150, width=256, heads=8, key_heads=4, dk=32, dv=64, dtype=torch.bfloat16, steps=3, seed=0):
    """Returns the largest difference between both ways of serving a prompt, relative to the
    outputs' largest value, and the losses of a few gradient steps."""
    torch.manual_seed(seed)
    block = Block(width, heads, key_heads, dk, dv, dtype)
    x = torch.randn(batch, length, width, device="cuda").to(dtype)
    residual = torch.randn(batch, length, width, device="cuda")
    with torch.no_grad():
        whole, _, last = block(x, residual)
        cut = length - 5
        head, _, state = block(x[:, :cut].contiguous(), residual[:, :cut].contiguous())
        tail = [block.step(x[:, t].contiguous(), residual[:, t].contiguous(), state)[0] for t in range(cut, length)]
    served = torch.cat([head, torch.stack(tail, 1)], 1)
    diff = float((served.float() - whole.float()).abs().max() / whole.float().abs().max())
    diff = max(diff, float((state - last).abs().max() / last.abs().max()))

    target = torch.randn(batch, length, width, device="cuda")
    opt = torch.optim.SGD(block.parameters(), lr=0.05)
    losses = []
    for _ in range(steps):
        opt.zero_grad()
        y, h, _ = block(x, residual)
        loss = ((y.float() + h - target) ** 2).mean()
        loss.backward()
        opt.step()
        losses.append(float(loss.detach()))
    return diff, losses


if __name__ == "__main__":
    diff, losses = run()
    print(f"prompt at once against prompt and single tokens: {diff:.2e} of the largest value")
    print("losses:", ", ".join(f"{v:.4f}" for v in losses))

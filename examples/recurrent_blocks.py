"""Two blocks of a recurrent language model, trained on packed and padded sequences and
served token by token.

    RecurrentBlock                                   LinearAttentionBlock
    y, h = residual_norm(x, residual)                y, h = residual_norm(x, residual)
    u, z, g, i = projections of y                    q, k, v, z, a = projections of y
    u = causal_conv(u)                               q, k, v = causal_conv of q, k and v together
    o = gated_recurrence(u, g, i, decay, z)          q, k = head_norm_rotary(q, k)
    x = projection of o                              x = projection of gated_norm(decay_attention(q, k, v), z)

A document starts where ``starts`` says so: convolution, recurrence and decay attention
carry nothing over it, the recurrence takes its first input in full, and positions begin
anew.  A prompt's first token is marked too, so that serving computes what was trained.

``python examples/recurrent_blocks.py`` checks on the GPU that a prompt taken at once, and
the same prompt in one piece followed by single tokens, give the same outputs.
"""
from __future__ import annotations

import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import selective_state_space_10_amd as ssm  # noqa: E402


def _linear(n, m, dtype, device):
    return torch.nn.Linear(n, m, bias=False, dtype=dtype, device=device)


class RecurrentBlock(torch.nn.Module):
    def __init__(self, width, inner, taps=4, dtype=torch.bfloat16, device="cuda"):
        super().__init__()
        f32 = dict(dtype=torch.float32, device=device)
        self.inner, self.taps = inner, taps
        self.project, self.out = _linear(width, 4 * inner, dtype, device), _linear(inner, width, dtype, device)
        self.norm = torch.nn.Parameter(torch.ones(width, **f32))
        self.conv = torch.nn.Parameter(torch.randn(inner, taps, **f32) * taps ** -0.5)
        self.conv_bias = torch.nn.Parameter(torch.zeros(inner, **f32))
        # a = 0.9 ... 0.999 where the gate is open
        self.decay = torch.nn.Parameter(torch.log(torch.expm1(-torch.log(torch.linspace(0.9, 0.999, inner, **f32)) / 8.0)))

    def forward(self, x, residual, state=None, starts=None, lengths=None):
        """x, residual (batch, length, width); state: of the convolution and of the recurrence.
        Returns x, the residual stream and the last state."""
        conv0, h0 = (None, None) if state is None else state
        y, h = ssm.residual_norm(x, residual, self.norm)
        u, z, g, i = self.project(y).split(self.inner, -1)
        u, conv1 = ssm.causal_conv(u, self.conv, self.conv_bias, conv0, starts, lengths)
        o, h1 = ssm.gated_recurrence(u, g, i, self.decay, z, h0, starts, lengths)
        return self.out(o), h, (conv1, h1)

    def prompt(self, x, residual, lengths=None):
        """The beginnings of documents, which forward or step go on from: the first tokens are
        marked, as packed documents' are in training."""
        starts = torch.zeros(x.shape[:2], dtype=torch.bool, device=x.device)
        starts[:, 0] = True
        return self(x, residual, None, starts, lengths)

    @torch.no_grad()
    def step(self, x, residual, state):
        """One token: x, residual (batch, width); the state is updated in place."""
        y, h, _ = ssm.residual_norm_fwd(x, residual, self.norm)
        u, z, g, i = self.project(y).split(self.inner, -1)
        u = ssm.causal_conv_update(state[0], u, self.conv, self.conv_bias)
        return self.out(ssm.gated_recurrence_update(state[1], u, g, i, self.decay, z)), h


class LinearAttentionBlock(torch.nn.Module):
    def __init__(self, width, heads, key_heads, dk, dv, taps=4, dtype=torch.bfloat16, device="cuda"):
        super().__init__()
        f32 = dict(dtype=torch.float32, device=device)
        self.sizes = heads, key_heads, dk, dv
        self.mixed = 2 * key_heads * dk + heads * dv  # q, k and v
        pad = -heads % 8  # rows of the projection stay 16-byte aligned
        self.parts = [self.mixed, heads * dv, heads + pad]
        self.project, self.out = _linear(width, sum(self.parts), dtype, device), _linear(heads * dv, width, dtype, device)
        self.norm = torch.nn.Parameter(torch.ones(width, **f32))
        self.conv = torch.nn.Parameter(torch.randn(self.mixed, taps, **f32) * taps ** -0.5)
        self.q_norm, self.k_norm = torch.nn.Parameter(torch.ones(dk, **f32)), torch.nn.Parameter(torch.ones(dk, **f32))
        self.gate_norm = torch.nn.Parameter(torch.ones(heads * dv, **f32))
        self.decay_bias = torch.nn.Parameter(torch.linspace(-6.0, -1.0, heads, **f32))
        self.register_buffer("inv_freq", (10000.0 ** (-torch.arange(0, dk, 2, dtype=torch.float64) / dk)).to(device))

    def _heads(self, u):
        H, G, dk, dv = self.sizes
        q, k, v = u.split([G * dk, G * dk, H * dv], -1)
        return q.unflatten(-1, (G, dk)), k.unflatten(-1, (G, dk)), v.unflatten(-1, (H, dv))

    def _decay(self, a):
        return -torch.nn.functional.softplus(a[..., :self.sizes[0]].float() + self.decay_bias)

    def forward(self, x, residual, positions, state=None, starts=None):
        """As RecurrentBlock, with the tokens' positions (batch, length); state: of the
        convolution and of the attention."""
        conv0, s0 = (None, None) if state is None else state
        y, h = ssm.residual_norm(x, residual, self.norm)
        u, z, a = self.project(y).split(self.parts, -1)
        u, conv1 = ssm.causal_conv(u, self.conv, None, conv0, starts)
        q, k, v = self._heads(u)
        q, k = ssm.head_norm_rotary(q, k, self.q_norm, self.k_norm, positions, self.inv_freq)
        g = self._decay(a)
        if starts is not None:
            g = g.masked_fill(starts.unsqueeze(-1), -math.inf)
        o, s1 = ssm.decay_attention(q, k, v, g, None, s0)
        return self.out(ssm.gated_norm(o.flatten(2), z, self.gate_norm, self.sizes[3])), h, (conv1, s1)

    @torch.no_grad()
    def step(self, x, residual, positions, state):
        """One token: x, residual (batch, width), positions (batch,)."""
        y, h, _ = ssm.residual_norm_fwd(x, residual, self.norm)
        u, z, a = self.project(y).split(self.parts, -1)
        q, k, v = self._heads(ssm.causal_conv_update(state[0], u, self.conv))
        q, k = ssm.head_norm_rotary_fwd(q, k, self.q_norm, self.k_norm, positions, self.inv_freq)
        o = ssm.decay_attn_update(state[1], q, k, v, self._decay(a))
        o, _ = ssm.gated_norm_fwd(o.flatten(1), z, self.gate_norm, self.sizes[3])
        return self.out(o), h


def document_positions(starts):
    """Each token's distance from its document's first."""
    t = torch.arange(starts.shape[1], device=starts.device)
    first = torch.where(starts, t, torch.zeros_like(t)).cummax(1).values
    return t - first


def served(dtype=torch.bfloat16, batch=3, length=150, width=128, seed=0):
    """The largest difference, relative to the outputs' largest value, between a prompt taken at
    once by both blocks and the same prompt with its last five tokens one by one."""
    torch.manual_seed(seed)
    one = RecurrentBlock(width, 192, dtype=dtype)
    two = LinearAttentionBlock(width, 6, 2, 32, 32, dtype=dtype)
    x = torch.randn(batch, length, width, device="cuda").to(dtype)
    residual = torch.randn(batch, length, width, device="cuda")
    positions = torch.arange(length, device="cuda").expand(batch, -1).contiguous()
    with torch.no_grad():
        y, h, _ = one.prompt(x, residual)
        whole, _, _ = two(y, h, positions)
        cut = length - 5
        y, h, state1 = one.prompt(x[:, :cut].contiguous(), residual[:, :cut].contiguous())
        _, _, state2 = two(y, h, positions[:, :cut].contiguous())
        tail = []
        for t in range(cut, length):
            y, h = one.step(x[:, t], residual[:, t].contiguous(), state1)
            tail.append(two.step(y, h, positions[:, t].contiguous(), state2)[0])
    got, want = torch.stack(tail, 1).float(), whole[:, cut:].float()
    return float((got - want).abs().max() / want.abs().max())


if __name__ == "__main__":
    print(f"prompt at once against prompt and single tokens: {served():.2e} of the largest value")

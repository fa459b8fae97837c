"""Plain 64-bit references of the block operators, straight from their definitions
(step by step over time, one head at a time where heads are shared), and the
inputs the tests draw.  CPU only; shares no code with the kernels."""
from __future__ import annotations

import math

import torch

F64 = torch.float64


def attn_inputs(B, L, H, G, dk, dv, *, seed=0, decay="weak", per_token=True, state0=True, dtype=torch.float32):
    """Inputs in the storage types the kernels take (CPU)."""
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    shape = (B, L, H) if per_token else (H,)
    u = torch.rand(*shape, generator=g)
    ld = {"weak": -0.05 * u, "strong": -20.0 * u, "mixed": -torch.exp(6 * u - 4), "none": 0.0 * u,
          "growing": 0.02 * (u - 0.5), "reset": -0.1 * u}[decay]
    if decay == "reset":
        ld = ld.masked_fill(torch.rand(*shape, generator=g) < 0.15, -math.inf)
    return dict(q=r(B, L, G, dk).to(dtype), k=r(B, L, G, dk).to(dtype), v=r(B, L, H, dv).to(dtype), g=ld,
                state0=r(B, H, dk, dv) if state0 else None, do=r(B, L, H, dv).to(dtype), dfinal=r(B, H, dk, dv))


def _expand(p):
    q, k, v = (p[n].to(F64) for n in ("q", "k", "v"))
    share = v.shape[2] // q.shape[2]
    g = p["g"].to(F64)
    if g.dim() == 1:
        g = g.expand(v.shape[0], v.shape[1], -1)
    return q.repeat_interleave(share, 2), k.repeat_interleave(share, 2), v, g, share


def attn_fwd(p, scale):
    q, k, v, g, _ = _expand(p)
    B, L, H, dk = q.shape
    S = torch.zeros(B, H, dk, v.shape[3], dtype=F64) if p["state0"] is None else p["state0"].to(F64)
    o = torch.empty(v.shape, dtype=F64)
    for t in range(L):
        S = torch.exp(g[:, t])[..., None, None] * S + k[:, t, :, :, None] * v[:, t, :, None, :]
        o[:, t] = scale * (q[:, t, :, :, None] * S).sum(-2)
    return o, S


def attn_bwd(p, scale, dfinal=None):
    q, k, v, g, share = _expand(p)
    do = p["do"].to(F64)
    B, L, H, dk = q.shape
    S = torch.zeros(B, H, dk, v.shape[3], dtype=F64) if p["state0"] is None else p["state0"].to(F64)
    states = [S]
    for t in range(L):
        states.append(torch.exp(g[:, t])[..., None, None] * states[-1] + k[:, t, :, :, None] * v[:, t, :, None, :])
    R = torch.zeros_like(S) if dfinal is None else dfinal.to(F64)
    dq, dk_, dv, dg = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v), torch.empty_like(do[..., 0])
    for t in range(L - 1, -1, -1):
        R = R + scale * q[:, t, :, :, None] * do[:, t, :, None, :]
        dq[:, t] = scale * (states[t + 1] * do[:, t, :, None, :]).sum(-1)
        dk_[:, t] = (R * v[:, t, :, None, :]).sum(-1)
        dv[:, t] = (R * k[:, t, :, :, None]).sum(-2)
        e = torch.exp(g[:, t])
        dg[:, t] = e * (states[t] * R).sum((-1, -2))
        R = e[..., None, None] * R
    fold = lambda x: x.unflatten(2, (-1, share)).sum(3)  # noqa: E731
    return dict(dq=fold(dq), dk=fold(dk_), dv=dv, dlog_decay=dg if p["g"].dim() == 3 else dg.sum((0, 1)), dstate0=R)


def error(got, want):
    """The largest difference beyond what rounding the result to its type takes
    (half a unit in the last place of bf16 is 2^-8 of the value, of fp32 2^-24),
    over the largest reference value.  Values below fp32's range count as zero."""
    want = want.detach().float().to(F64)
    got = got.detach().cpu()
    u = 2.0 ** -8 if got.dtype == torch.bfloat16 else 2.0 ** -24
    assert got.shape == want.shape, (got.shape, want.shape)
    got = got.to(F64)
    assert not torch.isnan(got).any(), "NaN in result"
    over = ((got - want).abs() - u * want.abs()).clamp(min=0).max()
    scale = want.abs().max()
    return float(over if scale == 0 else over / scale)


def residual_norm_bwd(dy, dh, h, rstd, w, x, scale):
    """Gradients at the h and rstd that the forward kept."""
    dy, h, w, r = dy.to(F64), h.to(F64), w.to(F64), rstd.to(F64)[..., None]
    hat, u = h * r, dy * w
    dres = r * (u - hat * (u * hat).mean(-1, keepdim=True)) + (0 if dh is None else dh.to(F64))
    sums = lambda t: t.reshape(-1, t.shape[-1]).sum(0)  # noqa: E731
    return dict(dresidual=dres, dx=dres if scale is None else dres * scale.to(F64), dweight=sums(dy * hat),
                dscale=None if scale is None else sums(dres * x.to(F64)))


def residual_norm(x, res, w, scale, eps):
    h = res.to(F64) + x.to(F64) * (1.0 if scale is None else scale.to(F64))
    rstd = 1 / torch.sqrt((h * h).mean(-1) + eps)
    return h * rstd[..., None] * w.to(F64), h, rstd


def gated_norm(x, z, w, group, eps, gate_first, dy):
    x, w = x.to(F64).requires_grad_(), w.to(F64).requires_grad_()
    zz = None if z is None else z.to(F64).requires_grad_()
    gate = 1.0 if z is None else zz / (1 + torch.exp(-zz))
    t = x * gate if gate_first else x
    s = t.unflatten(-1, (-1, group))
    rstd = 1 / torch.sqrt((s * s).mean(-1) + eps)
    y = (s * rstd[..., None]).flatten(-2) * w
    y = y if gate_first else y * gate
    g = torch.autograd.grad(y, [x, w] + ([] if z is None else [zz]), dy.to(F64))
    return y.detach(), rstd.detach(), dict(zip(("dx", "dweight", "dz"), g))

"""Plain 64-bit references of the gated recurrence, the causal convolution and the
norm and rotation of heads, step by step from their definitions, with gradients by
autograd, and the inputs the tests draw.  CPU only; shares no code with the kernels."""
from __future__ import annotations

import torch

from tests.block_reference import F64, error  # noqa: F401


def draw(seed):
    g = torch.Generator().manual_seed(seed)
    return lambda *s: torch.randn(*s, generator=g), lambda *s: torch.rand(*s, generator=g)


def marks(B, L, starts, lengths, seed):
    g = torch.Generator().manual_seed(seed + 1000)
    st = torch.rand(B, L, generator=g) < (0.1 if L < 200 else 0.01) if starts else None
    ln = torch.randint(0, L + 1, (B,), generator=g, dtype=torch.int32) if lengths else None
    if lengths and B > 2:
        ln[0], ln[1] = 0, L
    return st, ln


# ---- gated recurrence

REC_INPUTS = ("x", "decay_gate", "input_gate", "decay", "z", "state0")


def recurrence_inputs(B, L, D, *, form="power", input_gate=True, z=True, state0=True, starts=False, lengths=False, dtype=torch.float32, seed=0):
    r, u = draw(seed)
    p = dict(x=r(B, L, D).to(dtype), decay_gate=(r(B, L, D) + (0.0 if form == "power" else 2.0)).to(dtype),
             input_gate=r(B, L, D).to(dtype) if input_gate else None,
             decay=torch.log(torch.expm1(-torch.log(0.5 + 0.499 * u(D)) / 8.0)) if form == "power" else None,
             z=r(B, L, D).to(dtype) if z else None, state0=r(B, D) if state0 else None, dy=r(B, L, D).to(dtype), dfinal=r(B, D))
    p["starts"], p["lengths"] = marks(B, L, starts, lengths, seed)
    return p


def recurrence(p, sharpness=8.0, grads=True):
    """y, final state, the state before every step, and the gradients of <y, dy> + <final, dfinal>."""
    v = {n: None if p[n] is None else p[n].detach().to(F64).clone().requires_grad_(grads) for n in REC_INPUTS}
    B, L, D = p["x"].shape
    g = torch.sigmoid(v["decay_gate"])
    if v["decay"] is not None:
        log_a = -sharpness * torch.nn.functional.softplus(v["decay"]) * g
        m = -torch.expm1(2 * log_a)
        # where the gate is zero even in 64 bits, so is the limit of all gradients through it (which go like its root)
        a, s = torch.exp(log_a), torch.where(m > 0, torch.sqrt(torch.where(m > 0, m, 1.0)), 0.0)
    else:
        a, s = g, torch.sigmoid(-v["decay_gate"])
    u = v["x"] if v["input_gate"] is None else torch.sigmoid(v["input_gate"]) * v["x"]
    h = torch.zeros(B, D, dtype=F64) if v["state0"] is None else v["state0"]
    hs, before = [], []
    for t in range(L):
        before.append(h)
        new = a[:, t] * h + s[:, t] * u[:, t]
        if p["starts"] is not None:
            new = torch.where(p["starts"][:, t, None], u[:, t], new)
        if p["lengths"] is not None:
            new = torch.where((t < p["lengths"])[:, None], new, h)
        h = new
        hs.append(h)
    y = torch.stack(hs, 1)
    if v["z"] is not None:
        y = y * v["z"] * torch.sigmoid(v["z"])
    if p["lengths"] is not None:
        y = torch.where((torch.arange(L) < p["lengths"][:, None])[..., None], y, torch.zeros_like(y))
    if not grads:
        return y, h, torch.stack(before, 1), None
    names = [n for n in REC_INPUTS if v[n] is not None]
    gr = torch.autograd.grad((y * p["dy"].to(F64)).sum() + (h * p["dfinal"].to(F64)).sum(), [v[n] for n in names], allow_unused=True)
    gr = {"d" + n: torch.zeros_like(v[n]) if t is None else t for n, t in zip(names, gr)}
    return y.detach(), h.detach(), torch.stack(before, 1).detach(), gr


# ---- causal convolution

CONV_INPUTS = ("x", "weight", "bias", "state0")


def conv_inputs(B, L, D, K, *, bias=True, state0=True, starts=False, lengths=False, dtype=torch.float32, seed=0):
    r, u = draw(seed)
    p = dict(x=r(B, L, D).to(dtype), weight=(2 * u(D, K) - 1) * K ** -0.5, bias=r(D) if bias else None,
             state0=r(B, K - 1, D).to(dtype) if state0 else None, dy=r(B, L, D).to(dtype), dfinal=r(B, K - 1, D).to(dtype))
    p["starts"], p["lengths"] = marks(B, L, starts, lengths, seed)
    return p


def conv(p, silu=True, grads=True):
    """y, final state, gradients of <y, dy> + <final, dfinal>; one row and step at a time."""
    v = {n: None if p[n] is None else p[n].detach().to(F64).clone().requires_grad_(grads) for n in CONV_INPUTS}
    B, L, D = p["x"].shape
    K = p["weight"].shape[1]
    zero = torch.zeros(D, dtype=F64)
    ys, finals = [], []
    for b in range(B):
        win = [zero] * (K - 1) if v["state0"] is None else [v["state0"][b, j] for j in range(K - 1)]
        n = L if p["lengths"] is None else int(p["lengths"][b])
        for t in range(L):
            if t >= n:
                ys.append(zero)
                continue
            if p["starts"] is not None and p["starts"][b, t]:
                win = [zero] * (K - 1)
            taps = win + [v["x"][b, t]]
            pre = sum(v["weight"][:, k] * taps[k] for k in range(K))
            if v["bias"] is not None:
                pre = pre + v["bias"]
            ys.append(pre * torch.sigmoid(pre) if silu else pre)
            win = taps[1:]
        finals += win
    y = torch.stack(ys).view(B, L, D)
    final = torch.stack(finals).view(B, K - 1, D) if K > 1 else torch.zeros(B, 0, D, dtype=F64)
    if not grads:
        return y, final, None
    names = [n for n in CONV_INPUTS if v[n] is not None]
    gr = torch.autograd.grad((y * p["dy"].to(F64)).sum() + (final * p["dfinal"].to(F64)).sum(), [v[n] for n in names], allow_unused=True)
    return y.detach(), final.detach(), {"d" + n: torch.zeros_like(v[n]) if t is None else t for n, t in zip(names, gr)}


# ---- norm and rotation of heads

HEAD_INPUTS = ("q", "k", "q_weight", "k_weight")


def head_inputs(B, L, Hq, Hk, d, rot, *, weights="shared", per_batch=True, far=False, dtype=torch.float32, seed=0):
    r, _ = draw(seed)
    lead = (B,) if L is None else (B, L)
    shape = lambda H: (H, d) if weights == "per head" else (d,)  # noqa: E731
    p = dict(q=(2 * r(*lead, Hq, d)).to(dtype), k=(2 * r(*lead, Hk, d)).to(dtype) if Hk else None,
             q_weight=1 + 0.2 * r(*shape(Hq)) if weights else None, k_weight=1 + 0.2 * r(*shape(Hk)) if weights and Hk else None,
             dq_out=r(*lead, Hq, d).to(dtype), dk_out=r(*lead, Hk, d).to(dtype) if Hk else None, positions=None, inv_freq=None)
    if rot:
        g = torch.Generator().manual_seed(seed + 7)
        shape = lead if per_batch or L is None else lead[1:]
        p["positions"] = torch.randint(-5, 2 ** 31 if far else 5000, shape, generator=g)
        p["inv_freq"] = 10000.0 ** (-torch.arange(0, rot, 2, dtype=F64) / rot)
    return p


def heads(p, eps=1e-6, norm=True, interleaved=False, grads=True):
    v = {n: None if p[n] is None else p[n].detach().to(F64).clone().requires_grad_(grads) for n in HEAD_INPUTS}
    outs = {}
    for n in ("q", "k"):
        x = v[n]
        if x is None:
            continue
        if norm:
            x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
        if v[n + "_weight"] is not None:
            x = x * v[n + "_weight"]
        if p["positions"] is not None:
            rot = 2 * p["inv_freq"].numel()
            ang = (p["positions"].to(F64)[..., None, None] * p["inv_freq"])
            cos, sin = torch.cos(ang), torch.sin(ang)
            i = torch.arange(rot // 2)
            a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
            xa, xb = x[..., a], x[..., b]
            new = x.clone()
            new[..., a] = xa * cos - xb * sin
            new[..., b] = xb * cos + xa * sin
            x = new
        outs[n] = x
    if not grads:
        return outs, None
    names = [n for n in HEAD_INPUTS if v[n] is not None]
    loss = sum((outs[n] * p["d" + n + "_out"].to(F64)).sum() for n in outs)
    gr = torch.autograd.grad(loss, [v[n] for n in names])
    return {n: t.detach() for n, t in outs.items()}, {"d" + n: t for n, t in zip(names, gr)}


def on_gpu(p):
    return {n: None if t is None else t.cuda() for n, t in p.items()}


# ---- the convolution at sizes of training, all steps at once


def conv_at_once(p, silu=True):
    """As conv, on the inputs' device: every tap as a shifted tensor, masked where a document starts between."""
    v = {n: None if p[n] is None else p[n].detach().to(F64).clone().requires_grad_() for n in CONV_INPUTS}
    B, L, D = p["x"].shape
    K, dev = p["weight"].shape[1], p["x"].device
    end = torch.full((B,), L, device=dev) if p["lengths"] is None else p["lengths"].long()
    on = (torch.arange(L, device=dev) < end[:, None])[..., None]
    doc = torch.zeros(B, L, dtype=torch.int64, device=dev) if p["starts"] is None else p["starts"].long().cumsum(1)
    doc = torch.cat([doc.new_zeros(B, K - 1), doc], 1)  # a state's inputs belong to the row's first document
    head = v["x"].new_zeros(B, K - 1, D) if v["state0"] is None else v["state0"]
    xs = torch.cat([head, torch.where(on, v["x"], 0.0)], 1)
    pre = torch.zeros_like(v["x"]) if v["bias"] is None else v["bias"].expand(B, L, D)
    for k in range(K):
        pre = pre + v["weight"][:, k] * torch.where((doc[:, k:k + L] == doc[:, K - 1:])[..., None], xs[:, k:k + L], 0.0)
    y = torch.where(on, pre * torch.sigmoid(pre) if silu else pre, 0.0)
    at = end[:, None] + torch.arange(K - 1, device=dev)  # the last K - 1 inputs; at - (K - 1) is a step
    last = doc.gather(1, (end + K - 2).clamp(min=0)[:, None])
    final = torch.where((doc.gather(1, at) == last)[..., None], xs.gather(1, at[..., None].expand(-1, -1, D)), 0.0)
    names = [n for n in CONV_INPUTS if v[n] is not None]
    gr = torch.autograd.grad((y * p["dy"].to(F64)).sum() + (final * p["dfinal"].to(F64)).sum(), [v[n] for n in names], allow_unused=True)
    return y.detach(), final.detach(), {"d" + n: torch.zeros_like(v[n]) if t is None else t for n, t in zip(names, gr)}

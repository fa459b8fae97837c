"""The 64-bit references of the block operators: the gradient formulas of decay
attention against differences of its definition, and against its closed forms."""
from __future__ import annotations

import pytest
import torch

from tests import block_reference as ref


def _double(p):
    return {n: None if t is None else t.double() for n, t in p.items()}


@pytest.mark.parametrize("H,G,per_token", [(2, 2, True), (4, 2, True), (3, 1, False)])
def test_gradients_are_differences(H, G, per_token):
    p = _double(ref.attn_inputs(2, 5, H, G, 4, 3, seed=H, decay="mixed", per_token=per_token))
    scale, step = 0.7, 1e-6
    grads = ref.attn_bwd(p, scale, p["dfinal"])
    loss = lambda q: sum((a * b).sum() for a, b in zip(ref.attn_fwd(q, scale), (q["do"], q["dfinal"])))  # noqa: E731
    names = dict(q="dq", k="dk", v="dv", g="dlog_decay", state0="dstate0")
    gen = torch.Generator().manual_seed(1)
    for n, dn in names.items():
        d = torch.randn(p[n].shape, generator=gen, dtype=torch.float64)
        up, down = dict(p), dict(p)
        up[n], down[n] = p[n] + step * d, p[n] - step * d
        diff = float(loss(up) - loss(down)) / (2 * step)
        # central difference: error step^2 of the third derivative and 1e-16 / step of the loss
        assert diff == pytest.approx(float((grads[dn] * d).sum()), rel=1e-6, abs=1e-6), n


def test_no_decay_is_a_plain_sum():
    p = _double(ref.attn_inputs(1, 6, 1, 1, 3, 2, decay="none", state0=False))
    o, S = ref.attn_fwd(p, 1.0)
    q, k, v = (p[n][0, :, 0] for n in "qkv")
    assert torch.allclose(o[0, :, 0], torch.tril(q @ k.T) @ v, atol=1e-13)
    assert torch.allclose(S[0, 0], k.T @ v, atol=1e-13)


def test_reset_forgets():
    p = _double(ref.attn_inputs(1, 6, 1, 1, 3, 2, decay="weak"))
    p["g"][0, 4, 0] = -float("inf")
    o, S = ref.attn_fwd(p, 1.0)
    tail = {n: (t[:, 4:] if n in ("q", "k", "v", "g", "do") else t) for n, t in p.items()}
    tail["state0"] = None
    tail["g"] = tail["g"].clamp(min=-1.0)
    o2, S2 = ref.attn_fwd(tail, 1.0)
    assert torch.equal(o[:, 4:], o2) and torch.equal(S, S2)


@pytest.mark.parametrize("scaled,with_dh", [(True, True), (False, False)])
def test_residual_norm_gradients_are_differences(scaled, with_dh):
    gen = torch.Generator().manual_seed(2)
    r = lambda *s: torch.randn(*s, generator=gen, dtype=torch.float64)  # noqa: E731
    p = dict(x=r(3, 6), res=r(3, 6), w=r(6), scale=r(6) if scaled else None)
    dy, dh = r(3, 6), r(3, 6) if with_dh else None
    f = lambda p: ref.residual_norm(p["x"], p["res"], p["w"], p["scale"], 1e-3)  # noqa: E731
    y, h, rstd = f(p)
    g = ref.residual_norm_bwd(dy, dh, h, rstd, p["w"], p["x"], p["scale"])
    loss = lambda p: float((f(p)[0] * dy).sum() + (0 if dh is None else (f(p)[1] * dh).sum()))  # noqa: E731
    for n, dn in (("x", "dx"), ("res", "dresidual"), ("w", "dweight"), ("scale", "dscale")):
        if p[n] is None:
            continue
        d, step = r(*p[n].shape), 1e-6
        diff = (loss({**p, n: p[n] + step * d}) - loss({**p, n: p[n] - step * d})) / (2 * step)
        assert diff == pytest.approx(float((g[dn] * d).sum()), rel=1e-6, abs=1e-7), n

"""The block operators' autograd functions without a GPU, with plain stand-ins
for the kernels' calls: their backward is not differentiable, and says so."""
from __future__ import annotations

import pytest
import torch

from selective_state_space_10_amd import block_ops


def _gated(monkeypatch):
    monkeypatch.setattr(block_ops, "gated_norm_fwd", lambda x, z, w, *a: ((x * w * z).detach(), x.detach().mean(-1, keepdim=True)))
    monkeypatch.setattr(block_ops, "gated_norm_bwd", lambda dy, x, z, w, r, *a: {n: t.detach() for n, t in dict(
        dx=dy * w * z, dz=dy * x * w, dweight=(dy * x * z).sum(0)).items()})
    x, z, w = torch.rand(3, 8), torch.rand(3, 8), torch.rand(8)
    return (x, z, w), lambda x, z, w: block_ops.gated_norm(x, z, w)


def _residual(monkeypatch):
    monkeypatch.setattr(block_ops, "residual_norm_fwd", lambda x, r, w, *a: (((x + r) * w).detach(), (x + r).detach(), x.detach().mean(-1)))
    monkeypatch.setattr(block_ops, "residual_norm_bwd", lambda dy, dh, h, rstd, w, *a: {n: t.detach() if t is not None else None for n, t in dict(
        dx=dy * w, dresidual=dy * w, dweight=(dy * h).sum(0), dscale=None).items()})
    return (torch.rand(3, 8), torch.rand(3, 8), torch.rand(8)), lambda x, r, w: block_ops.residual_norm(x, r, w)[0]


def _attention(monkeypatch):
    monkeypatch.setattr(block_ops, "decay_attn_fwd", lambda q, k, v, *a, **kw: ((q * k * v).detach(), torch.zeros(1)))
    monkeypatch.setattr(block_ops, "decay_attn_bwd", lambda q, k, v, g, do, *a, **kw: {n: t.detach() if t is not None else None for n, t in dict(
        dq=do * k * v, dk=do * q * v, dv=do * q * k, dlog_decay=None, dstate0=None).items()})
    return tuple(torch.rand(1, 4, 2, 8) for _ in range(3)), lambda q, k, v: block_ops.decay_attention(q, k, v, torch.zeros(2))[0]


@pytest.mark.parametrize("make", [_gated, _residual, _attention])
def test_a_second_derivative_is_refused(monkeypatch, make):
    """Without an error the operator's part of it would be missing."""
    inputs, f = make(monkeypatch)
    inputs = [t.requires_grad_() for t in inputs]
    y = f(*inputs)
    loss = y.square().sum() + inputs[0].pow(3).sum()  # another term keeps the graph alive
    first, = torch.autograd.grad(loss, inputs[0], create_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        first.square().sum().backward()


@pytest.mark.parametrize("make", [_gated, _residual, _attention])
def test_first_derivatives_are_as_before(monkeypatch, make):
    inputs, f = make(monkeypatch)
    inputs = [t.requires_grad_() for t in inputs]
    y = f(*inputs)
    a = torch.autograd.grad(y.sum(), inputs, retain_graph=True)
    b = torch.autograd.grad(y.sum(), inputs, create_graph=True)
    assert all(torch.equal(s, t) for s, t in zip(a, b))

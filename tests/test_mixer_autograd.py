"""The autograd functions of the gated recurrence, the causal convolution and the norm
and rotation of heads without a GPU, with plain stand-ins for the kernels' calls:
their backward is not differentiable, and says so."""
from __future__ import annotations

import pytest
import torch

from selective_state_space_10_amd import mixer_ops


def _detached(d):
    return {n: None if t is None else t.detach() for n, t in d.items()}


def _recurrence(monkeypatch):
    monkeypatch.setattr(mixer_ops, "gated_recurrence_fwd", lambda x, g, *a, **kw: ((x * g).detach(), torch.zeros(1), torch.zeros(1)))
    monkeypatch.setattr(mixer_ops, "gated_recurrence_bwd", lambda dy, x, g, *a, **kw: _detached(dict(
        dx=dy * g, ddecay_gate=dy * x, dinput_gate=None, ddecay=None, dz=None, dstate0=None)))
    return (torch.rand(2, 3, 8), torch.rand(2, 3, 8)), lambda x, g: mixer_ops.gated_recurrence(x, g)[0]


def _conv(monkeypatch):
    monkeypatch.setattr(mixer_ops, "causal_conv_fwd", lambda x, w, *a, **kw: ((x * w[:, 0]).detach(), torch.zeros(1)))
    monkeypatch.setattr(mixer_ops, "causal_conv_bwd", lambda dy, x, w, *a, **kw: _detached(dict(
        dx=dy * w[:, 0], dweight=(dy * x).sum((0, 1))[:, None], dbias=None, dstate0=None)))
    return (torch.rand(2, 3, 8), torch.rand(8, 1)), lambda x, w: mixer_ops.causal_conv(x, w)[0]


def _heads(monkeypatch):
    monkeypatch.setattr(mixer_ops, "head_norm_rotary_fwd", lambda q, k, w, *a, **kw: ((q * w).detach(), k.detach().clone()))
    monkeypatch.setattr(mixer_ops, "head_norm_rotary_bwd", lambda dq, dk, q, k, w, *a, **kw: _detached(dict(
        dq=dq * w, dk=dk, dq_weight=(dq * q).sum((0, 1, 2)), dk_weight=None)))
    return (torch.rand(2, 3, 2, 8), torch.rand(2, 3, 2, 8), torch.rand(8)), lambda q, k, w: sum(mixer_ops.head_norm_rotary(q, k, w, w))


@pytest.mark.parametrize("make", [_recurrence, _conv, _heads])
def test_a_second_derivative_is_refused(monkeypatch, make):
    """Without an error the operator's part of it would be missing."""
    inputs, f = make(monkeypatch)
    inputs = [t.requires_grad_() for t in inputs]
    loss = f(*inputs).square().sum() + inputs[0].pow(3).sum()  # another term keeps the graph alive
    first, = torch.autograd.grad(loss, inputs[0], create_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        first.square().sum().backward()


@pytest.mark.parametrize("make", [_recurrence, _conv, _heads])
def test_first_derivatives(monkeypatch, make):
    inputs, f = make(monkeypatch)
    inputs = [t.requires_grad_() for t in inputs]
    y = f(*inputs)
    a = torch.autograd.grad(y.sum(), inputs, retain_graph=True)
    b = torch.autograd.grad(y.sum(), inputs, create_graph=True)
    assert all(torch.equal(s, t) for s, t in zip(a, b))


def test_functions_with_the_fewest_arguments(monkeypatch):
    """The functions' own defaults: apply() sees only the arguments that it was given."""
    from selective_state_space_10_amd import block_ops
    (x, g), _ = _recurrence(monkeypatch)
    x.requires_grad_()
    mixer_ops.GatedRecurrenceFn.apply(x, g)[0].sum().backward()
    assert torch.equal(x.grad, g)
    (x, w), _ = _conv(monkeypatch)
    x.requires_grad_()
    mixer_ops.CausalConvFn.apply(x, w)[0].sum().backward()
    assert torch.equal(x.grad, w[:, 0].expand_as(x))
    monkeypatch.setattr(block_ops, "decay_attn_fwd", lambda q, k, v, *a, **kw: ((q * v).detach(), torch.zeros(1)))
    monkeypatch.setattr(block_ops, "decay_attn_bwd", lambda q, k, v, g, do, *a, **kw: dict(
        dq=do * v, dk=None, dv=None, dlog_decay=None, dstate0=None))
    q, v = torch.rand(2, 3, 2, 8, requires_grad=True), torch.rand(2, 3, 2, 8)
    block_ops.DecayAttentionFn.apply(q, v, v, torch.rand(2))[0].sum().backward()
    assert torch.equal(q.grad, v)


def test_tensors_must_be_on_a_gpu():
    t = torch.zeros(2, 3, 8)
    with pytest.raises(ValueError, match="GPU"):
        mixer_ops.gated_recurrence_fwd(t, t)
    with pytest.raises(ValueError, match="GPU"):
        mixer_ops.causal_conv_fwd(t, torch.zeros(8, 4))
    with pytest.raises(ValueError, match="GPU"):
        mixer_ops.head_norm_rotary_fwd(t)

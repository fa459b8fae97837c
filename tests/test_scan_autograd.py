"""The scan's autograd functions without a GPU, with plain stand-ins for the
kernels' calls: their backward is not differentiable, and says so."""
from __future__ import annotations

import pytest
import torch

from selective_state_space_10_amd import ops

N, L, D = 2, 4, 8
NAMES = ("ddelta", "dA", "dB", "dC", "dD", "dz", "ddelta_bias", "dh0", "dconv_w", "dconv_b")


def _scan(monkeypatch):
    monkeypatch.setattr(ops, "scan_fwd", lambda u, delta, *a, **kw: ((u * delta).detach(), torch.zeros(1), torch.zeros(1)))
    monkeypatch.setattr(ops, "scan_bwd", lambda u, delta, *a, **kw: dict.fromkeys(NAMES) | {"du": (a[9] * delta).detach()})
    return lambda u, t: ops.selective_scan(u, t, *[torch.zeros(1)] * 3)[0]


def _conv(monkeypatch):
    monkeypatch.setattr(ops, "scan_fwd_conv", lambda x, w, b, delta, *a, **kw: ((x * delta).detach(), torch.zeros(1), torch.zeros(1)))
    monkeypatch.setattr(ops, "scan_bwd_conv", lambda x, w, b, delta, *a, **kw: dict.fromkeys(NAMES) | {"dx": (a[9] * delta).detach()})
    return lambda u, t: ops.conv_selective_scan(u, torch.zeros(1), None, t, *[torch.zeros(1)] * 3)[0]


@pytest.mark.parametrize("make", [_scan, _conv])
def test_a_second_derivative_is_refused(monkeypatch, make):
    """Without an error the scan's part of it would be missing."""
    f = make(monkeypatch)
    u, delta = torch.rand(1, L, D, requires_grad=True), torch.rand(1, L, D)
    y = f(u, delta)
    first, = torch.autograd.grad(y.square().sum() + u.pow(3).sum(), u, create_graph=True)
    assert torch.allclose(first, 2 * y * delta + 3 * u.square())
    with pytest.raises(RuntimeError, match="once_differentiable"):
        first.square().sum().backward()

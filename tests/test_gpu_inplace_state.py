"""Tensors that a call writes in place count as modified: a backward that saved
one before is refused, as with PyTorch's own operations."""
from __future__ import annotations

import pytest
import torch

from tests import block_reference as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ssm():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import selective_state_space_10_amd as m
    m.load()
    return m


def _token(ssm, d, state):
    return ssm.decay_attn_update(state, d["q"][:, 0], d["k"][:, 0], d["v"][:, 0], d["g"][:, 0].contiguous())


def test_a_decay_attention_state_updated_after_it_was_saved(ssm):
    d = {n: t.cuda() for n, t in ref.attn_inputs(1, 5, 2, 2, 16, 16).items()}
    state, q = d["state0"], d["q"].clone().requires_grad_()
    o, _ = ssm.decay_attention(q, d["k"], d["v"], d["g"], None, state)
    version = state._version
    _token(ssm, d, state)
    assert state._version > version
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        o.sum().backward()


def test_states_made_in_inference_mode_are_taken(ssm):
    with torch.inference_mode():
        d = {n: t.cuda() for n, t in ref.attn_inputs(1, 5, 2, 2, 16, 16).items()}
        inside = _token(ssm, d, d["state0"].clone())
        state = d["state0"].clone()
    assert torch.equal(_token(ssm, d, state), inside)


def _scan_inputs():
    gen = torch.Generator().manual_seed(1)
    r = lambda *s: torch.randn(*s, generator=gen).cuda()  # noqa: E731
    B, L, D, N = 1, 20, 64, 16
    return r(B, L, D), r(B, L, D) - 2, -r(D, N).exp(), r(B, L, N), r(B, L, N), r(B, D, N)


def test_a_scan_state_updated_after_it_was_saved(ssm):
    u, delta, A, B, C, h0 = _scan_inputs()
    y, _ = ssm.selective_scan(u.requires_grad_(), delta, A, B, C, h0=h0)
    version = h0._version
    ssm.state_update(h0, u.detach()[:, 0].contiguous(), delta[:, 0].contiguous(), A, B[:, 0].contiguous(), C[:, 0].contiguous())
    assert h0._version > version
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.sum().backward()


@pytest.mark.parametrize("conv", [False, True])
def test_an_output_that_is_added_to(ssm, conv):
    u, delta, A, B, C, _ = _scan_inputs()
    x = torch.ones_like(u, requires_grad=True)
    out = torch.zeros_like(u)
    y = (x * out).sum()
    if conv:
        ssm.scan_fwd_conv(u, torch.ones(u.shape[-1], 4, device="cuda"), None, delta, A, B, C, out=out)
    else:
        ssm.scan_fwd(u, delta, A, B, C, out=out)
    assert out.any()
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward()

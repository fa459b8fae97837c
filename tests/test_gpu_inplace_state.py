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

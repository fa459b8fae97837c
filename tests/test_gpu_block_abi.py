"""The block operators' C ABI on the GPU: what it does not use it does not check."""
from __future__ import annotations

import ctypes

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("step", [-1, 3, 1 << 50])
def test_a_single_token_has_no_step_stride(step):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import selective_state_space_10_amd as m
    from selective_state_space_10_amd import _lib
    lib = m.load()
    B, H, dk, dv = 2, 3, 16, 24
    gen = torch.Generator().manual_seed(0)
    r = lambda *s: torch.randn(*s, generator=gen).cuda()  # noqa: E731
    q, k, v, g, state = r(B, H, dk), r(B, H, dk), r(B, H, dv), -r(B, H).abs(), r(B, H, dk, dv)
    other, o = state.clone(), torch.empty_like(v)
    view = lambda t: ctypes.byref(_lib.View4(t.data_ptr(), t.stride(0), step, t.stride(1)))  # noqa: E731
    status = lib.ssm_decay_attn_update(B, H, H, dk, dv, 0, state.data_ptr(), view(q), view(k), view(v), g.data_ptr(), 1, 0.5,
                                       o.data_ptr(), torch.cuda.current_stream().cuda_stream)
    assert status == 0, lib.ssm_last_error()
    assert torch.equal(o, m.decay_attn_update(other, q, k, v, g, 0.5)) and torch.equal(state, other)

"""How decay attention splits sequences, read from its workspaces (host queries,
256 CUs).  The shapes' times by segments, us, forward: 1 x 512, 8 heads of 64,
bf16: 4 segments 17.1, 8: 13.1; 32 heads 17.4 and 13.9.  The states before fewer
than 24 segments are folded without a kernel of their own, so none is charged."""
from __future__ import annotations

import pytest


def _segments(B, L, H, dk, dv, io):
    from selective_state_space_10_amd import _lib
    nbytes = _lib.load().ssm_decay_attn_fwd_workspace_bytes(B, L, H, H, dk, dv, io)
    pad = next(p for p in (32, 64, 128, 256) if dk <= p)
    cols = 64 if dv <= 64 else -(-dv // 128) * 128
    return max(1, round(nbytes / (B * H * (pad * cols + 2) * 4)))


@pytest.mark.parametrize("shape,want", [((1, 512, 8, 64, 64, 1), 8), ((1, 512, 32, 64, 64, 1), 8), ((8, 2048, 16, 128, 128, 1), 4),
                                        ((1, 32768, 40, 128, 128, 1), 12), ((3, 1111, 8, 72, 96, 0), 9), ((1, 37, 4, 32, 32, 0), 1)])
def test_segments(shape, want):
    assert _segments(*shape) == want

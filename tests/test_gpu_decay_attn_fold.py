"""Decay attention split into so many segments that the workgroups of the backward
fold the states before them (dv's transposed) where states are narrow, and a
kernel of its own computes them where they are wide.

References and tolerances are those of tests/test_gpu_decay_attn.py."""
from __future__ import annotations

import pytest
import torch

from tests import block_reference as ref
from tests.test_gpu_decay_attn import _compare
from tests.test_gpu_decay_attn_split import _segments

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module")
def ssm():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import selective_state_space_10_amd as m
    m.load()
    return m


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("B,L,H,G,dk,dv", [(1, 512, 8, 4, 64, 64), (2, 500, 3, 1, 24, 136), (1, 330, 4, 2, 136, 40), (1, 576, 2, 2, 72, 200),
                                           (1, 570, 3, 1, 48, 40), (1, 440, 4, 2, 72, 104)])
@pytest.mark.parametrize("decay,per_token", [("weak", True), ("reset", True), ("mixed", False)])
def test_five_to_nine_segments(ssm, dtype, B, L, H, G, dk, dv, decay, per_token):
    n = _segments(ssm, B, L, H, G, dk, dv, dtype)
    print("segments", n, flush=True)
    assert 5 <= n <= 9
    _compare(ssm, ref.attn_inputs(B, L, H, G, dk, dv, seed=L, decay=decay, per_token=per_token, dtype=dtype))

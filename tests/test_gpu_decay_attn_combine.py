"""Decay attention, forward, with the states before so many segments that they
are computed by a kernel of their own.

References and tolerances are those of tests/test_gpu_decay_attn.py."""
from __future__ import annotations

import pytest
import torch

from tests import block_reference as ref
from tests.test_gpu_decay_attn import _check, _gpu
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
@pytest.mark.parametrize("L,H,G,dk,dv", [(1100, 2, 1, 24, 40), (1700, 3, 3, 72, 200), (2100, 1, 1, 136, 24), (4133, 2, 2, 32, 32)])
@pytest.mark.parametrize("decay", ["weak", "reset"])
def test_states_before_many_segments(ssm, dtype, L, H, G, dk, dv, decay):
    n = _segments(ssm, 1, L, H, G, dk, dv, dtype)
    print("segments", n, flush=True)
    assert n >= 16
    cpu = ref.attn_inputs(1, L, H, G, dk, dv, seed=L, decay=decay, dtype=dtype)
    want_o, want_s = ref.attn_fwd(cpu, dk ** -0.5)
    d = _gpu(cpu)
    o, s = ssm.decay_attn_fwd(d["q"], d["k"], d["v"], d["g"], None, d["state0"], return_final_state=True)
    _check(o, want_o, dtype)
    _check(s, want_s, F32)

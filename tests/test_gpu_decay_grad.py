"""The gradient of the decays, which is put together from sums between edges.

References and tolerances are those of tests/test_gpu_decay_attn.py: 64 bits, and
for the decays' gradient twice the bound of fp32."""
from __future__ import annotations

import math

import pytest
import torch

from tests import block_reference as ref
from tests.test_gpu_decay_attn import _check, _gpu

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
@pytest.mark.parametrize("at", [0, 100, 300, 698])
def test_a_nan_stays_before_later_steps(ssm, dtype, at):
    """A NaN in do at a step leaves the gradient at later decays as it was."""
    cpu = ref.attn_inputs(1, 700, 2, 1, 40, 64, seed=at, dtype=dtype)
    want = ref.attn_bwd(cpu, 40 ** -0.5, cpu["dfinal"])["dlog_decay"]
    d = _gpu(cpu)
    d["do"][:, at] = math.nan
    g = ssm.decay_attn_bwd(d["q"], d["k"], d["v"], d["g"], d["do"], None, d["state0"], d["dfinal"])["dlog_decay"]
    assert torch.isnan(g[:, :at + 1]).all()
    _check(g[:, at + 1:], want[:, at + 1:], F32, 2)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("state0,dfinal", [(False, False), (True, False), (False, True), (True, True)])
@pytest.mark.parametrize("L,dk,dv", [(1, 32, 32), (63, 64, 64), (256, 104, 112), (1025, 104, 112), (2353, 128, 40)])
@pytest.mark.parametrize("per_token", [True, False])
def test_edges_and_given_states(ssm, dtype, state0, dfinal, L, dk, dv, per_token):
    cpu = ref.attn_inputs(1, L, 2, 2, dk, dv, seed=L, per_token=per_token, dtype=dtype)
    if not state0:
        cpu["state0"] = None
    df = cpu["dfinal"] if dfinal else None
    want = ref.attn_bwd(cpu, dk ** -0.5, df)["dlog_decay"]
    d = _gpu(cpu)
    g = ssm.decay_attn_bwd(d["q"], d["k"], d["v"], d["g"], d["do"], None, d["state0"], None if df is None else d["dfinal"],
                           want_dstate0=state0)["dlog_decay"]
    _check(g, want, F32, 2)

"""Decays above one: factors of many steps that exceed fp32's range, where the
recurrence itself stays within it.

References and tolerances are those of tests/test_gpu_decay_attn.py."""
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


def _quiet(p, steps, *names):
    for n in names:
        p[n][:, steps] = 0
    return p


def _cases(dtype, L):
    """(name, inputs, whether the gradients' states stay in range as well)."""
    new = lambda **kw: ref.attn_inputs(1, L, 2, 1, 32, 40, seed=L, dtype=dtype, **{"state0": False, **kw})  # noqa: E731
    p = new()
    p["g"][:, 0] = p["g"][:, 1] = 60.0
    yield "two large steps from nothing", p, True
    p = new()
    p["g"][:, 0] = 100.0
    yield "one decay beyond fp32 from nothing", p, True
    p = new()
    p["g"][:, :L - 5] = 5.0
    yield "growth before anything is there", _quiet(p, slice(0, L - 3), "q", "k", "v", "do"), False
    p = new()
    p["g"][:, :12] = 12.0
    yield "growth over steps without keys", _quiet(p, slice(0, 12), "q", "k", "do"), False
    p = new()
    p["g"][:, :12] = 12.0
    yield "growth over steps without values", _quiet(p, slice(0, 12), "q", "v", "do"), False
    p = new(state0=True)
    p["state0"] *= 1e-30
    p["g"][:, :20] = 5.0
    yield "a small state grows", _quiet(p, slice(0, 20), "q", "k", "v", "do"), False
    p = new(state0=True)
    p["g"][:, 3:L - 2:7] = 70.0
    p["g"][:, 4:L - 1:7] = -80.0
    yield "up and down", p, True


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("L", [33, 64, 130, 700])
@pytest.mark.parametrize("case", range(7))
def test_factors_beyond_the_range_of_fp32(ssm, dtype, L, case):
    name, p, back = list(_cases(dtype, L))[case]
    print(name, L, flush=True)
    ro, rs = ref.attn_fwd(p, 32 ** -0.5)
    rg = ref.attn_bwd(p, 32 ** -0.5)
    assert float(ro.abs().max()) < 1e38 and float(rs.abs().max()) < 1e38
    d = _gpu(p)
    o, s = ssm.decay_attn_fwd(d["q"], d["k"], d["v"], d["g"], None, d["state0"], return_final_state=True)
    g = ssm.decay_attn_bwd(d["q"], d["k"], d["v"], d["g"], d["do"], None, d["state0"], want_dstate0=False)
    _check(o, ro, dtype)
    _check(s, rs, F32)
    for n in ("dq", "dk", "dv") if back else ("dq",):
        _check(g[n], rg[n], dtype)
    if back:
        _check(g["dlog_decay"], rg["dlog_decay"], F32, 2)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_gradients_from_the_end_grow(ssm, dtype):
    """No gradient reaches the last steps, whose decays exceed fp32's range together."""
    p = ref.attn_inputs(1, 150, 2, 1, 32, 40, seed=1, state0=False, dtype=dtype)
    p["g"][:, 120:] = 11.0
    p["do"][:, 110:] = 0
    rg = ref.attn_bwd(p, 32 ** -0.5)
    d = _gpu(p)
    g = ssm.decay_attn_bwd(d["q"], d["k"], d["v"], d["g"], d["do"], want_dlog_decay=False, want_dstate0=False)
    for n in ("dk", "dv"):
        _check(g[n], rg[n], dtype)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_infinite_growth_reaches_no_earlier_step(ssm, dtype, bad):
    p = ref.attn_inputs(1, 150, 2, 2, 32, 32, seed=6, dtype=dtype)
    p["g"][:, 5::9] = 4.0
    p["g"][:, 6::9] = -4.0
    ro, _ = ref.attn_fwd(p, 32 ** -0.5)
    d = _gpu(p)
    d["g"][:, 70] = bad
    o, _ = ssm.decay_attn_fwd(d["q"], d["k"], d["v"], d["g"], None, d["state0"])
    _check(o[:, :70], ro[:, :70], dtype)
    assert not torch.isfinite(o[:, 70:]).any()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("L,at", [(60, 10), (700, 10), (700, 500), (5000, 10)])
def test_a_cleared_state_leaves_nothing(ssm, dtype, L, at):
    """However large it was: not 2^-256 of it."""
    d = _gpu(ref.attn_inputs(1, L, 2, 2, 32, 40, seed=3, decay="none", dtype=dtype))
    d["g"][:, at] = -math.inf
    d["k"].zero_()
    large = torch.full_like(d["state0"], 2.0 ** 110)
    o, s = ssm.decay_attn_fwd(d["q"], d["k"], d["v"], d["g"], None, large, return_final_state=True)
    assert o[:, at - 1].any()
    assert not o[:, at:].any() and not s.any()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("L", [64, 700])
def test_growth_after_a_cleared_state(ssm, dtype, L):
    """By more than 2^256, which is how small a cleared state may be counted."""
    p = ref.attn_inputs(1, L, 2, 1, 32, 40, seed=3, dtype=dtype)
    p["g"][:, 10] = -math.inf
    p["g"][:, 11:51] = 6.0
    _quiet(p, slice(10, 51), "k", "do")
    ro, rs = ref.attn_fwd(p, 32 ** -0.5)
    rg = ref.attn_bwd(p, 32 ** -0.5)
    d = _gpu(p)
    o, s = ssm.decay_attn_fwd(d["q"], d["k"], d["v"], d["g"], None, d["state0"], return_final_state=True)
    g = ssm.decay_attn_bwd(d["q"], d["k"], d["v"], d["g"], d["do"], None, d["state0"], want_dlog_decay=False, want_dstate0=False)
    _check(o, ro, dtype)
    _check(s, rs, F32)
    _check(g["dq"], rg["dq"], dtype)

"""Decay attention with inputs that show how many bits its products keep.

Exact sums: every operand is a bf16 value or a sum of powers of two 2^0 .. 2^-20,
and so is every partial sum (at most 22 bits), so fp32 arithmetic gives 2^-20
where operands that were cut to two bf16 pieces (16 bits) give 0 or 2^-12.

Like-signed sums: errors that all point one way add up.  Units of 2^-24 of the
result: a product of operands in three bf16 pieces rounded to nearest leaves out
at most 1, its sum is rounded last to 1 (2 if cut off), the multiplication by a
decay rounds to 1."""
from __future__ import annotations

import pytest
import torch

from tests import block_reference as ref

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
TINY = 2.0 ** -20
ONE, CANCEL = (1.0, 1.0, 1.0), ((1.0, 2.0 ** -8, TINY), (-1.0, -2.0 ** -8, 0.0))


@pytest.fixture(scope="module")
def ssm():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import selective_state_space_10_amd as m
    m.load()
    return m


def _rows(d, dtype, *rows):
    """(1, steps, 1, d): the given leading elements of each step, zeros after them."""
    t = torch.zeros(1, len(rows), 1, d, dtype=dtype)
    for i, r in enumerate(rows):
        t[0, i, 0, :len(r)] = torch.tensor(r)
    return t.cuda()


def _ones(d, dtype, steps=2):
    return torch.ones(1, steps, 1, d, dtype=dtype, device="cuda")


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("dk,dv", [(32, 16), (64, 72), (128, 128), (256, 40)])
def test_weights_of_steps_keep_their_bits(ssm, dtype, dk, dv):
    g = torch.zeros(1, 2, 1, device="cuda")
    o, _ = ssm.decay_attn_fwd(_rows(dk, dtype, ONE, ONE), _rows(dk, dtype, *CANCEL), _ones(dv, dtype), g, 1.0)
    assert (o[0, 1] == TINY).all()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("dk,dv", [(32, 16), (64, 72), (128, 128), (256, 40)])
def test_the_state_keeps_its_bits(ssm, dtype, dk, dv):
    state = torch.zeros(1, 1, dk, dv, device="cuda")
    state[0, 0, 0], state[0, 0, 1] = 1 + 2.0 ** -8 + TINY, -(1 + 2.0 ** -8)
    q, k, v = _rows(dk, dtype, ONE), _rows(dk, dtype, ()), _ones(dv, dtype, 1)
    o, final = ssm.decay_attn_fwd(q, k, v, torch.zeros(1, 1, 1, device="cuda"), 1.0, state, return_final_state=True)
    assert (o == TINY).all()
    assert torch.equal(final, state)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("want_dlog_decay", [True, False])
@pytest.mark.parametrize("dk,dv", [(32, 32), (128, 128)])
def test_gradients_keep_their_bits(ssm, dtype, want_dlog_decay, dk, dv):
    g = torch.zeros(1, 2, 1, device="cuda")

    def grads(q, k, v, do, state0=None, dfinal=None):
        return ssm.decay_attn_bwd(q, k, v, g, do, 1.0, state0, dfinal, want_dlog_decay, False)

    # dq_1 = sum_s (do_1 . v_s) k_s, dk_0 = sum_t (do_t . v_0) q_t, dv_0 = sum_t (q_t . k_0) do_t
    r = grads(_ones(dk, dtype), _ones(dk, dtype), _rows(dv, dtype, *CANCEL), _rows(dv, dtype, ONE, ONE))
    assert (r["dq"][0, 1] == TINY).all()
    r = grads(_ones(dk, dtype), _ones(dk, dtype), _rows(dv, dtype, ONE, ONE), _rows(dv, dtype, *CANCEL))
    assert (r["dk"][0, 0] == TINY).all()
    r = grads(_rows(dk, dtype, *CANCEL), _rows(dk, dtype, ONE, ONE), _ones(dv, dtype), _ones(dv, dtype))
    assert (r["dv"][0, 0] == TINY).all()
    # from the states: dq_0 = S do_0, dk_1 = R v_1, dv_1 = R^T k_1
    state = torch.zeros(1, 1, dk, dv, device="cuda")
    state[0, 0, :, 0], state[0, 0, :, 1] = 1 + 2.0 ** -8 + TINY, -(1 + 2.0 ** -8)
    none_k, none_v = torch.zeros_like(_ones(dk, dtype)), torch.zeros_like(_ones(dv, dtype))
    r = grads(none_k, none_k, none_v, _rows(dv, dtype, ONE, ()), state)
    assert (r["dq"][0, 0] == TINY).all()
    r = grads(none_k, none_k, _rows(dv, dtype, (), ONE), none_v, None, state)
    assert (r["dk"][0, 1] == TINY).all()
    state = state.new_zeros(1, 1, dk, dv)
    state[0, 0, 0], state[0, 0, 1] = 1 + 2.0 ** -8 + TINY, -(1 + 2.0 ** -8)
    r = grads(none_k, _rows(dk, dtype, (), ONE), none_v, none_v, None, state)
    assert (r["dv"][0, 1] == TINY).all()


def _one_signed(heads):
    """A value per head: mantissas whose lower bits are all set behind an 8-bit piece, and random ones."""
    x = 1 + torch.rand(heads, generator=torch.Generator().manual_seed(1))
    x[0], x[1], x[2] = 1 + 2.0 ** -7 - 2.0 ** -23, 2 - 2.0 ** -23, 1 + 2.0 ** -8 - 2.0 ** -23
    x[3], x[4], x[5] = 1 + 2.0 ** -8 + 2.0 ** -17, 1 + 2.0 ** -8 + 2.0 ** -16 - 2.0 ** -23, 1 + 2.0 ** -7 + 2.0 ** -15 - 2.0 ** -23
    return x


def _units(got, want):
    return float(((got.double().cpu() - want).abs() / want.abs()).max() * 2 ** 24)


def test_like_signed_products_fp32(ssm):
    """One step, one value per head: o = 32 x^3 (two products of full operands, the
    weight rounded between: 1 + 2 + 1 + 1 + 2 units, and 1 to spare), the last state
    x^2 (1 + 2, and 1 to spare)."""
    H = 256
    x = _one_signed(H)
    full = lambda d: x[None, None, :, None].expand(1, 1, H, d).contiguous().cuda()  # noqa: E731
    o, state = ssm.decay_attn_fwd(full(32), full(32), full(16), torch.zeros(1, 1, H, device="cuda"), 1.0, return_final_state=True)
    x = x.double()
    assert _units(o, 32 * x[None, None, :, None] ** 3) <= 8
    assert _units(state, x[None, :, None, None] ** 2) <= 4


def test_like_signed_state_products_fp32(ssm):
    """o = 32 x^2 from the state alone (1 + 2 units, the decay's 1 and 1 to spare)."""
    H = 256
    x = _one_signed(H)
    q = x[None, None, :, None].expand(1, 1, H, 32).contiguous().cuda()
    state = x[None, :, None, None].expand(1, H, 32, 16).contiguous().cuda()
    o, _ = ssm.decay_attn_fwd(q, torch.zeros_like(q), q[..., :16].contiguous(), torch.zeros(1, 1, H, device="cuda"), 1.0, state)
    assert _units(o, 32 * x.double()[None, None, :, None] ** 2) <= 5


@pytest.mark.parametrize("H,G", [(4, 4), (6, 2)])
def test_results_in_bf16_are_the_rounded_fp32_results(ssm, H, G):
    """A result whose fp32 error is e is rounded the other way where it lies within
    e of a boundary: of bf16's roundings a share of 2 e / 2^-8 at most.  With e up
    to 2^-20 of the values (16 effective roundings) below 2^-11; operands of 16
    bits give 2^-7 and more."""
    p = ref.attn_inputs(2, 512, H, G, 64, 64, seed=3, dtype=BF16)
    d = {n: None if t is None else t.cuda() for n, t in p.items()}
    o, _ = ssm.decay_attn_fwd(d["q"], d["k"], d["v"], d["g"], None, d["state0"])
    g = ssm.decay_attn_bwd(d["q"], d["k"], d["v"], d["g"], d["do"], None, d["state0"], d["dfinal"], want_dlog_decay=False)
    want = dict(o=ref.attn_fwd(p, 0.125)[0], **ref.attn_bwd(p, 0.125, p["dfinal"]))
    for n, t in dict(o=o, dq=g["dq"], dk=g["dk"], dv=g["dv"]).items():
        w = want[n].to(BF16)
        # values near zero are sums of much larger terms: only those of usual size
        usual = want[n].abs() > 0.25 * want[n].abs().mean()
        share = float((t.cpu() != w)[usual].double().mean())
        print(n, share, flush=True)
        assert share <= 2.0 ** -11, (n, share)


@pytest.mark.parametrize("value", [3.3961e38, 3.4e38])
def test_the_largest_values_reach_no_earlier_step(ssm, value):
    """fp32 values next to 2^128, whose first piece is the largest bf16 value or infinite."""
    p = ref.attn_inputs(1, 100, 2, 2, 32, 32, seed=6)
    want, _ = ref.attn_fwd(p, 32 ** -0.5)
    p["v"][:, 70] = value
    d = {n: t.cuda() for n, t in p.items()}
    o, _ = ssm.decay_attn_fwd(d["q"], d["k"], d["v"], d["g"], None, d["state0"])
    assert ref.error(o[:, :70], want[:, :70]) <= 1e-5

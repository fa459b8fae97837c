"""Decay attention (forward, gradients, single token) on the GPU against the
64-bit step-by-step reference.

Tolerances (of the largest difference beyond the result's own rounding to its
type, over the largest reference value, per output).  A result in fp32 is a sum
of at most a few hundred effective terms with fp32 products: sqrt(400) roundings
of 2^-24, and decays whose exponents, sums of up to 64 fp32 numbers kept to more
than fp32, add a few 2^-24 more: about 2e-6 of a typical value; 1e-5 is allowed.
Its operands are whole (bf16 values are split into pieces that hold every bit),
so states and the decays' gradient are held to fp32's bound for bf16 inputs too;
the decays' gradient is a running sum of differences and is allowed twice that.
A bf16 result is rounded once and its operands (the products inside a chunk and
the state) carry 2^-15 each, of terms whose absolute sum is up to 5 times the
largest result: 3e-4."""
from __future__ import annotations

import math

import pytest
import torch

from tests import block_reference as ref

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
TOL = {F32: 1e-5, BF16: 3e-4}


@pytest.fixture(scope="module")
def ssm():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import selective_state_space_10_amd as m
    m.load()
    return m


def _gpu(p):
    return {n: None if t is None else t.cuda() for n, t in p.items()}


def _check(got, want, kind, factor=1):
    err = ref.error(got, want)
    assert err <= factor * TOL[kind], err


def _compare(ssm, p, scale=None, dfinal=True, tag=""):
    print("decay attention", tag, {n: tuple(t.shape) for n, t in p.items() if t is not None}, flush=True)
    dt = p["q"].dtype
    sc = p["q"].shape[-1] ** -0.5 if scale is None else scale
    d = _gpu(p)
    o, final = ssm.decay_attn_fwd(d["q"], d["k"], d["v"], d["g"], scale, d["state0"], return_final_state=True)
    df = d["dfinal"] if dfinal else None
    g = ssm.decay_attn_bwd(d["q"], d["k"], d["v"], d["g"], d["do"], scale, d["state0"], df)
    torch.cuda.synchronize()
    ro, rs = ref.attn_fwd(p, sc)
    rg = ref.attn_bwd(p, sc, p["dfinal"] if dfinal else None)
    _check(o, ro, dt)
    _check(final, rs, F32)
    for n in ("dq", "dk", "dv"):
        _check(g[n], rg[n], dt)
    _check(g["dlog_decay"], rg["dlog_decay"], F32, 2)
    _check(g["dstate0"], rg["dstate0"], F32)
    return o, final, g


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("L", [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 200])
def test_lengths(ssm, dtype, L):
    _compare(ssm, ref.attn_inputs(2, L, 4, 2, 32, 40, seed=L, decay="mixed", dtype=dtype))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("dk,dv", [(8, 8), (16, 24), (24, 16), (32, 64), (40, 72), (64, 64), (72, 96), (128, 128),
                                   (128, 32), (136, 64), (256, 256), (8, 256), (256, 8)])
def test_head_sizes(ssm, dtype, dk, dv):
    _compare(ssm, ref.attn_inputs(1, 70, 2, 1, dk, dv, seed=dk + dv, decay="mixed", dtype=dtype))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("H,G", [(1, 1), (5, 5), (6, 1), (6, 2), (12, 3), (33, 11)])
def test_shared_heads(ssm, dtype, H, G):
    _compare(ssm, ref.attn_inputs(3, 37, H, G, 24, 16, seed=H, dtype=dtype))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("per_token", [True, False])
@pytest.mark.parametrize("decay", ["weak", "strong", "mixed", "none", "growing", "reset"])
def test_decays(ssm, dtype, per_token, decay):
    _compare(ssm, ref.attn_inputs(2, 150, 3, 3, 32, 32, seed=5, decay=decay, per_token=per_token, dtype=dtype))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("at", [[0], [149], [64], [63, 64, 65], list(range(150))])
def test_cleared_states(ssm, dtype, at):
    """-inf at the first step, the last, the edges of a chunk, and everywhere: then
    a step sees itself alone, and no gradient reaches an earlier one or a decay."""
    p = ref.attn_inputs(1, 150, 2, 2, 32, 48, seed=2, dtype=dtype)
    p["g"][:, at] = -math.inf
    _, _, g = _compare(ssm, p)
    assert not g["dlog_decay"][:, at].any()


def test_decays_far_below_zero_next_to_weak_ones(ssm):
    """Sums of very strong decays must not cost the weak ones their last bits."""
    p = ref.attn_inputs(1, 130, 2, 2, 32, 32, seed=3, decay="weak")
    p["g"][:, ::7] = -150.0
    p["g"][:, 3::11] = -1e4
    _compare(ssm, p)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("state0,dfinal", [(False, False), (True, False), (False, True)])
@pytest.mark.parametrize("L", [40, 700])
def test_optional_parts(ssm, dtype, state0, dfinal, L):
    _compare(ssm, ref.attn_inputs(1, L, 2, 2, 32, 32, seed=4, state0=state0, decay="mixed", dtype=dtype), dfinal=dfinal)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("B,L,H,G,dk,dv", [(1, 1025, 2, 1, 64, 64), (2, 2500, 1, 1, 128, 32), (1, 4096, 1, 1, 32, 128),
                                           (1, 1999, 3, 3, 24, 72)])
@pytest.mark.parametrize("decay", ["weak", "reset"])
def test_long(ssm, dtype, B, L, H, G, dk, dv, decay):
    """Lengths that are split over workgroups where there are few heads."""
    _compare(ssm, ref.attn_inputs(B, L, H, G, dk, dv, seed=L, decay=decay, dtype=dtype))


@pytest.mark.parametrize("scale", [0.0, 1.0, -2.5])
def test_scale(ssm, scale):
    _compare(ssm, ref.attn_inputs(1, 50, 2, 2, 16, 16), scale=scale)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_strided_views(ssm, dtype):
    """q, k, v as slices of one projection, heads before steps, broadcast inputs."""
    B, L, H, G, dk, dv = 2, 90, 4, 2, 24, 40
    p = ref.attn_inputs(B, L, H, G, dk, dv, seed=8, dtype=dtype)
    want = _compare(ssm, p)
    d = _gpu(p)
    qkv = torch.cat([d["q"].flatten(2), d["k"].flatten(2), d["v"].flatten(2), d["do"].flatten(2)], -1)
    q, k, v, do = qkv.split([G * dk, G * dk, H * dv, H * dv], -1)
    q, k, v, do = q.unflatten(-1, (G, dk)), k.unflatten(-1, (G, dk)), v.unflatten(-1, (H, dv)), do.unflatten(-1, (H, dv))
    assert not q.is_contiguous()
    for a in ((q, k, v, do), tuple(d[n].transpose(1, 2).contiguous().transpose(1, 2) for n in ("q", "k", "v", "do"))):
        o, final = ssm.decay_attn_fwd(a[0], a[1], a[2], d["g"], None, d["state0"], return_final_state=True)
        g = ssm.decay_attn_bwd(a[0], a[1], a[2], d["g"], a[3], None, d["state0"], d["dfinal"])
        assert torch.equal(o, want[0]) and torch.equal(final, want[1])
        assert all(torch.equal(g[n], want[2][n]) for n in g)
    one = d["q"][:, :1]
    o, _ = ssm.decay_attn_fwd(one.expand(B, L, G, dk), d["k"], d["v"], d["g"])
    o2, _ = ssm.decay_attn_fwd(one.repeat(1, L, 1, 1), d["k"], d["v"], d["g"])
    assert torch.equal(o, o2)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("bad", [math.nan, math.inf])
@pytest.mark.parametrize("name", ["q", "k", "v", "g"])
def test_nothing_reaches_an_earlier_step(ssm, dtype, bad, name):
    p = ref.attn_inputs(1, 150, 2, 2, 32, 32, seed=6, dtype=dtype)
    d = _gpu(p)
    o, _ = ssm.decay_attn_fwd(d["q"], d["k"], d["v"], d["g"], None, d["state0"])
    at = 70
    d[name][:, at] = bad
    o2, _ = ssm.decay_attn_fwd(d["q"], d["k"], d["v"], d["g"], None, d["state0"])
    # the chunk of the bad step sums in another order: equal to rounding, not to the bit
    _check(o2[:, :at], o[:, :at].double().cpu(), dtype)
    assert not torch.isfinite(o2[:, at]).all()
    if name == "q":
        _check(o2[:, at + 1:], o[:, at + 1:].double().cpu(), dtype)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_same_bits_again_and_on_another_stream(ssm, dtype):
    d = _gpu(ref.attn_inputs(2, 777, 4, 2, 64, 64, seed=9, decay="mixed", dtype=dtype))
    run = lambda: ssm.decay_attn_bwd(d["q"], d["k"], d["v"], d["g"], d["do"], None, d["state0"], d["dfinal"])  # noqa: E731
    a = run()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        b = run()
    torch.cuda.current_stream().wait_stream(s)
    assert all(torch.equal(a[n], b[n]) for n in a)


def test_gradients_are_differences(ssm):
    """Along random directions, fp32: the loss is summed in fp64 from fp32 outputs,
    so a step of 1e-2 leaves 1e-7 / 1e-2 of rounding and 1e-4 of third order."""
    p = ref.attn_inputs(2, 45, 4, 2, 16, 24, seed=10, decay="weak")
    d = _gpu(p)
    t = {n: d[n].clone().requires_grad_() for n in ("q", "k", "v", "g", "state0")}
    o, final = ssm.decay_attention(t["q"], t["k"], t["v"], t["g"], 0.3, t["state0"])
    torch.autograd.backward([o, final], [d["do"], d["dfinal"]])

    def loss(x):
        o, f = ssm.decay_attn_fwd(x["q"], x["k"], x["v"], x["g"], 0.3, x["state0"], return_final_state=True)
        return float((o.double() * d["do"]).sum() + (f.double() * d["dfinal"]).sum())

    gen = torch.Generator(device="cuda").manual_seed(3)
    for n in t:
        u = torch.randn(d[n].shape, generator=gen, device="cuda")
        step = 1e-2 if n != "g" else 1e-3
        up, down = dict(d), dict(d)
        up[n], down[n] = d[n] + step * u, d[n] - step * u
        diff = (loss(up) - loss(down)) / (2 * step)
        want = float((t[n].grad.double() * u).sum())
        assert diff == pytest.approx(want, rel=5e-3, abs=5e-3 * float(t[n].grad.norm())), n


def test_autograd_leaves_out_what_is_not_asked(ssm):
    d = _gpu(ref.attn_inputs(1, 33, 2, 2, 16, 16))
    v = d["v"].clone().requires_grad_()
    o, _ = ssm.decay_attention(d["q"], d["k"], v, d["g"])
    o.sum().backward()
    want = ssm.decay_attn_bwd(d["q"], d["k"], d["v"], d["g"], torch.ones_like(o), want_dlog_decay=False, want_dstate0=False)
    assert want["dlog_decay"] is None and want["dstate0"] is None
    assert torch.equal(v.grad, want["dv"])


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("B,H,G,dk,dv", [(1, 1, 1, 8, 8), (3, 4, 2, 24, 40), (2, 6, 1, 128, 128), (1, 16, 16, 64, 136),
                                         (5, 3, 3, 256, 256), (70, 5, 5, 40, 16), (1, 2, 2, 256, 8)])
@pytest.mark.parametrize("per_token", [True, False])
def test_single_tokens_follow_the_sequence(ssm, dtype, B, H, G, dk, dv, per_token):
    L = 5
    p = ref.attn_inputs(B, L, H, G, dk, dv, seed=B, decay="mixed", per_token=per_token, dtype=dtype)
    ro, rs = ref.attn_fwd(p, dk ** -0.5)
    d = _gpu(p)
    state = d["state0"].clone()
    for t in range(L):
        g = d["g"][:, t].contiguous() if per_token else d["g"]
        o = ssm.decay_attn_update(state, d["q"][:, t], d["k"][:, t], d["v"][:, t], g)  # strided views
        _check(o, ro[:, t], dtype)
    _check(state, rs, F32)


def test_single_token_clears(ssm):
    d = _gpu(ref.attn_inputs(2, 1, 3, 3, 32, 16, seed=1))
    g = torch.full((2, 3), -math.inf, device="cuda")
    state = d["state0"].clone()
    ssm.decay_attn_update(state, d["q"][:, 0], d["k"][:, 0], d["v"][:, 0], g)
    assert torch.equal(state, d["k"][:, 0, :, :, None] * d["v"][:, 0, :, None, :])


def test_prompt_in_pieces(ssm):
    """A prompt taken in two pieces and single tokens is the prompt taken at once."""
    p = ref.attn_inputs(2, 100, 2, 1, 40, 32, seed=11, decay="mixed")
    d = _gpu(p)
    part = lambda a, b: {n: d[n][:, a:b].contiguous() for n in ("q", "k", "v", "g")}  # noqa: E731
    ro, rs = ref.attn_fwd(p, 40 ** -0.5)
    x = part(0, 33)
    o1, s = ssm.decay_attn_fwd(x["q"], x["k"], x["v"], x["g"], None, d["state0"], return_final_state=True)
    x = part(33, 98)
    o2, s = ssm.decay_attn_fwd(x["q"], x["k"], x["v"], x["g"], None, s, return_final_state=True)
    o = [o1, o2]
    for t in (98, 99):
        o.append(ssm.decay_attn_update(s, d["q"][:, t], d["k"][:, t], d["v"][:, t], d["g"][:, t].contiguous())[:, None])
    _check(torch.cat(o, 1), ro, F32)
    _check(s, rs, F32)


def test_refusals(ssm):
    d = _gpu(ref.attn_inputs(1, 16, 4, 2, 16, 16))
    q, k, v, g = d["q"], d["k"], d["v"], d["g"]
    fwd = ssm.decay_attn_fwd
    with pytest.raises(ValueError):
        fwd(q[0], k, v, g)
    with pytest.raises(ValueError):
        fwd(q, k[:, :8], v, g)
    with pytest.raises(ValueError):
        fwd(q, k, v[:, :, :3], g[:, :, :3].contiguous())  # 3 heads on 2 key heads
    with pytest.raises(TypeError):
        fwd(q, k.bfloat16(), v, g)
    with pytest.raises(TypeError):
        fwd(q.half(), k.half(), v.half(), g)
    with pytest.raises(TypeError):
        fwd(q, k, v, g.double())
    with pytest.raises(ValueError):
        fwd(q, k, v, g[:, :8])
    with pytest.raises(ValueError):
        fwd(q, k, v, g.transpose(0, 1).contiguous().transpose(0, 1)[:, ::1].expand(1, 16, 4)[:, :, ::2])
    with pytest.raises(ValueError):
        fwd(q.cpu(), k, v, g)
    with pytest.raises(ValueError):
        fwd(q, k.cpu(), v, g)
    with pytest.raises(ValueError):
        fwd(q.transpose(-1, -2).contiguous().transpose(-1, -2), k, v, g)  # elements not adjacent
    odd = torch.empty(1, 16, 2, 17, device="cuda")[..., :16]
    with pytest.raises(ValueError):
        fwd(odd, k, v, g)  # rows not 16-byte aligned
    with pytest.raises(ValueError):
        fwd(q, k, v, g, state0=d["state0"][:, :, :8].contiguous())
    with pytest.raises((ssm.SSMError, ValueError)):
        fwd(q[..., :12].contiguous(), k[..., :12].contiguous(), v, g)  # dk not a multiple of 8
    with pytest.raises((ssm.SSMError, ValueError)):
        fwd(q[:, :0], k[:, :0], v[:, :0], g[:, :0].contiguous())
    with pytest.raises(ValueError):
        ssm.decay_attn_bwd(q, k, v, g, d["do"][:, :8])
    with pytest.raises(ValueError):
        ssm.decay_attn_update(d["state0"][:, :2], q[:, 0], k[:, 0], v[:, 0], g[:, 0].contiguous())
    with pytest.raises(TypeError):
        ssm.decay_attn_update(d["state0"].bfloat16(), q[:, 0], k[:, 0], v[:, 0], g[:, 0].contiguous())

"""The 64-bit references of the gated recurrence, the causal convolution and the norm
and rotation of heads, against closed forms and differences, and the formulas that
the kernels' backward passes use against them (CPU)."""
from __future__ import annotations

import pytest
import torch

from tests import mixer_reference as ref

F64 = torch.float64


def _differences(loss, p, names, gr, n=3, h=1e-6):
    """Central differences along random directions of all inputs together."""
    for seed in range(n):
        r, _ = ref.draw(100 + seed)
        way = {k: r(*p[k].shape).to(F64) for k in names}
        move = lambda e: {**p, **{k: p[k] + e * way[k] for k in names}}  # noqa: E731
        slope = (loss(move(h)) - loss(move(-h))) / (2 * h)
        want = sum((gr["d" + k] * way[k]).sum() for k in names)
        assert abs(slope - want) <= 1e-7 * (1 + abs(want)), (slope, want)


def _double(p):
    return {k: t.to(F64) if t is not None and t.is_floating_point() else t for k, t in p.items()}


@pytest.mark.parametrize("form", ["power", "logistic"])
@pytest.mark.parametrize("starts,lengths", [(False, False), (True, True)])
def test_recurrence_gradients_by_differences(form, starts, lengths):
    p = _double(ref.recurrence_inputs(3, 9, 8, form=form, starts=starts, lengths=lengths))
    gr = ref.recurrence(p)[3]
    names = [n for n in ref.REC_INPUTS if p[n] is not None]

    def loss(q):
        y, h, _, _ = ref.recurrence(q, grads=False)
        return (y * p["dy"]).sum() + (h * p["dfinal"]).sum()
    _differences(loss, p, names, gr)


def test_recurrence_closed_form():
    """Constant gates: h_t = a^(t+1) h_0 + s u (1 - a^(t+1)) / (1 - a)."""
    p = ref.recurrence_inputs(1, 6, 8, input_gate=False, z=False, dtype=F64)
    p["x"][:], p["decay_gate"][:] = 1.5, 0.3
    y = ref.recurrence(p, grads=False)[0]
    log_a = -8 * torch.log1p(torch.exp(p["decay"].double())) / (1 + torch.exp(torch.tensor(-0.3, dtype=F64)))
    a = torch.exp(log_a)
    for t in range(6):
        want = a ** (t + 1) * p["state0"].double() + torch.sqrt(1 - a * a) * 1.5 * (1 - a ** (t + 1)) / (1 - a)
        assert torch.allclose(y[:, t], want, rtol=1e-10)


@pytest.mark.parametrize("form", ["power", "logistic"])
def test_recurrence_backward_formulas(form):
    """The adjoint recurrence and the gates' gradients as the kernels form them."""
    p = _double(ref.recurrence_inputs(2, 11, 8, form=form, starts=True))
    y, _, before, gr = ref.recurrence(p)
    r = torch.sigmoid(p["decay_gate"])
    i = torch.sigmoid(p["input_gate"])
    u = i * p["x"]
    first = p["starts"][..., None]
    if form == "power":
        la = -8 * torch.nn.functional.softplus(p["decay"]) * r
        a, s = torch.exp(la), torch.sqrt(-torch.expm1(2 * la))
    else:
        a, s = r, 1 - r
    a, s = torch.where(first, 0.0, a), torch.where(first, 1.0, s)
    sig = torch.sigmoid(p["z"])
    w, carry = torch.empty_like(y), p["dfinal"]
    for t in range(10, -1, -1):
        w[:, t] = p["dy"][:, t] * p["z"][:, t] * sig[:, t] + carry
        carry = a[:, t] * w[:, t]
    ok = lambda got, n: torch.allclose(got, gr[n], rtol=1e-9, atol=1e-12)  # noqa: E731
    assert ok(carry, "dstate0") and ok(w * s * i, "dx") and ok(w * s * u * (1 - i), "dinput_gate")
    if form == "power":
        f = torch.where(first, 0.0, w * a * (la * before - u * a * la / s))
        assert ok(f * (1 - r), "ddecay_gate")
        assert ok(f.sum((0, 1)) * torch.sigmoid(p["decay"]) / torch.nn.functional.softplus(p["decay"]), "ddecay")
    else:
        assert ok(w * a * s * (before - u), "ddecay_gate")


@pytest.mark.parametrize("K", [1, 2, 3, 4])
@pytest.mark.parametrize("starts,lengths", [(False, False), (True, True)])
def test_conv_gradients_by_differences(K, starts, lengths):
    p = _double(ref.conv_inputs(3, 7, 8, K, starts=starts, lengths=lengths))
    gr = ref.conv(p)[2]
    names = [n for n in ref.CONV_INPUTS if p[n] is not None and p[n].numel()]

    def loss(q):
        y, f, _ = ref.conv(q, grads=False)
        return (y * p["dy"]).sum() + (f * p["dfinal"]).sum()
    _differences(loss, p, names, gr)


def test_conv_impulse_and_pieces():
    """An impulse returns the taps reversed; a sequence in two pieces is the sequence."""
    p = ref.conv_inputs(1, 9, 8, 4, bias=False, state0=False, dtype=F64)
    p["x"][:] = 0
    p["x"][:, 2] = 1
    y, _, _ = ref.conv(p, silu=False, grads=False)
    for k in range(4):
        assert torch.allclose(y[0, 2 + k], p["weight"][:, 3 - k].double())
    p = ref.conv_inputs(2, 9, 8, 3, dtype=F64)
    y, f, _ = ref.conv(p, grads=False)
    y1, f1, _ = ref.conv({**p, "x": p["x"][:, :4]}, grads=False)
    y2, f2, _ = ref.conv({**p, "x": p["x"][:, 4:], "state0": f1}, grads=False)
    assert torch.allclose(torch.cat([y1, y2], 1), y) and torch.equal(f, f2)


@pytest.mark.parametrize("norm,weights", [(True, "shared"), (True, "per head"), (True, None), (False, None)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_head_gradients_by_differences(norm, weights, interleaved):
    p = _double(ref.head_inputs(2, 3, 4, 2, 16, 8, weights=weights))
    gr = ref.heads(p, norm=norm, interleaved=interleaved)[1]
    names = [n for n in ref.HEAD_INPUTS if p[n] is not None]

    def loss(q):
        o, _ = ref.heads(q, norm=norm, interleaved=interleaved, grads=False)
        return sum((o[n] * p["d" + n + "_out"]).sum() for n in o)
    _differences(loss, p, names, gr)


def test_rotation_depends_on_distances_alone():
    """The products of rotated queries and keys do not change when all positions move on."""
    p = _double(ref.head_inputs(1, 5, 2, 2, 16, 16, weights=None))
    prod = lambda q: (lambda o: torch.einsum("blhd,bmhd->bhlm", o["q"], o["k"]))(ref.heads(q, grads=False)[0])  # noqa: E731
    assert torch.allclose(prod(p), prod({**p, "positions": p["positions"] + 1234}), atol=1e-9)

"""The gated recurrence on the GPU against the 64-bit reference.

Tolerances (largest difference beyond the result's own rounding to its type, over
the largest reference value, per output): a step's decay and input are off by up to 4
units of 2^-24 (an exponential of one, the roundings of its argument and of the
products), of either sign, and a state remembers at most L steps, so that their sum
goes like a random walk: twice its deviation, and 16 units for what follows, is
2^-24 (16 + 8 sqrt L).  A gradient holds a state and an adjoint state and the
roundings of its own few products: three times that; ddecay a sum of such over the steps, in
fp32 and of either sign: four times."""
from __future__ import annotations

import math

import pytest
import torch

from tests import mixer_reference as ref
from tests.test_mixer_plans import RECURRENCE

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
FORMS = ("power", "logistic")


@pytest.fixture(scope="module")
def ssm():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import selective_state_space_10_amd as m
    m.load()
    return m


def tol(L):
    return 2.0 ** -24 * (16 + 8 * math.sqrt(L))


def forward(ssm, g, sharpness=8.0):
    return ssm.gated_recurrence_fwd(g["x"], g["decay_gate"], g["input_gate"], g["decay"], g["z"], g["state0"], g["starts"], g["lengths"],
                                    sharpness, return_final_state=True, save_states=True)


def backward(ssm, g, states, sharpness=8.0):
    return ssm.gated_recurrence_bwd(g["dy"], g["x"], g["decay_gate"], g["input_gate"], g["decay"], g["z"], states, g["starts"], g["lengths"],
                                    sharpness, g["dfinal"])


def check(ssm, B, L, D, sharpness=8.0, **kw):
    print("recurrence", B, L, D, kw, flush=True)
    p = ref.recurrence_inputs(B, L, D, **kw)
    compare(ssm, p, ref.on_gpu(p), sharpness)


def compare(ssm, p, g, sharpness=8.0, t=None, want=None):
    L = p["x"].shape[1]
    y, final, states = forward(ssm, g, sharpness)
    d = backward(ssm, g, states, sharpness)
    ry, rf, rb, rg = want or ref.recurrence(p, sharpness)
    normal = lambda w: torch.where(w.abs() < 2.0 ** -126, 0.0, w)  # noqa: E731
    rg = {n: normal(w) for n, w in rg.items()}
    t = tol(L) if t is None else t
    assert y.dtype == p["x"].dtype and final.dtype == states.dtype == F32
    for n, got, want, most in [("y", y, ry, t), ("final", final, rf, t), ("states", states, rb[:, ::128], t)]:
        assert ref.error(got, want) <= most, (n, ref.error(got, want), most)
    for n, got in d.items():
        if n == "dstate0" and p["state0"] is None:
            continue
        if got is None:
            assert p[n[1:]] is None, n
            continue
        most = t * (4 if n == "ddecay" else 3)
        assert ref.error(got, rg[n]) <= most, (n, ref.error(got, rg[n]), most)
    if p["lengths"] is not None:
        off = torch.arange(L) >= p["lengths"][:, None]
        for n, got in [("y", y)] + [(n, t) for n, t in d.items() if t is not None and t.dim() == 3]:
            assert not got.cpu()[off].any(), n


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("L", [1, 2, 7, 8, 9, 15, 16, 17, 63, 64, 65, 127, 128, 129, 255, 257, 500])
def test_lengths_of_sequences(ssm, form, dtype, L):
    check(ssm, 2, L, 72, form=form, dtype=dtype, seed=L)


@pytest.mark.parametrize("D", [8, 56, 64, 72, 128, 136, 1000])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_widths(ssm, D, dtype):
    check(ssm, 3, 140, D, dtype=dtype, seed=D)


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("input_gate", [True, False])
@pytest.mark.parametrize("z", [True, False])
@pytest.mark.parametrize("state0", [True, False])
@pytest.mark.parametrize("starts", [True, False])
@pytest.mark.parametrize("lengths", [True, False])
def test_options(ssm, form, input_gate, z, state0, starts, lengths):
    check(ssm, 4, 150, 40, form=form, input_gate=input_gate, z=z, state0=state0, starts=starts, lengths=lengths, dtype=BF16 if z else F32)


@pytest.mark.parametrize("sizes", RECURRENCE, ids=str)
@pytest.mark.parametrize("marks", [False, True])
@pytest.mark.parametrize("form", FORMS)
def test_states_handed_on(ssm, sizes, marks, form):
    """Decays so close to 1 that a state is felt over many chunks, at sizes where states are published every 1, 2, 4, 8
    and 16 chunks, and more than once.

    The tolerance: a decay next to 1 is off by up to 2^-24 from its exponential (1 step of numbers in [1/2, 1)), and not
    of either sign alike: over 65536 decays between 1 - 1e-4 and 1 the instruction is off by -0.116 of that on average
    (as torch's fp32 exponential is), where rounding would be off by 0.00.  What a state keeps of a step k steps
    back is then off by up to k of these at once, and a state by up to L: L 2^-24 more than tol(L), which has the
    random part.  (tol(L) alone failed by 6% at 2 x 2100 x 520.)"""
    B, L, D, es = sizes
    print("recurrence", sizes, marks, form, flush=True)
    p = ref.recurrence_inputs(B, L, D, form=form, dtype=BF16 if es == 2 else F32, seed=L)
    u = torch.rand(D, generator=torch.Generator().manual_seed(D))
    if form == "power":
        p["decay"] = torch.log(torch.expm1(-torch.log(0.99 + 0.0099 * u) / 8.0))
    else:
        p["decay_gate"] += 3.0  # (a mean of 5)
    if marks:
        p["starts"] = torch.rand(B, L, generator=torch.Generator().manual_seed(L)) < 0.002
        p["starts"][:, 300] = True
        p["lengths"] = torch.tensor([L, L - 130, L, 0, L, 290, L, L - 1][:B], dtype=torch.int32)
    g = ref.on_gpu(p)
    with torch.device("cuda"):  # (the reference's many small steps are quicker there)
        y, final, before, grads = ref.recurrence(g)
    want = y.cpu(), final.cpu(), before.cpu(), {n: t.cpu() for n, t in grads.items()}
    compare(ssm, p, g, t=tol(L) + L * 2.0 ** -24, want=want)


def test_states_handed_on_over_the_longest_rows(ssm):
    """More than 2^31 elements of output, a state felt over many chunks: every row of a batch, whose states are published
    after each chunk, against a row by itself, published after every second, and against 64 bits.  Gates of 6 forget
    in 404 steps, of which each has the same error in its decay, of up to 2 units (the reciprocal's 1, the sum's
    and the exponential's parts in 1 + e^-6): 2 x 404 units of 2^-24 over tol(404).  Between the two calls, whose decays
    are the same, twice tol(404)."""
    B, L, D = 3, 87500, 8192
    gen = torch.Generator(device="cuda").manual_seed(0)
    row = torch.randn(1, L, D, generator=gen, device="cuda").to(BF16)
    gate = torch.full((1, 1, D), 6.0, dtype=BF16, device="cuda")
    y, f, _ = ssm.gated_recurrence_fwd(row.expand(B, L, D), gate.expand(B, L, D), return_final_state=True)
    y1, f1, _ = ssm.gated_recurrence_fwd(row, gate.expand(1, L, D), return_final_state=True)
    t = tol(404) + 808 * 2.0 ** -24
    some = slice(5, None, 127)
    a, h, d = torch.full((L, 1), 1 / (1 + math.exp(-6.0)), dtype=torch.float64, device="cuda"), row[0, :, some].double() / (1 + math.exp(6.0)), 1
    while d < L:  # each step's sum of the 2 d steps up to it
        h[d:] += a[d:] * h[:-d]
        a[d:] = a[d:] * a[:-d]
        d *= 2
    for b in range(B):
        assert ref.error(y[b][:, some], h.cpu()) <= t
        assert float((f[b] - f1[0]).abs().max() / f1.abs().max()) <= 2 * tol(404)
    assert ref.error(y1[0][:, some], h.cpu()) <= t


@pytest.mark.parametrize("L", [4095, 4097, 4500, 8200])
@pytest.mark.parametrize("marks", [False, True])
def test_long(ssm, L, marks):
    check(ssm, 1, L, 16, starts=marks, lengths=marks, dtype=F32, seed=L)


@pytest.mark.parametrize("B", [1, 5, 33])
def test_batches(ssm, B):
    check(ssm, B, 260, 24, starts=True, lengths=True)


@pytest.mark.parametrize("sharpness", [1e-3, 1.0, 64.0])
def test_sharpness(ssm, sharpness):
    check(ssm, 2, 70, 24, sharpness=sharpness)


@pytest.mark.parametrize("seed", range(24))
def test_random(ssm, seed):
    gen = torch.Generator().manual_seed(seed)
    pick = lambda lo, hi: int(torch.randint(lo, hi + 1, (1,), generator=gen))  # noqa: E731
    coin = lambda: bool(pick(0, 1))  # noqa: E731
    check(ssm, pick(1, 6), pick(1, 700), 8 * pick(1, 20), form=FORMS[pick(0, 1)], input_gate=coin(), z=coin(), state0=coin(), starts=coin(),
          lengths=coin(), dtype=(F32, BF16)[pick(0, 1)], seed=seed)


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("gate", [-1e4, -200.0, -90.0, -50.0, -20.0, 20.0, 50.0, 90.0, 200.0, 1e4])
def test_saturated_gates(ssm, form, gate):
    """Gates so far closed or open that their exponentials leave fp32: the results stay
    those of the reference.  (A sigmoid below 2^-126, where 1 + e^-g overflows its
    reciprocal's range, is taken as zero: its square root, the power form's input, is then off
    by up to 2^-62, and what it multiplies may be below 2^-126 and be zero, where outputs
    are compared as zero.)"""
    p = ref.recurrence_inputs(2, 130, 16, form=form)
    p["decay_gate"][:, ::3] = gate
    p["input_gate"][:, 1::4] = -gate
    p["z"][:, ::5] = gate / 100
    compare(ssm, p, ref.on_gpu(p))


@pytest.mark.parametrize("decay", [-110.0, -60.0, -20.0, 30.0, 80.0])
def test_extreme_decays(ssm, decay):
    """softplus(decay) from nothing at all to where every step forgets."""
    p = ref.recurrence_inputs(2, 130, 16)
    p["decay"][::2] = decay
    compare(ssm, p, ref.on_gpu(p))


def test_infinite_decays(ssm):
    """softplus(-inf) = 0: nothing is forgotten and nothing comes in; softplus(inf) = inf: every step forgets all."""
    p = ref.recurrence_inputs(2, 130, 16)
    p["decay"][::2] = -math.inf
    compare(ssm, p, ref.on_gpu(p))
    p["decay"][::2] = math.inf
    y, final, _, _ = ref.recurrence(p, grads=False)
    got = forward(ssm, ref.on_gpu(p))
    assert ref.error(got[0], y) <= tol(130) and ref.error(got[1], final) <= tol(130)
    state = p["state0"].cuda()
    ssm.gated_recurrence_update(state, *(p[n][:, 0].cuda() for n in ("x", "decay_gate", "input_gate")), p["decay"].cuda())
    assert ref.error(state[:, ::2], (torch.sigmoid(p["input_gate"]) * p["x"])[:, 0, ::2].double()) <= tol(1)
    p["decay"][3] = math.nan
    assert torch.isnan(forward(ssm, ref.on_gpu(p))[1][:, 3]).all()


def gates(D, dtype, form, seed=0):
    """One step whose factors do not cancel in any gradient: state and adjoints of one sign, inputs of the other."""
    p = ref.recurrence_inputs(3, 1, D, form=form, z=False, dtype=dtype, seed=seed)
    for n in ("x", "dy", "dfinal"):
        p[n] = 0.5 + p[n].abs()
    p["state0"] = -0.5 - p["state0"].abs()
    p["decay_gate"], p["input_gate"] = (p[n].clamp(-1, 1) for n in ("decay_gate", "input_gate"))
    return p


def every_value(ssm, p, name):
    """Each value of a gradient against its own size.  In units of 2^-24 of it: a gate's smaller side 21 (the exponent
    v log2(e) up to 29, rounded to half of 2^-19 and with log2(e) itself off by 1.3e-8, makes 16, exponential 2,
    reciprocal 2, product 1) and half of that again in s; the decay's rate 5, s 10, a 3, sigmoid(i) x 5, reciprocal 2,
    the adjoint 3, products 6: 65, taken as 80."""
    g = ref.on_gpu(p)
    d = backward(ssm, g, forward(ssm, g)[2])[name].cpu().double()
    want = ref.recurrence(p)[3]["d" + name[1:]]
    u = torch.finfo(p["x"].dtype).eps / 2
    off = float(((d - want).abs() / want.abs()).max())
    assert off <= u + 80 * 2.0 ** -24, off  # (no reference value is 0: off would be NaN or infinite)


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_gradient_of_far_decay_gates(ssm, form, dtype):
    """Open and closed gates keep the digits of their gradients, which are e^-|v| of the others'."""
    p = gates(136, dtype, form)
    p["decay_gate"][:] = torch.linspace(-20, 20, 136)
    every_value(ssm, p, "ddecay_gate")


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_gradient_of_far_input_gates(ssm, form, dtype):
    p = gates(136, dtype, form)
    p["input_gate"][:] = torch.linspace(-20, 20, 136)
    every_value(ssm, p, "dinput_gate")


def test_gradient_of_gates_of_the_smallest_rates(ssm):
    """softplus(decay) close to the end of fp32's range: 1 - sigmoid stays in the gate's gradient.  (The gate's
    exponent is below 16, and log a, about 2^-120, has four bits to spare above the range's end.)"""
    p = gates(136, F32, "power")
    p["decay"][:] = -86.0
    p["decay_gate"][:] = torch.linspace(-1, 8, 136)
    every_value(ssm, p, "ddecay_gate")


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_tokens_are_the_sequence(ssm, dtype):
    for form in FORMS:
        for input_gate, z in [(True, True), (False, False)]:
            p = ref.recurrence_inputs(5, 40, 104, form=form, input_gate=input_gate, z=z, dtype=dtype)
            g = ref.on_gpu(p)
            ry, rf, _, _ = ref.recurrence(p, grads=False)
            state = g["state0"].clone()
            part = lambda n, t: None if g[n] is None else g[n][:, t]  # noqa: E731
            for t in range(40):
                version = state._version
                y = ssm.gated_recurrence_update(state, *(part(n, t) for n in ("x", "decay_gate", "input_gate")), g["decay"], part("z", t))
                assert state._version > version
                assert ref.error(y, ry[:, t]) <= tol(40)
            assert ref.error(state, rf) <= tol(40)


@pytest.mark.parametrize("B,D", [(1, 8), (3, 2056), (300, 264)])
def test_single_tokens(ssm, B, D):
    for form in FORMS:
        p = ref.recurrence_inputs(B, 1, D, form=form, dtype=BF16)
        g = ref.on_gpu(p)
        ry, rf, _, _ = ref.recurrence(p, grads=False)
        state = g["state0"].clone()
        y = ssm.gated_recurrence_update(state, g["x"][:, 0], g["decay_gate"][:, 0], g["input_gate"][:, 0], g["decay"], g["z"][:, 0])
        assert ref.error(y, ry[:, 0]) <= tol(1) and ref.error(state, rf) <= tol(1)


def test_pieces_are_the_sequence(ssm):
    """The state of one call continues in the next."""
    p = ref.recurrence_inputs(2, 300, 24)
    g = ref.on_gpu(p)
    y, final, _ = forward(ssm, g)
    at, state, ys = 0, g["state0"], []
    for n in (1, 127, 128, 44):
        cut = {k: v[:, at:at + n] if v is not None and v.dim() == 3 else v for k, v in g.items()}
        o, state, _ = forward(ssm, {**cut, "state0": state})
        ys.append(o)
        at += n
    assert ref.error(torch.cat(ys, 1), y.cpu()) <= 2 * tol(300) and ref.error(state, final.cpu()) <= 2 * tol(300)


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("form", FORMS)
def test_nothing_crosses_a_start(ssm, form, bad):
    """Infinities and NaN of one document, of a state that a start drops and behind a
    row's length reach no other document, forward and backward."""
    p = ref.recurrence_inputs(3, 300, 16, form=form, state0=True)
    p["starts"] = torch.zeros(3, 300, dtype=torch.bool)
    p["starts"][:, [0, 50, 129, 200]] = True
    p["lengths"] = torch.tensor([300, 250, 0], dtype=torch.int32)
    clean = {k: None if v is None else v.clone() for k, v in p.items()}
    p["state0"][:2] = bad
    where = {"x": 60, "decay_gate": 140, "input_gate": 61, "z": 150, "dy": 199}
    for n, t in where.items():
        p[n][0, t, 3] = bad
        p[n][1, 250:] = bad
    g = ref.on_gpu(p)
    y, final, states = forward(ssm, g)
    d = backward(ssm, g, states)
    ry, rf, _, rg = ref.recurrence(clean)
    spans = [(0, 50), (200, 300)]  # documents without a bad value
    t = tol(300)
    for name, got, want in [("y", y, ry)] + [(n, d[n], rg[n]) for n in ("dx", "ddecay_gate", "dinput_gate", "dz")]:
        got = got.cpu()
        for a, b in spans:
            assert ref.error(got[:, a:b], want[:, a:b]) <= 3 * t, (name, a)
        assert ref.error(got[1:], want[1:]) <= 3 * t, name
        assert not got[1, 250:].any() and not got[2].any(), name
    assert ref.error(final[:2], rf[:2]) <= t and torch.equal(final[2].cpu(), p["state0"][2])
    assert not d["dstate0"][:2].any()


@pytest.mark.parametrize("form", FORMS)
def test_packed_documents_are_the_documents_alone(ssm, form):
    """A document in a packed row and in a call of its own, its first step marked in both: outputs, last state and
    gradients.  A first step without a mark has the gate's s instead of 1."""
    p = ref.recurrence_inputs(1, 300, 24, form=form, z=False, state0=False)
    p["starts"] = torch.zeros(1, 300, dtype=torch.bool)
    ends = (0, 1, 140, 300)
    p["starts"][0, list(ends[:-1])] = True
    p["dfinal"].zero_()
    g = ref.on_gpu(p)
    y, final, states = forward(ssm, g)
    d = backward(ssm, g, states)
    for a, b in zip(ends, ends[1:]):
        one = {n: t[:, a:b] if t is not None and t.dim() == 3 else t for n, t in g.items()}
        one["starts"] = g["starts"][:, a:b].contiguous()
        y1, final1, states1 = forward(ssm, one)
        d1 = backward(ssm, one, states1)
        assert ref.error(y1, y[:, a:b].cpu()) <= 2 * tol(b - a)
        assert all(ref.error(d1[n], d[n][:, a:b].cpu()) <= 6 * tol(b - a) for n in ("dx", "dinput_gate", "ddecay_gate"))
    assert ref.error(final1, final.cpu()) <= 2 * tol(b - a)
    one["starts"] = None
    gate = p["decay_gate"][:, a].double()
    if form == "power":
        rate = 8 * torch.nn.functional.softplus(p["decay"].double()) * torch.sigmoid(gate)
        s = torch.sqrt(-torch.expm1(-2 * rate))
    else:
        s = torch.sigmoid(-gate)
    assert ref.error(forward(ssm, one)[0][:, 0], s * y[:, a].cpu()) <= 2 * tol(1)


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("form", FORMS)
def test_the_decay_gate_of_a_start_is_not_used(ssm, form, bad):
    p = ref.recurrence_inputs(2, 150, 72, form=form)
    p["starts"] = torch.zeros(2, 150, dtype=torch.bool)
    p["starts"][:, [0, 17, 128, 149]] = True
    clean = {k: None if v is None else v.clone() for k, v in p.items()}
    p["decay_gate"][p["starts"]] = bad
    compare(ssm, clean, ref.on_gpu(p))


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("L", [20, 150])
@pytest.mark.parametrize("form", FORMS)
def test_an_unused_row_is_not_in_ddecay(ssm, form, L, bad):
    """A row of length 0 whose state, and what comes back for it, are not finite: they pass through, and the
    gradients of all other rows and of the parameter that the rows share stay those without it."""
    p = ref.recurrence_inputs(3, L, 72, form=form)
    p["lengths"] = torch.tensor([L, 0, 7], dtype=torch.int32)
    clean = {k: None if v is None else v.clone() for k, v in p.items()}
    p["state0"][1] = p["dfinal"][1] = bad
    g = ref.on_gpu(p)
    y, final, states = forward(ssm, g)
    d = backward(ssm, g, states)
    ry, _, _, rg = ref.recurrence(clean)
    assert ref.error(y, ry) <= tol(L) and torch.equal(final[1].cpu().isnan(), p["state0"][1].isnan())
    for n in ("dx", "ddecay_gate", "dinput_gate", "dz", "ddecay"):
        if d[n] is not None:
            assert ref.error(d[n], rg[n]) <= 4 * tol(L), n
    keep = [0, 2]
    assert ref.error(d["dstate0"][keep], rg["dstate0"][keep]) <= 3 * tol(L)


def test_a_bad_value_reaches_later_steps_of_its_document_alone(ssm):
    p = ref.recurrence_inputs(1, 400, 16)
    p["x"][0, 130, 5] = math.nan
    y, final, states = forward(ssm, ref.on_gpu(p))
    bad = torch.isnan(y.cpu())
    assert bad[0, 130:, 5].all() and bad.sum() == 270 and torch.isnan(final.cpu()).sum() == 1
    assert torch.isnan(states.cpu()).sum() == 2


def test_strides(ssm):
    """Slices of a fused projection, a batch that shares its rows, time before batch."""
    p = ref.recurrence_inputs(3, 140, 24, dtype=BF16)
    g = ref.on_gpu(p)
    want_y, want_f, states = forward(ssm, g)
    want = backward(ssm, g, states)
    fused = torch.cat([g[n] for n in ("x", "decay_gate", "input_gate", "z", "dy")], -1)
    cut = dict(zip(("x", "decay_gate", "input_gate", "z", "dy"), fused.split(24, -1)))
    swapped = {n: g[n].transpose(0, 1).contiguous().transpose(0, 1) for n in cut}
    for views in (cut, swapped):
        v = {**g, **views}
        assert not v["x"].is_contiguous()
        y, f, s = forward(ssm, v)
        got = backward(ssm, v, s)
        assert torch.equal(y, want_y) and torch.equal(f, want_f) and torch.equal(s, states)
        assert all(torch.equal(got[n], want[n]) for n in want)
    one = {**g, "x": g["x"][:1].expand(3, -1, -1), "decay_gate": g["decay_gate"][:, :1].expand(-1, 140, -1)}
    y, _, s = forward(ssm, one)
    full = {n: t if t is None else t.contiguous() for n, t in one.items()}
    y2, _, s2 = forward(ssm, full)
    assert torch.equal(y, y2) and torch.equal(backward(ssm, one, s)["dx"], backward(ssm, full, s2)["dx"])


def test_offsets_beyond_32_bits(ssm):
    """Rows more than 2^31 elements apart."""
    B, L, D = 2, 130, 16
    p = ref.recurrence_inputs(B, L, D, dtype=BF16)
    g = ref.on_gpu(p)
    gap = 2 ** 31 + 64
    big = torch.empty(gap + L * D, dtype=BF16, device="cuda")
    for n in ("x", "decay_gate", "dy"):
        v = {**g, n: big.as_strided((B, L, D), (gap, D, 1))}
        v[n].copy_(g[n])
        y, f, s = forward(ssm, g)
        y2, f2, s2 = forward(ssm, v)
        assert torch.equal(y, y2) and torch.equal(f, f2)
        a, b = backward(ssm, g, s), backward(ssm, v, s2)
        assert all(torch.equal(a[k], b[k]) for k in a)


def test_outputs_beyond_32_bits(ssm):
    """More than 2^31 elements of output: the last rows are those of a call on them alone."""
    B, L, D = 3, 87500, 8192
    gen = torch.Generator(device="cuda").manual_seed(0)
    row = torch.randn(1, L, D, generator=gen, device="cuda").to(BF16)
    x = row.expand(B, L, D)
    y, f, _ = ssm.gated_recurrence_fwd(x, x, return_final_state=True)
    y1, f1, _ = ssm.gated_recurrence_fwd(row, row, return_final_state=True)
    assert torch.equal(y[2], y1[0]) and torch.equal(f[2], f1[0])


def test_same_bits_again(ssm):
    p = ref.recurrence_inputs(2, 5000, 136, dtype=BF16, starts=True)
    g = ref.on_gpu(p)
    y, f, s = forward(ssm, g)
    d = backward(ssm, g, s)
    for _ in range(5):
        y2, f2, s2 = forward(ssm, g)
        d2 = backward(ssm, g, s2)
        assert torch.equal(y, y2) and torch.equal(f, f2) and torch.equal(s, s2)
        assert all(torch.equal(d[n], d2[n]) for n in d)


def test_streams(ssm):
    """Calls on several streams at once, each on its own tensors."""
    ps = [ref.recurrence_inputs(2, 1500, 72, dtype=BF16, seed=i) for i in range(4)]
    gs = [ref.on_gpu(p) for p in ps]
    want = [forward(ssm, g) for g in gs]
    wantd = [backward(ssm, g, w[2]) for g, w in zip(gs, want)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in gs]
    for _ in range(3):
        got = []
        for st, g in zip(streams, gs):
            with torch.cuda.stream(st):
                f = forward(ssm, g)
                got.append((f, backward(ssm, g, f[2])))
        torch.cuda.synchronize()
        for (f, d), w, wd in zip(got, want, wantd):
            assert all(torch.equal(a, b) for a, b in zip(f, w)) and all(torch.equal(d[n], wd[n]) for n in wd)


@pytest.mark.parametrize("L", [100, 5000])
def test_in_a_graph(ssm, L):
    """Captured, and replayed on other inputs, with eager calls between."""
    p = ref.recurrence_inputs(2, L, 40, dtype=BF16)
    g = ref.on_gpu(p)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        s = forward(ssm, g)[2]
        backward(ssm, g, s)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, f, s = forward(ssm, g)
        d = backward(ssm, g, s)
    for i in range(4):
        other = ref.on_gpu(ref.recurrence_inputs(2, L, 40, dtype=BF16, seed=10 + i))
        for n in g:
            if g[n] is not None:
                g[n].copy_(other[n])
        graph.replay()
        torch.cuda.synchronize()
        y2, f2, s2 = forward(ssm, other)
        d2 = backward(ssm, other, s2)
        torch.cuda.synchronize()
        assert torch.equal(y, y2) and torch.equal(f, f2) and torch.equal(s, s2)
        assert all(torch.equal(d[n], d2[n]) for n in d)


def test_autograd(ssm):
    p = ref.recurrence_inputs(2, 150, 24, starts=True, lengths=True)
    g = ref.on_gpu(p)
    leaves = {n: g[n].clone().requires_grad_() for n in ref.REC_INPUTS}
    y, final = ssm.gated_recurrence(**leaves, starts=g["starts"], lengths=g["lengths"])
    ((y * g["dy"]).sum() + (final * g["dfinal"]).sum()).backward()
    _, _, _, rg = ref.recurrence(p)
    for n, t in leaves.items():
        assert ref.error(t.grad, rg["d" + n]) <= 4 * tol(150), n
    # only one output used, inputs without gradients, an input used twice
    x = g["x"].clone().requires_grad_()
    _, final = ssm.gated_recurrence(x, x, None, None, None)
    final.sum().backward()
    q = {**p, "decay_gate": p["x"], "input_gate": None, "decay": None, "z": None, "state0": None, "starts": None, "lengths": None,
         "dy": torch.zeros_like(p["dy"]), "dfinal": torch.ones_like(p["dfinal"])}
    rg = ref.recurrence(q)[3]
    assert ref.error(x.grad, rg["dx"] + rg["ddecay_gate"]) <= 4 * tol(150)
    with torch.no_grad():
        y2, _ = ssm.gated_recurrence(g["x"], g["decay_gate"])
    assert not y2.requires_grad


def test_refusals(ssm):
    g = ref.on_gpu(ref.recurrence_inputs(2, 10, 16))
    f = ssm.gated_recurrence_fwd
    x, gate = g["x"], g["decay_gate"]
    for args, kw, what in [
            ((x.cpu(), gate), {}, ValueError), ((x[0], gate), {}, ValueError), ((x.half(), gate), {}, TypeError), ((x, gate.bfloat16()), {}, TypeError),
            ((x, gate[:, :5]), {}, ValueError), ((x, gate, g["input_gate"][..., :8]), {}, ValueError), ((x, gate, None, g["decay"][:8]), {}, ValueError),
            ((x, gate, None, g["decay"].double()), {}, TypeError), ((x, gate), dict(state0=g["state0"][:1]), ValueError),
            ((x, gate), dict(starts=torch.zeros(2, 10, device="cuda")), TypeError), ((x, gate), dict(lengths=torch.zeros(2, dtype=torch.int64, device="cuda")), TypeError),
            ((x, gate), dict(lengths=torch.zeros(3, dtype=torch.int32, device="cuda")), ValueError), ((x.transpose(1, 2), gate), {}, ValueError),
            ((x[..., :12], gate[..., :12]), {}, ValueError), ((x[:, :0], gate[:, :0]), {}, ValueError), ((None, gate), {}, TypeError),
            ((x, gate, None, g["decay"]), dict(sharpness=0.0), ssm.SSMError), ((x, gate, None, g["decay"]), dict(sharpness=math.nan), ssm.SSMError)]:
        with pytest.raises(what):
            f(*args, **kw)
    _, _, states = forward(ssm, g)
    with pytest.raises(ValueError):
        ssm.gated_recurrence_bwd(g["dy"], x, gate, None, None, None, states[:, :, :8])
    with pytest.raises(ValueError):
        ssm.gated_recurrence_bwd(g["dy"], x, gate, None, None, None, None)
    with pytest.raises(TypeError):
        ssm.gated_recurrence_update(g["state0"].bfloat16(), x[:, 0], gate[:, 0])
    with pytest.raises(ValueError):
        ssm.gated_recurrence_update(g["state0"].t().contiguous().t(), x[:, 0], gate[:, 0])

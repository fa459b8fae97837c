"""The causal convolution on the GPU against the 64-bit reference.

Tolerances (largest difference beyond the result's own rounding to its type, over the
largest reference value, per output): up to five roundings of 2^-24 of a sum of taps
and about ten of the gate's exponential and products: 2e-6; 1e-5 for the gradients of
weights and bias, sums over up to thousands of steps in parts."""
from __future__ import annotations

import math

import pytest
import torch

from tests import mixer_reference as ref
from tests.test_mixer_plans import CONV

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
TOL, SUMS = 2e-6, 1e-5


@pytest.fixture(scope="module")
def ssm():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import selective_state_space_10_amd as m
    m.load()
    return m


def forward(ssm, g, silu=True):
    return ssm.causal_conv_fwd(g["x"], g["weight"], g["bias"], g["state0"], g["starts"], g["lengths"], silu, return_final_state=True)


def backward(ssm, g, silu=True):
    return ssm.causal_conv_bwd(g["dy"], g["x"], g["weight"], g["bias"], g["state0"], g["starts"], g["lengths"], silu, g["dfinal"])


def check(ssm, B, L, D, K, silu=True, **kw):
    print("conv", B, L, D, K, silu, kw, flush=True)
    p = ref.conv_inputs(B, L, D, K, **kw)
    compare(ssm, p, ref.on_gpu(p), silu)


def compare(ssm, p, g, silu):
    y, final = forward(ssm, g, silu)
    d = backward(ssm, g, silu)
    ry, rf, rg = ref.conv(p, silu)
    assert ref.error(y, ry) <= TOL, ref.error(y, ry)
    assert final.shape == rf.shape and torch.equal(final.cpu().double(), rf)
    for n, got in d.items():
        if got is None:
            assert p[n[1:]] is None, n
        elif got.numel():
            e = ref.error(got, rg[n])
            assert e <= (TOL if n in ("dx", "dstate0") else SUMS), (n, e)


@pytest.mark.parametrize("K", [1, 2, 3, 4])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("L", [1, 2, 3, 4, 5, 7, 8, 9, 31, 32, 33, 60, 61, 62, 63, 64, 65, 130])
def test_lengths_of_sequences(ssm, K, dtype, L):
    check(ssm, 2, L, 24, K, dtype=dtype, seed=L)


@pytest.mark.parametrize("D", [8, 16, 64, 120, 136, 264, 512, 520, 2056])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_widths(ssm, D, dtype):
    check(ssm, 2, 37, D, 4, dtype=dtype, starts=True, seed=D)


@pytest.mark.parametrize("K", [1, 2, 3, 4])
@pytest.mark.parametrize("silu", [True, False])
@pytest.mark.parametrize("bias", [True, False])
@pytest.mark.parametrize("state0", [True, False])
@pytest.mark.parametrize("starts", [True, False])
@pytest.mark.parametrize("lengths", [True, False])
def test_options(ssm, K, silu, bias, state0, starts, lengths):
    check(ssm, 4, 70, 16, K, silu, bias=bias, state0=state0, starts=starts, lengths=lengths, dtype=F32 if bias else BF16)


@pytest.mark.parametrize("L", [1, 2, 3, 6])
def test_dense_starts(ssm, L):
    """Starts next to each other, at the first step and at the last; rows as short as the taps."""
    for seed in range(6):
        p = ref.conv_inputs(8, L, 8, 4, lengths=True, seed=seed)
        p["starts"] = torch.rand(8, L, generator=torch.Generator().manual_seed(seed)) < 0.5
        compare(ssm, p, ref.on_gpu(p), True)


@pytest.mark.parametrize("B,L", [(1, 5000), (40, 300), (300, 20)])
def test_many_rows(ssm, B, L):
    check(ssm, B, L, 16, 4, starts=True, lengths=True)


@pytest.mark.parametrize("sizes", CONV, ids=str)
@pytest.mark.parametrize("marks", [False, True])
def test_training_sizes(ssm, sizes, marks):
    """Chunks of more than 64 steps, and several of them to a wave, with and without starts and lengths."""
    B, L, D, K, es = sizes
    print("conv", sizes, marks, flush=True)
    gen = torch.Generator("cuda").manual_seed(L + D)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    dtype = BF16 if es == 2 else F32
    g = dict(x=r(B, L, D).to(dtype), weight=r(D, K) * K ** -0.5, bias=r(D), state0=r(B, K - 1, D).to(dtype), dy=r(B, L, D).to(dtype),
             dfinal=r(B, K - 1, D).to(dtype), starts=None, lengths=None)
    if marks:
        g["starts"] = torch.rand(B, L, generator=gen, device="cuda") < 0.02
        g["lengths"] = torch.tensor([L, L - 3, 0, 70, 1, L // 2, L, L - 40][:B], dtype=torch.int32, device="cuda")
    y, final = forward(ssm, g)
    d = backward(ssm, g)
    ry, rf, rg = ref.conv_at_once(g)
    assert ref.error(y, ry.cpu()) <= TOL and torch.equal(final.double(), rf)
    for n, got in d.items():
        assert ref.error(got, rg[n].cpu()) <= (TOL if n in ("dx", "dstate0") else SUMS), n


@pytest.mark.parametrize("seed", range(16))
def test_random(ssm, seed):
    gen = torch.Generator().manual_seed(seed)
    pick = lambda lo, hi: int(torch.randint(lo, hi + 1, (1,), generator=gen))  # noqa: E731
    coin = lambda: bool(pick(0, 1))  # noqa: E731
    check(ssm, pick(1, 6), pick(1, 300), 8 * pick(1, 30), pick(1, 4), coin(), bias=coin(), state0=coin(), starts=coin(), lengths=coin(),
          dtype=(F32, BF16)[pick(0, 1)], seed=seed)


@pytest.mark.parametrize("K", [1, 2, 3, 4])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_tokens_are_the_sequence(ssm, K, dtype):
    p = ref.conv_inputs(5, 12, 104, K, dtype=dtype)
    g = ref.on_gpu(p)
    ry, rf, _ = ref.conv(p, grads=False)
    state = g["state0"].clone()
    for t in range(12):
        version = state._version
        y = ssm.causal_conv_update(state, g["x"][:, t], g["weight"], g["bias"])
        assert state._version > version
        assert ref.error(y, ry[:, t]) <= TOL
    assert torch.equal(state.cpu().double(), rf)


def test_pieces_are_the_sequence(ssm):
    p = ref.conv_inputs(2, 100, 24, 4)
    g = ref.on_gpu(p)
    y, final = forward(ssm, g)
    at, state, ys = 0, g["state0"], []
    for n in (1, 2, 33, 64):
        o, state = forward(ssm, {**g, "x": g["x"][:, at:at + n], "state0": state})
        ys.append(o)
        at += n
    assert torch.equal(torch.cat(ys, 1), y) and torch.equal(state, final)


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_nothing_crosses_a_start(ssm, bad):
    """Bad values of one document, of a dropped state and behind a row's length reach nothing else."""
    p = ref.conv_inputs(3, 150, 16, 4)
    p["starts"] = torch.zeros(3, 150, dtype=torch.bool)
    p["starts"][:, [0, 50, 52, 100]] = True
    p["lengths"] = torch.tensor([150, 120, 0], dtype=torch.int32)
    clean = {k: None if v is None else v.clone() for k, v in p.items()}
    p["state0"][:2] = bad
    p["x"][1, 120:] = bad
    p["dy"][1, 120:] = bad
    p["dy"][2] = bad
    ry, rf, rg = ref.conv(clean)
    g = ref.on_gpu(p)
    y, final = forward(ssm, g)
    d = backward(ssm, g)
    assert ref.error(y, ry) <= TOL and torch.equal(final[:2].cpu().double(), rf[:2]) and torch.equal(final[2].cpu(), p["state0"][2])
    assert ref.error(d["dx"], rg["dx"]) <= TOL and ref.error(d["dweight"], rg["dweight"]) <= SUMS and ref.error(d["dbias"], rg["dbias"]) <= SUMS
    assert not d["dstate0"][:2].any() and torch.equal(d["dstate0"][2].cpu(), p["dfinal"][2])
    p["x"][0, 49] = bad  # the last step of a document
    p["dy"][0, 99] = bad
    g = ref.on_gpu(p)
    y, d = forward(ssm, g)[0].cpu(), backward(ssm, g)["dx"].cpu()
    keep = torch.arange(150) != 49
    assert ref.error(y[0][keep], ry[0][keep]) <= TOL
    keep = (torch.arange(150) < 46) | ((torch.arange(150) >= 50) & (torch.arange(150) < 96)) | (torch.arange(150) >= 100)
    assert ref.error(d[0][keep], rg["dx"][0][keep]) <= TOL


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("K", [2, 4])
@pytest.mark.parametrize("L", [2, 70])
def test_an_unused_row_is_not_in_the_weights_gradients(ssm, K, L, bad):
    """A row of length 0 whose state, and what comes back for it, are not finite: they pass through, and the
    gradients of all other rows and of the weights stay those without it."""
    p = ref.conv_inputs(3, L, 24, K)
    p["lengths"] = torch.tensor([L, 0, 1], dtype=torch.int32)
    clean = {k: None if v is None else v.clone() for k, v in p.items()}
    p["state0"][1] = p["dfinal"][1] = bad
    g = ref.on_gpu(p)
    y, final = forward(ssm, g)
    d = backward(ssm, g)
    ry, rf, rg = ref.conv(clean)
    keep = [0, 2]
    assert ref.error(y, ry) <= TOL and torch.equal(final[keep].cpu().double(), rf[keep]) and torch.equal(final[1].cpu().isnan(), p["state0"][1].isnan())
    for n in ("dx", "dweight", "dbias"):
        assert ref.error(d[n], rg[n]) <= (TOL if n == "dx" else SUMS), n
    assert ref.error(d["dstate0"][keep], rg["dstate0"][keep]) <= TOL


def test_strides(ssm):
    p = ref.conv_inputs(3, 70, 24, 4, dtype=BF16)
    g = ref.on_gpu(p)
    want, wantd = forward(ssm, g), backward(ssm, g)
    fused = torch.cat([g["dy"], g["x"]], -1)
    swapped = {n: g[n].transpose(0, 1).contiguous().transpose(0, 1) for n in ("x", "dy")}
    for v in ({**g, "dy": fused[..., :24], "x": fused[..., 24:]}, {**g, **swapped}):
        got, gotd = forward(ssm, v), backward(ssm, v)
        assert all(torch.equal(a, b) for a, b in zip(got, want)) and all(torch.equal(gotd[n], wantd[n]) for n in wantd)
    one = {**g, "x": g["x"][:1].expand(3, -1, -1)}
    full = {**g, "x": one["x"].contiguous()}
    assert torch.equal(forward(ssm, one)[0], forward(ssm, full)[0]) and torch.equal(backward(ssm, one)["dx"], backward(ssm, full)["dx"])


def test_offsets_beyond_32_bits(ssm):
    p = ref.conv_inputs(2, 40, 16, 4, dtype=BF16)
    g = ref.on_gpu(p)
    gap = 2 ** 31 + 64
    big = torch.empty(gap + 40 * 16, dtype=BF16, device="cuda").as_strided((2, 40, 16), (gap, 16, 1))
    for n in ("x", "dy"):
        big.copy_(g[n])
        v = {**g, n: big}
        a, b = backward(ssm, g), backward(ssm, v)
        assert torch.equal(forward(ssm, g)[0], forward(ssm, v)[0]) and all(torch.equal(a[k], b[k]) for k in a)


def test_outputs_beyond_32_bits(ssm):
    B, L, D = 3, 87500, 8192
    row = torch.randn(1, L, D, generator=torch.Generator(device="cuda").manual_seed(0), device="cuda").to(BF16)
    w = torch.randn(D, 4, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda")
    x = row.expand(B, L, D)
    y, _ = ssm.causal_conv_fwd(x, w)
    assert torch.equal(y[2], ssm.causal_conv_fwd(row, w)[0][0])
    d = ssm.causal_conv_bwd(x, x, w)
    assert torch.equal(d["dx"][2], ssm.causal_conv_bwd(row, row, w)["dx"][0])


def test_same_bits_streams_and_graph(ssm):
    ps = [ref.conv_inputs(2, 900, 136, 4, dtype=BF16, starts=True, seed=i) for i in range(3)]
    gs = [ref.on_gpu(p) for p in ps]
    want = [(forward(ssm, g), backward(ssm, g)) for g in gs]
    torch.cuda.synchronize()
    same = lambda a, b: all(torch.equal(s, t) for s, t in zip(a[0], b[0])) and all(torch.equal(a[1][n], b[1][n]) for n in b[1])  # noqa: E731
    streams = [torch.cuda.Stream() for _ in gs]
    for _ in range(3):
        got = []
        for st, g in zip(streams, gs):
            with torch.cuda.stream(st):
                got.append((forward(ssm, g), backward(ssm, g)))
        torch.cuda.synchronize()
        assert all(same(a, b) for a, b in zip(got, want))
    static = {n: None if t is None else t.clone() for n, t in gs[0].items()}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = (forward(ssm, static), backward(ssm, static))
    for g, w in list(zip(gs, want)) + [(gs[0], want[0])]:
        for n in g:
            if g[n] is not None:
                static[n].copy_(g[n])
        graph.replay()
        torch.cuda.synchronize()
        assert same(out, w)
        forward(ssm, g)
        torch.cuda.synchronize()


def test_autograd(ssm):
    p = ref.conv_inputs(2, 70, 24, 4, starts=True, lengths=True)
    g = ref.on_gpu(p)
    leaves = {n: g[n].clone().requires_grad_() for n in ref.CONV_INPUTS}
    y, final = ssm.causal_conv(**leaves, starts=g["starts"], lengths=g["lengths"])
    ((y * g["dy"]).sum() + (final * g["dfinal"]).sum()).backward()
    rg = ref.conv(p)[2]
    for n, t in leaves.items():
        assert ref.error(t.grad, rg["d" + n]) <= SUMS, n
    x = g["x"].clone().requires_grad_()
    ssm.causal_conv(x, g["weight"])[1].sum().backward()  # the last inputs alone
    assert torch.equal(x.grad, torch.nn.functional.pad(torch.ones(2, 3, 24, device="cuda"), (0, 0, 67, 0)))
    w1 = g["weight"][:, :1].contiguous().requires_grad_()
    y, final = ssm.causal_conv(g["x"], w1)
    assert final.shape == (2, 0, 24)
    y.sum().backward()
    assert w1.grad.isfinite().all()


def test_refusals(ssm):
    g = ref.on_gpu(ref.conv_inputs(2, 10, 16, 4))
    f, x, w = ssm.causal_conv_fwd, g["x"], g["weight"]
    for args, kw, what in [
            ((x.cpu(), w), {}, ValueError), ((x[0], w), {}, ValueError), ((x.half(), w), {}, TypeError), ((x, w[:8]), {}, ValueError),
            ((x, w.bfloat16()), {}, TypeError), ((x, w[:, 0]), {}, ValueError), ((x, torch.cat([w, w], 1)), {}, ValueError), ((x, w[:, :0]), {}, ValueError),
            ((x, w, g["bias"][:8]), {}, ValueError), ((x, w), dict(state0=g["state0"][:, :2]), ValueError), ((x, w), dict(state0=g["state0"].bfloat16()), TypeError),
            ((x, w), dict(starts=torch.zeros(2, 9, dtype=torch.bool, device="cuda")), ValueError), ((x[..., :12], w[:12]), {}, ssm.SSMError),
            ((x, w), dict(lengths=torch.zeros(2, device="cuda")), TypeError)]:
        with pytest.raises(what):
            f(*args, **kw)
    with pytest.raises(ValueError):
        ssm.causal_conv_update(g["state0"][:, 1:], x[:, 0], w)
    with pytest.raises(TypeError):
        ssm.causal_conv_update(g["state0"].bfloat16(), x[:, 0], w)

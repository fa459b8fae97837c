"""The norm and rotation of heads on the GPU against the 64-bit reference.

Tolerances (largest difference beyond the result's own rounding to its type, over the
largest reference value, per output): a sum over a head taken pairwise over lanes and
about ten roundings of 2^-24, and for the farthest positions 2^31 2^-53 twice in
the angle: 2e-6; 1e-5 for the gradients of weights, sums over up to thousands of heads."""
from __future__ import annotations

import math

import pytest
import torch

from tests import mixer_reference as ref
from tests.test_mixer_plans import HEADS

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


ARGS = ("q", "k", "q_weight", "k_weight", "positions", "inv_freq")


def forward(ssm, g, **kw):
    return ssm.head_norm_rotary_fwd(*(g[n] for n in ARGS), **kw)


def backward(ssm, g, **kw):
    return ssm.head_norm_rotary_bwd(g["dq_out"], g["dk_out"], *(g[n] for n in ARGS), **kw)


def check(ssm, B, L, Hq, Hk, d, rot, eps=1e-6, norm=True, interleaved=False, **kw):
    print("heads", B, L, Hq, Hk, d, rot, norm, interleaved, kw, flush=True)
    p = ref.head_inputs(B, L, Hq, Hk, d, rot, **kw)
    compare(ssm, p, ref.on_gpu(p), eps=eps, norm=norm, interleaved=interleaved)


def compare(ssm, p, g, **kw):
    out = dict(zip(("q", "k"), forward(ssm, g, **kw)))
    d = backward(ssm, g, **kw)
    ro, rg = ref.heads(p, **kw)
    for n, got in out.items():
        assert (got is None) == (n not in ro)
        if got is not None:
            assert got.dtype == p["q"].dtype and got.is_contiguous()
            assert ref.error(got, ro[n]) <= TOL, (n, ref.error(got, ro[n]))
    for n, got in d.items():
        assert (got is None) == (n not in rg), n
        if got is not None:
            e = ref.error(got, rg[n])
            assert e <= (SUMS if n.endswith("weight") else TOL), (n, e)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("d,rot", [(8, 8), (16, 8), (24, 24), (32, 16), (40, 40), (64, 64), (72, 72), (72, 24), (96, 88), (128, 128), (128, 64),
                                   (136, 136), (192, 96), (256, 256), (256, 8), (248, 240)])
def test_head_sizes(ssm, dtype, interleaved, d, rot):
    check(ssm, 2, 19, 3, 2, d, rot, interleaved=interleaved, dtype=dtype, seed=d + rot)


@pytest.mark.parametrize("weights", ["shared", "per head", None])
@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("rot", [0, 32])
@pytest.mark.parametrize("Hk", [0, 2])
@pytest.mark.parametrize("per_batch", [True, False])
def test_options(ssm, weights, norm, rot, Hk, per_batch):
    check(ssm, 3, 21, 4, Hk, 32, rot, norm=norm, weights=weights if norm else None, per_batch=per_batch, dtype=BF16 if rot else F32)


@pytest.mark.parametrize("Hq,Hk", [(1, 1), (1, 0), (5, 1), (7, 3), (16, 16), (17, 1), (40, 8), (40, 40), (64, 1), (130, 2)])
@pytest.mark.parametrize("weights", ["shared", "per head"])
def test_head_counts(ssm, Hq, Hk, weights):
    check(ssm, 2, 11, Hq, Hk, 64, 64, weights=weights)
    check(ssm, 1, 5, Hq, Hk, 128, 64, weights=weights, dtype=BF16)


@pytest.mark.parametrize("B,L", [(1, 1), (2, 1), (1, 2), (300, 1), (1, 1000), (3, 333), (64, 9)])
def test_tokens(ssm, B, L):
    check(ssm, B, L, 4, 2, 32, 32, weights="per head")
    check(ssm, B, L, 2, 1, 128, 128, per_batch=False)


@pytest.mark.parametrize("B", [1, 7, 256])
@pytest.mark.parametrize("interleaved", [True, False])
def test_single_tokens(ssm, B, interleaved):
    check(ssm, B, None, 8, 2, 64, 64, interleaved=interleaved, dtype=BF16, far=True)
    check(ssm, B, None, 3, 0, 40, 16, interleaved=interleaved, weights="per head")


@pytest.mark.parametrize("interleaved", [True, False])
def test_far_positions(ssm, interleaved):
    """Positions up to 2^31, where fp32 has no digits of the angle left."""
    check(ssm, 2, 40, 2, 2, 64, 64, far=True, interleaved=interleaved)


def test_quarter_turns(ssm):
    """Angles at and next to the borders between quarters."""
    p = ref.head_inputs(1, 64, 1, 1, 16, 16, weights=None)
    p["positions"] = torch.arange(64)[None]
    p["inv_freq"] = torch.tensor([math.pi / 4, math.pi / 2, math.pi, -math.pi / 4, math.pi / 4 + 1e-9, math.pi / 4 - 1e-9, 0.0, 2 * math.pi], dtype=torch.float64)
    compare(ssm, p, ref.on_gpu(p))


@pytest.mark.parametrize("mag", [1e-12, 1e-3, 1e15])
def test_magnitudes(ssm, mag):
    p = ref.head_inputs(2, 9, 2, 1, 32, 32)
    p["q"] *= mag
    p["k"] *= mag
    compare(ssm, p, ref.on_gpu(p), eps=1e-5)


def test_zero_and_bad_heads_stay_by_themselves(ssm):
    p = ref.head_inputs(1, 6, 3, 2, 32, 32)
    p["q"][0, 2, 1] = 0
    compare(ssm, p, ref.on_gpu(p))
    clean, _ = ref.heads(p)
    p["q"][0, 3, 0, 5] = math.nan
    p["k"][0, 4, 1, 7] = math.inf
    q, k = (t.cpu() for t in forward(ssm, ref.on_gpu(p)))
    for got, want, t, h in [(q, clean["q"], 3, 0), (k, clean["k"], 4, 1)]:
        assert torch.isnan(got[0, t, h]).any()
        got[0, t, h] = want[0, t, h].float()
        assert ref.error(got, want) <= TOL


@pytest.mark.parametrize("sizes", sorted(HEADS), ids=str)
@pytest.mark.parametrize("weights,interleaved,strided", [("shared", False, False), ("per head", True, False), ("shared", True, True), ("per head", False, True)])
def test_training_sizes(ssm, sizes, weights, interleaved, strided):
    """Several chunks of tokens to a workgroup: the angles filled again, sums carried on, batch rows apart or as one."""
    B, L, Hq, Hk, d, es = sizes
    print("heads", sizes, weights, interleaved, strided, flush=True)
    p = ref.head_inputs(B, L, Hq, Hk, d, d, weights=weights, dtype=BF16 if es == 2 else F32, seed=L)
    g = ref.on_gpu(p)
    if strided:  # heads before steps: no row of the batch follows the one before it
        for n in ("q", "k", "dq_out", "dk_out"):
            g[n] = g[n].transpose(1, 2).contiguous().transpose(1, 2)
    out = dict(zip(("q", "k"), forward(ssm, g, interleaved=interleaved)))
    got = backward(ssm, g, interleaved=interleaved)
    with torch.device("cuda"):
        want, grads = ref.heads(g, interleaved=interleaved)
    for n, t in out.items():
        assert ref.error(t, want[n].cpu()) <= TOL, n
    for n, t in got.items():
        assert ref.error(t, grads[n].cpu()) <= (SUMS if n.endswith("weight") else TOL), n


@pytest.mark.parametrize("seed", range(20))
def test_random(ssm, seed):
    gen = torch.Generator().manual_seed(seed)
    pick = lambda lo, hi: int(torch.randint(lo, hi + 1, (1,), generator=gen))  # noqa: E731
    d = 8 * pick(1, 32)
    norm = pick(0, 3) > 0
    check(ssm, pick(1, 5), pick(1, 60), pick(1, 12), pick(0, 5), d, 8 * pick(0, d // 8), norm=norm, interleaved=bool(pick(0, 1)),
          weights=("shared", "per head", None)[pick(0, 2)] if norm else None, per_batch=bool(pick(0, 1)), dtype=(F32, BF16)[pick(0, 1)], seed=seed)


def test_strides(ssm):
    """Slices of a fused projection, heads before steps, a batch that shares its rows."""
    p = ref.head_inputs(3, 14, 4, 2, 32, 32, dtype=BF16)
    g = ref.on_gpu(p)
    want, wantd = forward(ssm, g), backward(ssm, g)
    fused = torch.cat([g["q"], g["k"], g["dq_out"], g["dk_out"]], 2)
    cut = dict(zip(("q", "k", "dq_out", "dk_out"), fused.split([4, 2, 4, 2], 2)))
    swapped = {n: g[n].transpose(1, 2).contiguous().transpose(1, 2) for n in cut}
    time_first = {n: g[n].transpose(0, 1).contiguous().transpose(0, 1) for n in cut}
    for views in (cut, swapped, time_first):
        v = {**g, **views}
        got, gotd = forward(ssm, v), backward(ssm, v)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        assert all(torch.equal(gotd[n], wantd[n]) for n in ("dq", "dk"))
        assert all(ref.error(gotd[n], wantd[n].cpu()) <= SUMS for n in ("dq_weight", "dk_weight"))  # (another order of the sum)
    one = {**g, "q": g["q"][:1].expand(3, -1, -1, -1), "k": g["k"][:, :, :1].expand(-1, -1, 2, -1)}
    full = {n: t.contiguous() for n, t in one.items()}
    assert all(torch.equal(a, b) for a, b in zip(forward(ssm, one), forward(ssm, full)))


def test_offsets_beyond_32_bits(ssm):
    p = ref.head_inputs(2, 9, 2, 1, 32, 32, dtype=BF16)
    g = ref.on_gpu(p)
    gap = 2 ** 31 + 64
    big = torch.empty(gap + 9 * 64, dtype=BF16, device="cuda").as_strided((2, 9, 2, 32), (gap, 64, 32, 1))
    for n in ("q", "dq_out"):
        big.copy_(g[n])
        v = {**g, n: big}
        a, b = backward(ssm, g), backward(ssm, v)
        assert torch.equal(forward(ssm, g)[0], forward(ssm, v)[0]) and torch.equal(a["dq"], b["dq"]) and torch.equal(a["dk"], b["dk"])


def test_outputs_beyond_32_bits(ssm):
    L, H, d = 33000, 512, 128
    row = torch.randn(1, H, d, generator=torch.Generator(device="cuda").manual_seed(0), device="cuda").to(BF16)
    pos = torch.zeros(1, L, dtype=torch.int64, device="cuda")
    inv = (10000.0 ** (-torch.arange(0, d, 2, dtype=torch.float64) / d)).cuda()
    pos[0, -1] = 77
    q, _ = ssm.head_norm_rotary_fwd(row.expand(1, L, H, d), positions=pos, inv_freq=inv)
    one, _ = ssm.head_norm_rotary_fwd(row, positions=pos[:, -1].contiguous(), inv_freq=inv)
    assert torch.equal(q[0, -1], one[0])


def test_same_bits_streams_and_graph(ssm):
    ps = [ref.head_inputs(2, 300, 8, 2, 64, 64, dtype=BF16, seed=i) for i in range(3)]
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
    for Hk in (0, 2):
        p = ref.head_inputs(2, 9, 4, Hk, 32, 32)
        g = ref.on_gpu(p)
        leaves = {n: g[n].clone().requires_grad_() for n in ref.HEAD_INPUTS if g[n] is not None}
        q, k = ssm.head_norm_rotary(leaves["q"], leaves.get("k"), leaves["q_weight"], leaves.get("k_weight"), g["positions"], g["inv_freq"])
        loss = (q * g["dq_out"]).sum()
        if Hk:
            loss = loss + (k * g["dk_out"]).sum()
        loss.backward()
        rg = ref.heads(p)[1]
        for n, t in leaves.items():
            assert ref.error(t.grad, rg["d" + n]) <= SUMS, n
    q = g["q"].clone().requires_grad_()
    a, b = ssm.head_norm_rotary(q, q, positions=g["positions"], inv_freq=g["inv_freq"])  # the same input twice, one output used
    b.square().sum().backward()
    want = q.detach().cpu().double().requires_grad_()
    (want / torch.sqrt((want * want).mean(-1, keepdim=True) + 1e-6)).square().sum().backward()
    assert float((q.grad.cpu() - want.grad).abs().max()) <= 1e-5


def test_refusals(ssm):
    g = ref.on_gpu(ref.head_inputs(2, 5, 4, 2, 32, 32))
    q, k, qw, kw_, pos, inv = (g[n] for n in ARGS)
    f = ssm.head_norm_rotary_fwd
    for args, kw, what in [
            ((q.cpu(),), {}, ValueError), ((q[0, 0],), {}, ValueError), ((q.half(),), {}, TypeError), ((q, k.bfloat16()), {}, TypeError), ((q, k[0]), {}, ValueError),
            ((q, k[..., :16]), {}, ValueError), ((q, k[:1]), {}, ValueError), ((q, k, qw), {}, ValueError), ((q, k, None, kw_), {}, ValueError), ((q, None, qw, kw_), {}, ValueError),
            ((q, k, qw[:16], kw_[:16]), {}, ValueError), ((q, k, qw.double(), kw_), {}, TypeError), ((q, k, qw, kw_.expand(2, 32).contiguous()), {}, ValueError),
            ((q, k, qw, kw_), dict(norm=False), ValueError), ((q, k, qw, kw_, pos), {}, ValueError), ((q, k, qw, kw_, None, inv), {}, ValueError),
            ((q, k, qw, kw_, pos.int(), inv), {}, TypeError), ((q, k, qw, kw_, pos[:1], inv), {}, ValueError), ((q, k, qw, kw_, pos, inv.float()), {}, TypeError),
            ((q, k, qw, kw_, pos, inv[:3].contiguous()), {}, ValueError), ((q, k, qw, kw_, pos, torch.cat([inv, inv])), {}, ValueError), ((q, k, qw, kw_, pos, inv[:0]), {}, ValueError),
            ((q[..., :20], k[..., :20]), {}, ssm.SSMError), ((q[:, :0], k[:, :0]), {}, ssm.SSMError), ((q, k), dict(eps=-1.0), ssm.SSMError), ((q, k), dict(eps=math.nan), ssm.SSMError)]:
        with pytest.raises(what):
            f(*args, **kw)
    with pytest.raises(ValueError):
        ssm.head_norm_rotary_bwd(q[:, :4], k, q, k)
    with pytest.raises(ssm.SSMError):
        ssm.head_norm_rotary_fwd(torch.zeros(1, 2, 2, 264, device="cuda"))

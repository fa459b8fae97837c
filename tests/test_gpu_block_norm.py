"""The norms around a block on the GPU against 64-bit references.

Tolerances (largest difference beyond the result's own rounding to its type,
over the largest reference value, per output): a few roundings of 2^-24 and one
sum over a row, taken pairwise over lanes: 2e-6; 1e-5 for the gradients of
weights and scales, sums over up to thousands of rows."""
from __future__ import annotations

import math

import pytest
import torch

from tests import block_reference as ref

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
TOL = 2e-6
SUMS = 1e-5
EPS = 1e-5


@pytest.fixture(scope="module")
def ssm():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import selective_state_space_10_amd as m
    m.load()
    return m


def _draw(seed):
    g = torch.Generator().manual_seed(seed)
    return lambda *s: torch.randn(*s, generator=g)


def _check(got, want, tol):
    err = ref.error(got, want)
    assert err <= tol, err


def _residual(ssm, shape, dtype, rdtype, scaled, with_dh=True, seed=0, eps=EPS, mag=1.0):
    print("residual norm", shape, dtype, rdtype, scaled, with_dh, flush=True)
    r = _draw(seed)
    D = shape[-1]
    x, res = (mag * r(*shape)).to(dtype), (mag * r(*shape)).to(rdtype)
    w, sc = 1 + 0.2 * r(D), (0.5 + 0.2 * r(D)) if scaled else None
    dy, dh = r(*shape).to(dtype), r(*shape).to(rdtype) if with_dh else None
    gx, gr, gw, gs, gy, gh = (None if t is None else t.cuda() for t in (x, res, w, sc, dy, dh))
    y, h, rstd = ssm.residual_norm_fwd(gx, gr, gw, gs, eps)
    ry, rh, rr = ref.residual_norm(x, res, w, sc, eps)
    _check(y, ry, TOL)
    _check(h, rh, TOL)
    _check(rstd, rr, TOL)
    g = ssm.residual_norm_bwd(gy, gh, h, rstd, gw, gx if scaled else None, gs)
    want = ref.residual_norm_bwd(dy, dh, h.cpu(), rstd.cpu(), w, x, sc)
    assert g["dresidual"].dtype == rdtype and g["dx"].dtype == dtype
    _check(g["dresidual"], want["dresidual"], TOL)
    _check(g["dx"], want["dx"], TOL)
    _check(g["dweight"], want["dweight"], SUMS)
    if scaled:
        _check(g["dscale"], want["dscale"], SUMS)
    else:
        assert g["dscale"] is None


@pytest.mark.parametrize("dtype,rdtype", [(F32, F32), (BF16, F32), (BF16, BF16)])
@pytest.mark.parametrize("D", [8, 16, 120, 128, 136, 512, 520, 1024, 1032, 2048, 2056, 4096, 4104, 5120, 8192, 8200, 16384])
def test_residual_row_lengths(ssm, dtype, rdtype, D):
    _residual(ssm, (5, D), dtype, rdtype, True, seed=D)


@pytest.mark.parametrize("scaled", [True, False])
@pytest.mark.parametrize("with_dh", [True, False])
@pytest.mark.parametrize("dtype,rdtype", [(F32, F32), (BF16, F32), (BF16, BF16)])
def test_residual_options(ssm, dtype, rdtype, scaled, with_dh):
    _residual(ssm, (3, 7, 264), dtype, rdtype, scaled, with_dh)


@pytest.mark.parametrize("rows", [1, 2, 15, 16, 17, 1023, 5000, 40000])
@pytest.mark.parametrize("D", [40, 264])
def test_residual_rows(ssm, rows, D):
    _residual(ssm, (rows, D), F32, F32, True, seed=rows)


@pytest.mark.parametrize("mag", [1e-12, 1e-3, 1e15])
def test_residual_magnitudes(ssm, mag):
    _residual(ssm, (4, 264), F32, F32, False, mag=mag)


def _gated(ssm, rows, D, group, dtype, gate_first, with_z=True, seed=0):
    print("gated norm", rows, D, group, dtype, gate_first, with_z, flush=True)
    r = _draw(seed)
    x, z, w, dy = (2 * r(rows, D)).to(dtype), r(rows, D).to(dtype) if with_z else None, 1 + 0.2 * r(D), r(rows, D).to(dtype)
    gx, gz, gw, gy = (None if t is None else t.cuda() for t in (x, z, w, dy))
    y, rstd = ssm.gated_norm_fwd(gx, gz, gw, group, EPS, gate_first)
    g = ssm.gated_norm_bwd(gy, gx, gz, gw, rstd, group, gate_first)
    ry, rr, rg = ref.gated_norm(x, z, w, group, EPS, gate_first, dy)
    _check(y, ry, TOL)
    _check(rstd, rr, TOL)
    _check(g["dx"], rg["dx"], TOL)
    _check(g["dweight"], rg["dweight"], SUMS)
    if with_z:
        _check(g["dz"], rg["dz"], TOL)
    else:
        assert g["dz"] is None


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("gate_first", [True, False])
@pytest.mark.parametrize("D,group", [(8, 8), (64, 8), (120, 24), (640, 128), (384, 192), (1536, 512), (1560, 520), (2048, 2048),
                                     (4112, 2056), (5120, 5120), (8192, 8192), (16400, 8200), (16384, 16384)])
def test_gated_groups(ssm, dtype, gate_first, D, group):
    _gated(ssm, 5, D, group, dtype, gate_first, seed=D)


@pytest.mark.parametrize("gate_first", [True, False])
@pytest.mark.parametrize("rows", [1, 3, 17, 1000, 30000])
def test_gated_rows(ssm, rows, gate_first):
    _gated(ssm, rows, 192, 64, F32, gate_first, seed=rows)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("group", [16, 264])
def test_no_gate(ssm, dtype, group):
    _gated(ssm, 9, 528, group, dtype, False, with_z=False)


def test_far_gates(ssm):
    """silu far out: 0 to the left, z to the right, and their derivatives."""
    z = torch.tensor([-200.0, -100.0, -90.0, -30.0, 30.0, 90.0, 200.0, 1e30] * 2)[None]
    x, w, dy = torch.ones(1, 16), torch.ones(16), torch.ones(1, 16)
    y, rstd = ssm.gated_norm_fwd(x.cuda(), z.cuda(), w.cuda())
    g = ssm.gated_norm_bwd(dy.cuda(), x.cuda(), z.cuda(), w.cuda(), rstd)
    s = torch.sigmoid(z.double())
    r = 1 / math.sqrt(1 + EPS)
    assert torch.allclose(y.cpu().double(), z.double() * s * r, rtol=1e-5, atol=1e-30)
    assert torch.allclose(g["dz"].cpu().double(), (s + z.double() * s * (1 - s)) * r, rtol=1e-5, atol=1e-30)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_slices_and_same_bits(ssm, dtype):
    r = _draw(3)
    both = r(3, 11, 2 * 264).to(dtype).cuda()
    x, z = both[..., :264], both[..., 264:]
    w, res = (1 + 0.1 * r(264)).cuda(), r(3, 11, 264).cuda()
    dy = r(3, 11, 264).to(dtype).cuda()
    a, ra = ssm.gated_norm_fwd(x, z, w, 88)
    b, rb = ssm.gated_norm_fwd(x.contiguous(), z.contiguous(), w, 88)
    assert torch.equal(a, b) and torch.equal(ra, rb)
    ga, gb = ssm.gated_norm_bwd(dy, x, z, w, ra, 88), ssm.gated_norm_bwd(dy, x.contiguous(), z.contiguous(), w, ra, 88)
    assert all(torch.equal(ga[n], gb[n]) for n in ga)
    a, b = ssm.residual_norm_fwd(x, res, w, w), ssm.residual_norm_fwd(x.contiguous(), res, w, w)
    assert all(torch.equal(p, q) for p, q in zip(a, b))


@pytest.mark.parametrize("gate_first", [True, False])
def test_autograd(ssm, gate_first):
    r = _draw(5)
    x, z, w = r(6, 48).cuda().requires_grad_(), r(6, 48).cuda().requires_grad_(), (1 + 0.1 * r(48)).cuda().requires_grad_()
    res, sc = r(6, 48).cuda().requires_grad_(), (0.5 + 0.1 * r(48)).cuda().requires_grad_()
    y, h = ssm.residual_norm(x, res, w, sc)
    u = ssm.gated_norm(y, z, w, 16, EPS, gate_first)
    dy, dh = r(6, 48).cuda(), r(6, 48).cuda()
    got = torch.autograd.grad([u, h], [x, z, w, res, sc], [dy, dh])
    xs = [t.detach().cpu().double().requires_grad_() for t in (x, z, w, res, sc)]
    X, Z, W, R, S = xs
    H = R + S * X
    Y = H / torch.sqrt((H * H).mean(-1, keepdim=True) + EPS) * W
    gate = Z * torch.sigmoid(Z)
    t = (Y * gate if gate_first else Y).view(6, 3, 16)
    U = (t / torch.sqrt((t * t).mean(-1, keepdim=True) + EPS)).view(6, 48) * W
    U = U if gate_first else U * gate
    want = torch.autograd.grad([U, H], xs, [dy.cpu().double(), dh.cpu().double()])
    for a, b in zip(got, want):
        _check(a, b, SUMS)


def test_only_one_gradient_arrives(ssm):
    r = _draw(6)
    x, res, w = r(4, 64).cuda().requires_grad_(), r(4, 64).cuda(), torch.ones(64).cuda()
    y, h = ssm.residual_norm(x, res, w)
    (gx,) = torch.autograd.grad(h.sum(), x)
    assert torch.equal(gx, torch.ones_like(gx))


def test_refusals(ssm):
    r = _draw(0)
    x, res, w = r(4, 64).cuda(), r(4, 64).cuda(), torch.ones(64).cuda()
    for bad in (lambda: ssm.residual_norm_fwd(x, res[:2], w), lambda: ssm.residual_norm_fwd(x, res, w[:32]),
                lambda: ssm.residual_norm_fwd(x.cpu(), res, w), lambda: ssm.residual_norm_fwd(x, res.cpu(), w),
                lambda: ssm.residual_norm_fwd(x[:, ::2], res[:, :32].contiguous(), w[:32]),
                lambda: ssm.residual_norm_fwd(x[:, :60].contiguous(), res[:, :60].contiguous(), w[:60].contiguous()),
                lambda: ssm.residual_norm_fwd(x[:0], res[:0], w),
                lambda: ssm.gated_norm_fwd(x, x, w, 24), lambda: ssm.gated_norm_fwd(x, x, w, 4), lambda: ssm.gated_norm_fwd(x, x[:2], w),
                lambda: ssm.gated_norm_bwd(x, x, x, w, torch.ones(4, 2).cuda(), 64)):
        with pytest.raises((ValueError, ssm.SSMError)):
            bad()
    for bad in (lambda: ssm.residual_norm_fwd(x, res.bfloat16(), w), lambda: ssm.residual_norm_fwd(x, res, w.bfloat16()),
                lambda: ssm.residual_norm_fwd(x.half(), res, w), lambda: ssm.gated_norm_fwd(x, x.bfloat16(), w)):
        with pytest.raises(TypeError):
            bad()
    big = torch.zeros(1, 16392, device="cuda")
    with pytest.raises(ssm.SSMError):
        ssm.residual_norm_fwd(big, big, big[0])

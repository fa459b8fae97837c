"""The convolution, the gated recurrence, the norm and rotation of heads, decay attention and
the norms together, as blocks use them (examples/recurrent_blocks.py): gradients on packed and
padded batches against the same blocks in 64 bits, and serving against the prompt."""
from __future__ import annotations

import math

import pytest
import torch

from tests.block_reference import error

pytestmark = pytest.mark.gpu
F64 = torch.float64


@pytest.fixture(scope="module")
def blocks():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from examples import recurrent_blocks as m
    return m


# ---- the operators in 64 bits, differentiable, on the CPU


def rms(x, eps):
    return x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)


def conv(x, w, b, starts, lengths=None):
    K, L = w.shape[1], x.shape[1]
    doc = torch.zeros(x.shape[:2]) if starts is None else starts.long().cumsum(1)
    y = torch.zeros_like(x) if b is None else b.expand_as(x)
    for back in range(min(K, L)):
        same = torch.nn.functional.pad(doc[:, back:] == doc[:, :L - back], (back, 0))
        tap = torch.nn.functional.pad(x[:, :L - back], (0, 0, back, 0))
        y = y + w[:, K - 1 - back] * torch.where(same[..., None], tap, 0.0)
    y = y * torch.sigmoid(y)
    return y if lengths is None else torch.where((torch.arange(L) < lengths[:, None])[..., None], y, 0.0)


def recurrence(x, g, i, decay, z, starts, lengths=None):
    la = -8 * torch.nn.functional.softplus(decay) * torch.sigmoid(g)
    a, u = torch.exp(la), torch.sigmoid(i) * x
    h, hs = torch.zeros_like(x[:, 0]), []
    for t in range(x.shape[1]):
        new = a[:, t] * h + torch.sqrt(-torch.expm1(2 * la[:, t])) * u[:, t]
        if starts is not None:
            new = torch.where(starts[:, t, None], u[:, t], new)
        h = new
        hs.append(h)
    y = torch.stack(hs, 1) * z * torch.sigmoid(z)
    return y if lengths is None else torch.where((torch.arange(x.shape[1]) < lengths[:, None])[..., None], y, 0.0)


def turned(x, w, pos, inv):
    x = rms(x, 1e-6) * w
    ang = pos.to(F64)[..., None, None] * inv
    one, two = x.chunk(2, -1)
    return torch.cat([one * torch.cos(ang) - two * torch.sin(ang), two * torch.cos(ang) + one * torch.sin(ang)], -1)


def attention(q, k, v, g):
    share = v.shape[2] // q.shape[2]
    q, k = q.repeat_interleave(share, 2), k.repeat_interleave(share, 2)
    s, o = torch.zeros(*v.shape[:1], v.shape[2], q.shape[3], v.shape[3], dtype=F64), []
    for t in range(q.shape[1]):
        s = torch.where(torch.isinf(g[:, t])[..., None, None], 0.0, torch.exp(g[:, t])[..., None, None] * s)
        s = s + k[:, t, :, :, None] * v[:, t, :, None, :]
        o.append((q[:, t, :, :, None] * s).sum(-2) * q.shape[3] ** -0.5)
    return torch.stack(o, 1)


def reference(p, block, x, residual, **kw):
    h = x + residual
    y = rms(h, 1e-5) * p["norm"]
    u = y @ p["project.weight"].T
    starts = kw.get("starts")
    if "decay" in p:
        u, z, g, i = u.split(block.inner, -1)
        u = conv(u, p["conv"], p["conv_bias"], starts, kw.get("lengths"))
        o = recurrence(u, g, i, p["decay"], z, starts, kw.get("lengths"))
        return o @ p["out.weight"].T, h
    u, z, a = u.split(block.parts, -1)
    q, k, v = block._heads(conv(u, p["conv"], None, starts))
    q, k = turned(q, p["q_norm"], kw["positions"], block.inv_freq.cpu()), turned(k, p["k_norm"], kw["positions"], block.inv_freq.cpu())
    g = -torch.nn.functional.softplus(a[..., :block.sizes[0]] + p["decay_bias"])
    if starts is not None:
        g = g.masked_fill(starts[..., None], -math.inf)
    o = attention(q, k, v, g)
    o = (rms(o, 1e-5)).flatten(2) * p["gate_norm"] * z * torch.sigmoid(z)
    return o @ p["out.weight"].T, h


@pytest.mark.parametrize("kind", ["recurrent", "attention"])
@pytest.mark.parametrize("packed", [False, True])
def test_gradients(blocks, kind, packed):
    """fp32: products of width up to 160 in another order and up to 70 steps of a recurrence,
    each off by a few units of 2^-24, through four operators and back: 200 roundings of
    either sign like 15 of one sign twice over, times four operators: 120 2^-24 = 7e-6, taken as 2e-5."""
    torch.manual_seed(1)
    B, L, width = 3, 70, 96
    block = blocks.RecurrentBlock(width, 72, dtype=torch.float32) if kind == "recurrent" else blocks.LinearAttentionBlock(width, 4, 2, 24, 32, dtype=torch.float32)
    gen = torch.Generator().manual_seed(2)
    r = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    x, residual, dy, dh = r(B, L, width), r(B, L, width), r(B, L, width), r(B, L, width)
    starts = torch.rand(B, L, generator=gen) < 0.1 if packed else None
    lengths = torch.tensor([L, 41, 0], dtype=torch.int32) if packed and kind == "recurrent" else None
    kw = {"starts": starts}
    if kind == "recurrent":
        kw["lengths"] = lengths
    else:
        kw["positions"] = blocks.document_positions(starts) if packed else torch.arange(L).expand(B, -1).contiguous()
    gx, gres = x.cuda().requires_grad_(), residual.cuda().requires_grad_()
    out, h, _ = block(gx, gres, **{n: None if t is None else t.cuda() for n, t in kw.items()})
    ((out * dy.cuda()).sum() + (h * dh.cuda()).sum()).backward()

    p = {n: t.detach().cpu().to(F64).requires_grad_() for n, t in block.named_parameters()}
    rx, rres = x.to(F64).requires_grad_(), residual.to(F64).requires_grad_()
    want, rh = reference(p, block, rx, rres, **kw)
    loss = (want * dy.to(F64)).sum() + (rh * dh.to(F64)).sum()
    loss.backward()
    assert error(out, want.detach()) <= 2e-5
    for n, got, ref in [("x", gx.grad, rx.grad), ("residual", gres.grad, rres.grad)] + [(n, t.grad, p[n].grad) for n, t in block.named_parameters()]:
        assert error(got, ref) <= 2e-5, (n, error(got, ref))


@pytest.mark.parametrize("dtype,tol", [(torch.float32, 1e-4), (torch.bfloat16, 6e-2)])
def test_serving(blocks, dtype, tol):
    """Serving differs from the prompt by rounding alone: fp32 products in another order; in bf16
    six roundings of 2^-8 (three products, a convolution, a norm and a mixing in each block) through
    a norm and two products of random sign."""
    assert blocks.served(dtype) <= tol


@pytest.mark.parametrize("documents", [(1, 40, 59), (100,)])
def test_packed_training_is_what_is_served(blocks, documents):
    """Documents packed into one training row, and each served by itself, as a prompt of a part of it and single
    tokens.  fp32: as in test_serving, products in another order."""
    torch.manual_seed(4)
    block = blocks.RecurrentBlock(64, 72, dtype=torch.float32)
    gen = torch.Generator().manual_seed(5)
    x, residual = torch.randn(1, 100, 64, generator=gen).cuda(), torch.randn(1, 100, 64, generator=gen).cuda()
    starts = torch.zeros(1, 100, dtype=torch.bool, device="cuda")
    at = 0
    for n in documents:
        starts[:, at] = True
        at += n
    with torch.no_grad():
        want = block(x, residual, starts=starts)[0]
        got, at = [], 0
        for n in documents:
            cut = max(1, n // 2)
            y, _, state = block.prompt(x[:, at:at + cut], residual[:, at:at + cut])
            got.append(y)
            got += [block.step(x[:, t], residual[:, t], state)[0][:, None] for t in range(at + cut, at + n)]
            at += n
    assert error(torch.cat(got, 1), want.cpu()) <= 1e-4


def test_training_steps_in_a_graph(blocks):
    """Forward, backward and gradients of both blocks captured once and replayed on other
    inputs, with eager steps of the same blocks between; all eager graphs are gone
    when the capture begins."""
    torch.manual_seed(3)
    width, B, L = 64, 2, 200
    one = blocks.RecurrentBlock(width, 64)
    two = blocks.LinearAttentionBlock(width, 2, 2, 32, 32)
    params = [*one.parameters(), *two.parameters()]
    starts = torch.rand(B, L, device="cuda") < 0.05
    positions = blocks.document_positions(starts)

    def step(x, residual):
        y, h, _ = one(x, residual, starts=starts)
        out, h, _ = two(y, h, positions, starts=starts)
        return torch.autograd.grad((out.float().square() + h.square()).mean(), params)

    draw = lambda i: (torch.randn(B, L, width, generator=torch.Generator("cuda").manual_seed(i), device="cuda").bfloat16(),  # noqa: E731
                      torch.randn(B, L, width, generator=torch.Generator("cuda").manual_seed(100 + i), device="cuda"))
    x, residual = (t.clone() for t in draw(0))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(x, residual)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        grads = step(x, residual)
    for i in (1, 2, 3):
        a, b = draw(i)
        x.copy_(a)
        residual.copy_(b)
        graph.replay()
        torch.cuda.synchronize()
        want = step(a, b)
        torch.cuda.synchronize()
        for got, ref in zip(grads, want):
            assert error(got, ref.cpu()) <= 2e-2  # (library products and sums may take another order)
        del want

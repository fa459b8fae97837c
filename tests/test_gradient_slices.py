"""Gradients that autograd hands to the operators as slices of a larger one: contiguous,
but not on a 16-byte boundary, as behind a concatenation of flattened outputs."""
from __future__ import annotations

import pytest
import torch

from selective_state_space_10_amd import block_ops, mixer_ops, ops


def test_a_gradient_is_aligned():
    t = torch.arange(64.0).reshape(8, 8)
    assert ops._gradient(None) is None and ops._gradient(t) is t
    for view in (t.flatten()[1:33].view(4, 8), t.t(), t[:1].expand(8, 8)):
        g = ops._gradient(view)
        assert g.is_contiguous() and g.data_ptr() % 16 == 0 and torch.equal(g, view)


R = lambda *s: torch.rand(*s, requires_grad=True)  # noqa: E731
# module, name of the calls, operator, its call, how many tensors the forward call returns
STAND_INS = [
    (mixer_ops, "gated_recurrence", "gated_recurrence", lambda f: f(R(2, 3, 8), R(2, 3, 8)), 3),
    (mixer_ops, "causal_conv", "causal_conv", lambda f: f(R(2, 3, 8), R(8, 2)), 2),
    (mixer_ops, "head_norm_rotary", "head_norm_rotary", lambda f: f(R(2, 3, 2, 8), R(2, 3, 2, 8)), 2),
    (block_ops, "decay_attn", "decay_attention", lambda f: f(R(2, 3, 2, 8), R(2, 3, 2, 8), R(2, 3, 2, 8), torch.rand(2)), 2),
    (block_ops, "residual_norm", "residual_norm", lambda f: f(R(2, 8), R(2, 8), R(8)), 3),
    (block_ops, "gated_norm", "gated_norm", lambda f: f(R(2, 8), None, R(8)), 2),
    (ops, "scan", "selective_scan", lambda f: f(R(2, 3, 8), R(2, 3, 8), R(8, 4), R(2, 3, 4), R(2, 3, 4)), 3),
    (ops, "scan_{}_conv", "conv_selective_scan", lambda f: f(R(2, 3, 8), R(8, 2), R(8), R(2, 3, 8), R(8, 4), R(2, 3, 4), R(2, 3, 4)), 3),
]


@pytest.mark.parametrize("module,name,operator,call,returned", STAND_INS, ids=[s[2] for s in STAND_INS])
def test_backward_calls_get_aligned_gradients(monkeypatch, module, name, operator, call, returned):
    """Plain stand-ins for the kernels' calls: outputs of a shape of their own, by which the backward finds its gradients."""
    seen, name = [], name if "{}" in name else name + "_{}"

    class NoGradients(dict):
        def __missing__(self, key):
            return None

    def backward(*args, **kw):
        seen.extend(t for t in args if isinstance(t, torch.Tensor) and t.shape == (5, 1, 8))
        return NoGradients()

    monkeypatch.setattr(module, name.format("fwd"), lambda *a, **kw: tuple(torch.zeros(5, 1, 8) for _ in range(returned)))
    monkeypatch.setattr(module, name.format("bwd"), backward)
    out = call(getattr(module, operator))
    out = out if isinstance(out, tuple) else (out,)
    joined = torch.cat([torch.zeros(1)] + [t.flatten() for t in out])
    (joined * torch.arange(1.0, 1 + joined.numel())).sum().backward()
    assert sum(t.unique().numel() == 40 for t in seen) == len(out)
    assert all(t.is_contiguous() and t.data_ptr() % 16 == 0 for t in seen)


def _operators(ssm):
    gen = torch.Generator().manual_seed(0)
    r = lambda *s: torch.randn(*s, generator=gen).cuda().requires_grad_()  # noqa: E731
    B, L, D = 2, 37, 16
    x, h = r(B, L, D), r(B, L, 2, 16)
    A = (-torch.rand(D, 8, generator=gen)).cuda()
    return {
        "gated_recurrence": ([x, r(B, L, D), r(D)], lambda x, g, d: ssm.gated_recurrence(x, g, None, d)),
        "causal_conv": ([x, r(D, 4)], lambda x, w: ssm.causal_conv(x, w)),
        "head_norm_rotary": ([h, r(B, L, 2, 16)], lambda q, k: ssm.head_norm_rotary(q, k)),
        "decay_attention": ([h, r(B, L, 2, 16), r(B, L, 2, 16)], lambda q, k, v: ssm.decay_attention(q, k, v, torch.full((2,), -0.1, device="cuda"))),
        "residual_norm": ([x, r(B, L, D), r(D)], lambda x, s, w: ssm.residual_norm(x, s, w)),
        "gated_norm": ([x, r(B, L, D), r(D)], lambda x, z, w: (ssm.gated_norm(x, z, w),)),
        "selective_scan": ([x, r(B, L, D), r(B, L, 8), r(B, L, 8)], lambda u, d, b, c: ssm.selective_scan(u, d, A, b, c)),
        "conv_selective_scan": ([x, r(D, 4), r(D), r(B, L, D), r(B, L, 8), r(B, L, 8)],
                                lambda u, w, b, d, p, c: ssm.conv_selective_scan(u, w, b, d, A, p, c)),
    }


@pytest.mark.gpu
@pytest.mark.parametrize("name", ["gated_recurrence", "causal_conv", "head_norm_rotary", "decay_attention", "residual_norm", "gated_norm",
                                  "selective_scan", "conv_selective_scan"])
def test_outputs_joined_behind_an_odd_element(name):
    """The gradients are those of the outputs weighted one by one."""
    import selective_state_space_10_amd as ssm
    inputs, f = _operators(ssm)[name]
    out = f(*inputs)
    weights = [torch.randn(t.shape, generator=torch.Generator().manual_seed(i)).cuda() for i, t in enumerate(out)]
    want = torch.autograd.grad(sum((t * w).sum() for t, w in zip(out, weights)), inputs, retain_graph=True)
    one = torch.zeros(1, device="cuda")
    joined = torch.cat([one] + [t.flatten() for t in out])
    got = torch.autograd.grad((joined * torch.cat([one] + [w.flatten() for w in weights])).sum(), inputs)
    for a, b in zip(got, want):
        torch.testing.assert_close(a, b)

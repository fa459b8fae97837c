"""Torch-facing wrappers of the C ABI (``include/ssm_block.h``) of the gated
recurrence, the causal convolution, and the norm and rotation of heads.  Shape,
dtype, stride and device checks, ``torch.empty`` for outputs and workspaces, and
the call on the current stream; nothing here computes.
"""
from __future__ import annotations

import torch
from torch.autograd.function import once_differentiable
from torch.autograd.graph import increment_version

from . import _lib
from .block_ops import _call, _gpu, _view, _want, _want_or_none, _workspace
from .ops import _gradient, _io_code, _ptr

_F32 = torch.float32
_View3 = _lib.View3
_CHUNK = _lib.RECURRENCE_CHUNK


def _view3(name, t, shape, dtype, dev):
    """A (batch, [step,] channel) tensor as an ssm_view3: any strides that keep
    16-byte alignment, with adjacent channels."""
    # (the usual tensor first: these calls are most of a small call's time)
    if (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.is_contiguous()
            and t.device == dev and not shape[-1] % 8):
        ptr = t.data_ptr()
        if not ptr % 16:
            d = shape[-1]
            return _View3(ptr, d * shape[1], d) if len(shape) == 3 else _View3(ptr, d, 0)
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor, got {type(t).__name__}")
    if t.device != dev:
        raise ValueError(f"{name} is on {t.device}, expected {dev}")
    if t.dtype is not dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.stride(-1) != 1 and shape[-1] != 1:
        raise ValueError(f"{name} must have adjacent channels (strides {t.stride()})")
    # strides of dimensions of size 1 are not used
    sb = t.stride(0) if shape[0] > 1 else 0
    st = t.stride(1) if len(shape) == 3 and shape[1] > 1 else 0
    ptr = t.data_ptr()
    if (sb | st) % (4 if dtype is _F32 else 8) or ptr % 16:
        raise ValueError(f"{name} must keep 16-byte alignment from row to row (strides "
                         f"{t.stride()}, address {ptr:#x}); make it contiguous")
    return _View3(ptr, sb, st)


def _view3_or_none(name, t, shape, dtype, dev):
    return None if t is None else _view3(name, t, shape, dtype, dev)


def _seq(x, rank):
    dev = _gpu("x", x)
    if x.dim() != rank:
        raise ValueError("x must be a " + ("(batch, seqlen, dim)" if rank == 3 else "(batch, dim)") + " tensor")
    return dev, _io_code(x), x.shape


def _marks(starts, lengths, B, L, dev):
    """The document starts and the rows' lengths, as pointers."""
    _want_or_none("starts", starts, (B, L), torch.bool, dev)
    _want_or_none("lengths", lengths, (B,), torch.int32, dev)
    return _ptr(starts), _ptr(lengths)


def _recurrence(x, decay_gate, input_gate, decay, z, rank):
    dev, io, shape = _seq(x, rank)
    views = (_view3("x", x, shape, x.dtype, dev), _view3("decay_gate", decay_gate, shape, x.dtype, dev),
             _view3_or_none("input_gate", input_gate, shape, x.dtype, dev),
             _view3_or_none("z", z, shape, x.dtype, dev))
    _want_or_none("decay", decay, (shape[-1],), _F32, dev)
    return dev, io, shape, views


def gated_recurrence_fwd(x, decay_gate, input_gate=None, decay=None, z=None, state0=None, starts=None,
                         lengths=None, sharpness=8.0, return_final_state=False, save_states=False):
    """A recurrence of one number per channel with gates for its decay and its input:
    h_t = a_t h_{t-1} + s_t sigmoid(input_gate_t) x_t, y_t = h_t (silu(z_t)).

    With ``decay`` (dim,) fp32, a = exp(-sharpness softplus(decay) sigmoid(decay_gate))
    and s = sqrt(1 - a^2); without, a = sigmoid(decay_gate) and s = 1 - a.
    x, decay_gate, input_gate, z (batch, seqlen, dim), strided views allowed; state0
    (batch, dim) fp32; ``starts`` (batch, seqlen) bool marks the first step of a
    document: there a = 0 and so s = 1, in both forms and whatever the gate holds: nothing
    crosses it, and its input counts in full.  A first step without a mark has the gate's s;
    a document is the same in a packed row and in a row of its own if its first step is
    marked in both.  ``lengths`` (batch,) int32 are the rows' lengths
    in a padded batch: behind them inputs are not used, y is zero, and the
    state stays.  Returns (y, final state or None, states or None): states
    (batch, ceil(seqlen / 128), dim), before every 128th step, are what the backward needs."""
    dev, io, (B, L, D), views = _recurrence(x, decay_gate, input_gate, decay, z, 3)
    _want_or_none("state0", state0, (B, D), _F32, dev)
    marks = _marks(starts, lengths, B, L, dev)
    lib = _lib.load()
    nbytes = lib.ssm_gated_recurrence_fwd_workspace_bytes(B, L, D, io)
    ws = _workspace(nbytes, dev)
    y = torch.empty_like(x, memory_format=torch.contiguous_format)
    final = torch.empty((B, D), dtype=_F32, device=dev) if return_final_state else None
    states = torch.empty((B, -(-L // _CHUNK), D), dtype=_F32, device=dev) if save_states else None
    _call(lib.ssm_gated_recurrence_fwd, dev, B, L, D, io, *views, _ptr(decay), sharpness, _ptr(state0),
          *marks, y.data_ptr(), _ptr(final), _ptr(states), _ptr(ws), nbytes)
    return y, final, states


def gated_recurrence_bwd(dy, x, decay_gate, input_gate, decay, z, states, starts=None, lengths=None,
                         sharpness=8.0, dstate_final=None, want_dstate0=True):
    """Gradients of gated_recurrence_fwd given dy and (optionally) dstate_final, and the
    states that it kept.  Returns a dict: dx, ddecay_gate, dinput_gate, ddecay, dz, dstate0
    (None where their input is None or they are not wanted)."""
    dev, io, (B, L, D), views = _recurrence(x, decay_gate, input_gate, decay, z, 3)
    dyv = _view3("dy", dy, (B, L, D), x.dtype, dev)
    _want("states", states, (B, -(-L // _CHUNK), D), _F32, dev)
    _want_or_none("dstate_final", dstate_final, (B, D), _F32, dev)
    marks = _marks(starts, lengths, B, L, dev)
    lib = _lib.load()
    nbytes = lib.ssm_gated_recurrence_bwd_workspace_bytes(B, L, D, io)
    ws = _workspace(nbytes, dev)
    like = lambda t: None if t is None else torch.empty((B, L, D), dtype=x.dtype, device=dev)  # noqa: E731
    g = dict(dx=like(x), ddecay_gate=like(x), dinput_gate=like(input_gate),
             ddecay=None if decay is None else torch.empty_like(decay), dz=like(z),
             dstate0=torch.empty((B, D), dtype=_F32, device=dev) if want_dstate0 else None)
    _call(lib.ssm_gated_recurrence_bwd, dev, B, L, D, io, dyv, *views, _ptr(decay), sharpness,
          states.data_ptr(), *marks, _ptr(dstate_final), g["dx"].data_ptr(), g["ddecay_gate"].data_ptr(),
          _ptr(g["dinput_gate"]), _ptr(g["dz"]), _ptr(g["ddecay"]), _ptr(g["dstate0"]), _ptr(ws), nbytes)
    return g


def gated_recurrence_update(state, x, decay_gate, input_gate=None, decay=None, z=None, sharpness=8.0):
    """One token of gated_recurrence_fwd; ``state`` (batch, dim) fp32 is updated in
    place.  x, decay_gate, input_gate, z (batch, dim).  Returns y.  It goes on in a document:
    the first token of one is a gated_recurrence_fwd of one marked step."""
    dev, io, (B, D), views = _recurrence(x, decay_gate, input_gate, decay, z, 2)
    _want("state", state, (B, D), _F32, dev)
    y = torch.empty_like(x, memory_format=torch.contiguous_format)
    _call(_lib.load().ssm_gated_recurrence_update, dev, B, D, io, state.data_ptr(), *views, _ptr(decay),
          sharpness, y.data_ptr())
    increment_version(state)  # a backward that saved it must not read it
    return y


def _conv_sizes(x, weight, bias, rank):
    dev, io, shape = _seq(x, rank)
    if not isinstance(weight, torch.Tensor) or weight.dim() != 2:
        raise ValueError("weight must be a (dim, width) tensor")
    K = weight.shape[1]
    if not 1 <= K <= 4:
        raise ValueError(f"convolution width {K} not in 1..4")
    _want("weight", weight, (shape[-1], K), _F32, dev)
    _want_or_none("bias", bias, (shape[-1],), _F32, dev)
    return dev, io, shape, K


def _held(t, K):
    """The pointer of a convolution's state; one of width 1 has none."""
    return None if t is None or K == 1 else t.data_ptr()


def causal_conv_fwd(x, weight, bias=None, state0=None, starts=None, lengths=None, silu=True,
                    return_final_state=False):
    """The causal depthwise convolution in front of a mixing:
    y_t = silu(bias + sum_k weight[:, k] x_{t - (width - 1) + k}), or without silu.

    x (batch, seqlen, dim), a strided view allowed; weight (dim, width) fp32, width 1
    to 4; bias (dim,) fp32; state0 (batch, width - 1, dim) in x's dtype, the inputs
    before the first; starts and lengths as of gated_recurrence_fwd.  Returns (y, final
    state or None): the last width - 1 inputs of each row's last document."""
    dev, io, (B, L, D), K = _conv_sizes(x, weight, bias, 3)
    xv = _view3("x", x, (B, L, D), x.dtype, dev)
    _want_or_none("state0", state0, (B, K - 1, D), x.dtype, dev)
    marks = _marks(starts, lengths, B, L, dev)
    y = torch.empty_like(x, memory_format=torch.contiguous_format)
    final = torch.empty((B, K - 1, D), dtype=x.dtype, device=dev) if return_final_state else None
    _call(_lib.load().ssm_causal_conv_fwd, dev, B, L, D, K, io, xv, weight.data_ptr(), _ptr(bias),
          _held(state0, K), *marks, int(bool(silu)), y.data_ptr(), _held(final, K))
    return y, final


def causal_conv_bwd(dy, x, weight, bias=None, state0=None, starts=None, lengths=None, silu=True,
                    dstate_final=None):
    """Gradients of causal_conv_fwd given dy and (optionally) dstate_final.  Returns a
    dict: dx, dweight, dbias and dstate0 (None without bias and state0)."""
    dev, io, (B, L, D), K = _conv_sizes(x, weight, bias, 3)
    xv, dyv = _view3("x", x, (B, L, D), x.dtype, dev), _view3("dy", dy, (B, L, D), x.dtype, dev)
    _want_or_none("state0", state0, (B, K - 1, D), x.dtype, dev)
    _want_or_none("dstate_final", dstate_final, (B, K - 1, D), x.dtype, dev)
    marks = _marks(starts, lengths, B, L, dev)
    lib = _lib.load()
    nbytes = lib.ssm_causal_conv_bwd_workspace_bytes(B, L, D, K)
    ws = _workspace(nbytes, dev)
    g = dict(dx=torch.empty((B, L, D), dtype=x.dtype, device=dev), dweight=torch.empty_like(weight),
             dbias=None if bias is None else torch.empty_like(bias),
             dstate0=None if state0 is None else torch.empty_like(state0))
    _call(lib.ssm_causal_conv_bwd, dev, B, L, D, K, io, dyv, xv, weight.data_ptr(), _ptr(bias),
          _held(state0, K), *marks, int(bool(silu)), _held(dstate_final, K), g["dx"].data_ptr(),
          g["dweight"].data_ptr(), _ptr(g["dbias"]), _held(g["dstate0"], K), _ptr(ws), nbytes)
    return g


def causal_conv_update(state, x, weight, bias=None, silu=True):
    """One token of causal_conv_fwd; ``state`` (batch, width - 1, dim) in x's dtype moves
    on by one input, in place.  x (batch, dim).  Returns y."""
    dev, io, (B, D), K = _conv_sizes(x, weight, bias, 2)
    xv = _view3("x", x, (B, D), x.dtype, dev)
    _want("state", state, (B, K - 1, D), x.dtype, dev)
    y = torch.empty_like(x, memory_format=torch.contiguous_format)
    _call(_lib.load().ssm_causal_conv_update, dev, B, D, K, io, _held(state, K), xv, weight.data_ptr(),
          _ptr(bias), int(bool(silu)), y.data_ptr())
    increment_version(state)
    return y


def _heads(q, k, q_weight, k_weight, positions, inv_freq, norm):
    dev = _gpu("q", q)
    if q.dim() not in (3, 4):
        raise ValueError("q must be a (batch, seqlen, heads, dim) or (batch, heads, dim) tensor")
    io, lead, d = _io_code(q), q.shape[:-2], q.shape[-1]
    Hq, Hk = q.shape[-2], 0
    if k is not None:
        if not isinstance(k, torch.Tensor) or k.dim() != q.dim():
            raise ValueError("k must be a tensor of q's dimensions")
        Hk = k.shape[-2]
    views = _view("q", q, q.shape, q.dtype, dev), _view("k", k, (*lead, Hk, d), q.dtype, dev) if Hk else None
    per_head = 0
    if q_weight is not None:
        per_head = int(isinstance(q_weight, torch.Tensor) and q_weight.dim() == 2)
        _want("q_weight", q_weight, (Hq, d) if per_head else (d,), _F32, dev)
    if Hk and q_weight is not None:
        _want("k_weight", k_weight, (Hk, d) if per_head else (d,), _F32, dev)
    elif k_weight is not None:
        raise ValueError("k_weight is given without " + ("q_weight" if Hk else "k"))
    if not norm and q_weight is not None:
        raise ValueError("weights are given without a norm")
    rot, per_batch = 0, 0
    if (positions is None) != (inv_freq is None):
        raise ValueError("positions and inv_freq must be given both or neither")
    if positions is not None:
        per_batch = int(not (len(lead) == 2 and isinstance(positions, torch.Tensor) and positions.dim() == 1))
        _want("positions", positions, lead if per_batch else lead[1:], torch.int64, dev)
        if not isinstance(inv_freq, torch.Tensor) or inv_freq.dim() != 1:
            raise ValueError("inv_freq must be a (rotary / 2,) tensor")
        rot = 2 * inv_freq.shape[0]
        _want("inv_freq", inv_freq, (rot // 2,), torch.float64, dev)
        if not 0 < rot <= d or rot % 8:
            raise ValueError(f"inv_freq's {rot // 2} frequencies rotate {rot} elements of heads of {d}: "
                             "not a multiple of 8 up to the head's size")
    B, L = (lead[0], 1) if len(lead) == 1 else lead
    return dev, io, (B, L, Hq, Hk, d, rot), views, (_ptr(q_weight), _ptr(k_weight), per_head, _ptr(positions), per_batch,
                                                    _ptr(inv_freq))


def head_norm_rotary_fwd(q, k=None, q_weight=None, k_weight=None, positions=None, inv_freq=None,
                         eps=1e-6, norm=True, interleaved=False):
    """The RMS norm of every head of q and k and the rotation of its elements by
    position: n = x / rms(x) * weight, then pairs (n_i, n_j) turned by
    position * inv_freq[p], p = 0 .. rotary / 2.

    q (batch, seqlen, heads, dim) or, for single tokens, (batch, heads, dim); k the same
    with its own heads, or None; strided views allowed.  Weights (dim,), or (heads, dim)
    for both, fp32, None = 1; norm=False leaves the norm out.  positions int64, (batch,
    seqlen) or (seqlen,), for single tokens (batch,); inv_freq (rotary / 2,) fp64; without them
    nothing is rotated.  Pair p is (p, p + rotary / 2), or with interleaved (2p, 2p + 1).
    Every row is one by itself, those of padding too: for the weights' gradients they should be
    finite, since 0 times what they hold is in the sum.
    Returns (q, k) normed and rotated, contiguous."""
    dev, io, sizes, views, rest = _heads(q, k, q_weight, k_weight, positions, inv_freq, norm)
    q_out = torch.empty_like(q, memory_format=torch.contiguous_format)
    k_out = None if k is None else torch.empty_like(k, memory_format=torch.contiguous_format)
    _call(_lib.load().ssm_head_norm_rotary_fwd, dev, *sizes, io, *views, *rest, eps, int(bool(norm)),
          int(bool(interleaved)), q_out.data_ptr(), _ptr(k_out) if sizes[3] else None)
    return q_out, k_out


def head_norm_rotary_bwd(dq_out, dk_out, q, k=None, q_weight=None, k_weight=None, positions=None,
                         inv_freq=None, eps=1e-6, norm=True, interleaved=False):
    """Gradients of head_norm_rotary_fwd given those of its outputs.  Returns a dict:
    dq, dk, dq_weight, dk_weight (None without their inputs)."""
    dev, io, sizes, views, rest = _heads(q, k, q_weight, k_weight, positions, inv_freq, norm)
    B, L, Hq, Hk, d, _ = sizes
    up = (_view("dq_out", dq_out, q.shape, q.dtype, dev), _view("dk_out", dk_out, k.shape, q.dtype, dev) if Hk else None)
    lib = _lib.load()
    nbytes = lib.ssm_head_norm_rotary_bwd_workspace_bytes(B, L, Hq, Hk, d) if q_weight is not None else 0
    ws = _workspace(nbytes, dev)
    like = lambda t: None if t is None else torch.empty_like(t, memory_format=torch.contiguous_format)  # noqa: E731
    g = dict(dq=like(q), dk=like(k), dq_weight=like(q_weight), dk_weight=like(k_weight))
    _call(lib.ssm_head_norm_rotary_bwd, dev, *sizes, io, *up, *views, *rest, eps, int(bool(norm)),
          int(bool(interleaved)), g["dq"].data_ptr(), _ptr(g["dk"]) if Hk else None, _ptr(g["dq_weight"]),
          _ptr(g["dk_weight"]), _ptr(ws), nbytes)
    return g


def _cotangent(dy, like):
    shape, dtype, dev = like
    return torch.zeros(shape, dtype=dtype, device=dev) if dy is None else _gradient(dy)


class GatedRecurrenceFn(torch.autograd.Function):
    """Autograd wrapper of the gated recurrence."""

    @staticmethod
    def forward(ctx, x, decay_gate, input_gate=None, decay=None, z=None, state0=None, starts=None,
                lengths=None, sharpness=8.0):
        y, final, states = gated_recurrence_fwd(x, decay_gate, input_gate, decay, z, state0, starts, lengths,
                                                sharpness, return_final_state=True,
                                                save_states=any(ctx.needs_input_grad))
        ctx.sharpness = sharpness
        ctx.set_materialize_grads(False)
        ctx.save_for_backward(x, decay_gate, input_gate, decay, z, states, starts, lengths)
        return y, final

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, dfinal):
        x, decay_gate, input_gate, decay, z, states, starts, lengths = ctx.saved_tensors
        # (a slice: apply() may have been given fewer arguments)
        g = gated_recurrence_bwd(_cotangent(dy, (x.shape, x.dtype, x.device)), x, decay_gate, input_gate, decay, z,
                                 states, starts, lengths, ctx.sharpness, _gradient(dfinal),
                                 want_dstate0=any(ctx.needs_input_grad[5:6]))
        return (g["dx"], g["ddecay_gate"], g["dinput_gate"], g["ddecay"], g["dz"], g["dstate0"], None, None, None)


def gated_recurrence(x, decay_gate, input_gate=None, decay=None, z=None, state0=None, starts=None, lengths=None,
                     sharpness=8.0):
    """Differentiable gated recurrence; returns (y, final state)."""
    return GatedRecurrenceFn.apply(x, decay_gate, input_gate, decay, z, state0, starts, lengths, sharpness)


class CausalConvFn(torch.autograd.Function):
    """Autograd wrapper of the causal convolution."""

    @staticmethod
    def forward(ctx, x, weight, bias=None, state0=None, starts=None, lengths=None, silu=True):
        y, final = causal_conv_fwd(x, weight, bias, state0, starts, lengths, silu, return_final_state=True)
        ctx.silu = silu
        ctx.set_materialize_grads(False)
        ctx.save_for_backward(x, weight, bias, state0, starts, lengths)
        return y, final

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, dfinal):
        x, weight, bias, state0, starts, lengths = ctx.saved_tensors
        g = causal_conv_bwd(_cotangent(dy, (x.shape, x.dtype, x.device)), x, weight, bias, state0, starts, lengths,
                            ctx.silu, _gradient(dfinal))
        return g["dx"], g["dweight"], g["dbias"], g["dstate0"], None, None, None


def causal_conv(x, weight, bias=None, state0=None, starts=None, lengths=None, silu=True):
    """Differentiable causal convolution; returns (y, final state)."""
    return CausalConvFn.apply(x, weight, bias, state0, starts, lengths, silu)


class HeadNormRotaryFn(torch.autograd.Function):
    """Autograd wrapper of the norm and rotation of heads."""

    @staticmethod
    def forward(ctx, q, k, q_weight, k_weight, positions, inv_freq, eps, norm, interleaved):
        q_out, k_out = head_norm_rotary_fwd(q, k, q_weight, k_weight, positions, inv_freq, eps, norm, interleaved)
        ctx.options = (eps, norm, interleaved)
        ctx.set_materialize_grads(False)
        ctx.save_for_backward(q, k, q_weight, k_weight, positions, inv_freq)
        return q_out, k_out

    @staticmethod
    @once_differentiable
    def backward(ctx, dq_out, dk_out):
        q, k = ctx.saved_tensors[:2]
        g = head_norm_rotary_bwd(_cotangent(dq_out, (q.shape, q.dtype, q.device)),
                                 None if k is None else _cotangent(dk_out, (k.shape, k.dtype, k.device)),
                                 *ctx.saved_tensors, *ctx.options)
        return g["dq"], g["dk"], g["dq_weight"], g["dk_weight"], None, None, None, None, None


def head_norm_rotary(q, k=None, q_weight=None, k_weight=None, positions=None, inv_freq=None, eps=1e-6, norm=True,
                     interleaved=False):
    """Differentiable norm and rotation of heads; returns (q, k)."""
    return HeadNormRotaryFn.apply(q, k, q_weight, k_weight, positions, inv_freq, eps, norm, interleaved)

"""Torch-facing wrappers of the block operators' C ABI (``include/ssm_block.h``):
decay attention (linear attention with a decay for each head), the norm before
a block with its residual sum, and the norm after a block's mixing with its
gate.  Shape, dtype, stride and device checks, ``torch.empty`` for outputs and
workspaces, and the call on the current stream; nothing here computes.
"""
from __future__ import annotations

import torch
from torch.autograd.function import once_differentiable
from torch.autograd.graph import increment_version

from . import _lib
from .ops import _IO, _io_code, _need, _ptr, _stream

_F32 = torch.float32
_View4 = _lib.View4


def _view(name, t, shape, dtype, dev):
    """A (batch, [step,] head, element) tensor as an ssm_view4: any strides that
    keep 16-byte alignment, with the elements of a head adjacent."""
    # (the usual tensor first: these calls are most of a small call's time)
    if (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.is_contiguous()
            and t.device == dev and not shape[-1] % 8):
        ptr = t.data_ptr()
        if not ptr % 16:
            st = shape[-1] * shape[-2]
            return _View4(ptr, st * shape[1] if len(shape) == 4 else st, st, shape[-1])
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor, got {type(t).__name__}")
    if t.device != dev:
        raise ValueError(f"{name} is on {t.device}, expected {dev}")
    if t.dtype is not dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    ptr = t.data_ptr()
    if len(shape) == 4:
        sb, st, sh, se = t.stride()
    else:
        sb, sh, se = t.stride()
        st = 0
    if se != 1 and shape[-1] != 1:
        raise ValueError(f"{name} must have adjacent elements in its last dimension "
                         f"(strides {t.stride()})")
    # strides of dimensions of size 1 are not used
    sb, sh = sb if shape[0] > 1 else 0, sh if shape[-2] > 1 else 0
    if len(shape) == 4 and shape[1] == 1:
        st = 0
    if (sb | st | sh) % (4 if dtype is _F32 else 8) or ptr % 16:
        raise ValueError(f"{name} must keep 16-byte alignment from head to head (strides "
                         f"{t.stride()}, address {ptr:#x}); make it contiguous")
    return _View4(ptr, sb, st, sh)


# what torch.cuda.current_stream and current_device ask, without their wrappers
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _call(fn, dev, *args):
    """fn(*args, current stream) with dev as the current device."""
    index = dev.index
    if _raw_stream is not None and index == _current_device():
        st = fn(*args, _raw_stream(index))
    else:
        with torch.cuda.device(dev):
            st = fn(*args, _stream(dev))
    if st:
        _lib.check(st)


def _is(t, shape, dtype, dev):
    return (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape
            and t.is_contiguous() and t.device == dev)


def _want(name, t, shape, dtype, dev):
    if not _is(t, shape, dtype, dev):
        _need(name, t, shape, dtype, dev)  # says what is wrong


def _want_or_none(name, t, shape, dtype, dev):
    if t is not None and not _is(t, shape, dtype, dev):
        _need(name, t, shape, dtype, dev)


def _gpu(name, t):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor, got {type(t).__name__}")
    if t.device.type != "cuda":
        raise ValueError(f"tensors must be on a GPU device, got {t.device}")
    return t.device


def _workspace(nbytes, dev):
    if nbytes < 0:
        raise ValueError("invalid sizes: " + _lib.load().ssm_last_error().decode())
    return torch.empty(nbytes, dtype=torch.uint8, device=dev) if nbytes else None


def _attn_sizes(q, v, rank):
    dev = _gpu("q", q)
    lead = "batch, seqlen" if rank == 4 else "batch"
    if q.dim() != rank:
        raise ValueError(f"q must be a ({lead}, key_heads, dk) tensor")
    if not isinstance(v, torch.Tensor) or v.dim() != rank:
        raise ValueError(f"v must be a ({lead}, heads, dv) tensor")
    _io_code(q)
    G, H = q.shape[-2], v.shape[-2]
    if G < 1 or H % max(G, 1):
        raise ValueError(f"v's {H} heads are not a multiple of q's {G}")
    return dev, G, H, q.shape[-1], v.shape[-1]


def _per_token(log_decay, shape, dev):
    """shape: of one decay per token and head."""
    if _is(log_decay, shape, _F32, dev):
        return 1
    per_token = isinstance(log_decay, torch.Tensor) and log_decay.dim() != 1
    _need("log_decay", log_decay, shape if per_token else shape[-1:], _F32, dev)
    return int(per_token)


def decay_attn_fwd(q, k, v, log_decay, scale=None, state0=None, return_final_state=False):
    """Linear attention with a decay for each head over whole sequences:
    S_t = exp(g_t) S_{t-1} + k_t v_t^T, o_t = scale S_t^T q_t.

    q, k (batch, seqlen, key_heads, dk); v (batch, seqlen, heads, dv), head h
    using key head h // (heads // key_heads); log_decay g (batch, seqlen,
    heads) or (heads,) fp32, -inf clears the state; scale defaults to
    dk ** -0.5; state0 (batch, heads, dk, dv) fp32.  q, k and v may be strided
    views.  Returns (o, final state or None)."""
    dev, G, H, dk, dv = _attn_sizes(q, v, 4)
    B, L = q.shape[:2]
    io, dt = _io_code(q), q.dtype
    qv, kv = _view("q", q, (B, L, G, dk), dt, dev), _view("k", k, (B, L, G, dk), dt, dev)
    vv = _view("v", v, (B, L, H, dv), dt, dev)
    per_token = _per_token(log_decay, (B, L, H), dev)
    _want_or_none("state0", state0, (B, H, dk, dv), _F32, dev)
    lib = _lib.load()
    nbytes = lib.ssm_decay_attn_fwd_workspace_bytes(B, L, H, G, dk, dv, io)
    ws = _workspace(nbytes, dev)
    o = torch.empty_like(v, memory_format=torch.contiguous_format)
    final = torch.empty((B, H, dk, dv), dtype=_F32, device=dev) if return_final_state else None
    _call(lib.ssm_decay_attn_fwd, dev, B, L, H, G, dk, dv, io, qv, kv, vv, log_decay.data_ptr(),
          per_token, dk ** -0.5 if scale is None else scale,
          _ptr(state0), _ptr(final), o.data_ptr(), _ptr(ws), nbytes)
    return o, final


def decay_attn_bwd(q, k, v, log_decay, do, scale=None, state0=None, dstate_final=None,
                   want_dlog_decay=True, want_dstate0=True):
    """Gradients of decay_attn_fwd, given do and (optionally) dstate_final.
    Returns a dict: dq, dk, dv, dlog_decay (log_decay's shape), dstate0.  dq and
    dk with and without dlog_decay are equal to fp32's rounding, not to the bit."""
    dev, G, H, dk, dv = _attn_sizes(q, v, 4)
    B, L = q.shape[:2]
    io, dt = _io_code(q), q.dtype
    qv, kv = _view("q", q, (B, L, G, dk), dt, dev), _view("k", k, (B, L, G, dk), dt, dev)
    vv, ov = _view("v", v, (B, L, H, dv), dt, dev), _view("do", do, (B, L, H, dv), dt, dev)
    per_token = _per_token(log_decay, (B, L, H), dev)
    _want_or_none("state0", state0, (B, H, dk, dv), _F32, dev)
    _want_or_none("dstate_final", dstate_final, (B, H, dk, dv), _F32, dev)
    lib = _lib.load()
    nbytes = lib.ssm_decay_attn_bwd_workspace_bytes(B, L, H, G, dk, dv, io)
    ws = _workspace(nbytes, dev)
    g = dict(dq=torch.empty((B, L, G, dk), dtype=dt, device=dev),
             dk=torch.empty((B, L, G, dk), dtype=dt, device=dev),
             dv=torch.empty((B, L, H, dv), dtype=dt, device=dev),
             dlog_decay=torch.empty_like(log_decay) if want_dlog_decay else None,
             dstate0=torch.empty((B, H, dk, dv), dtype=_F32, device=dev) if want_dstate0 else None)
    _call(lib.ssm_decay_attn_bwd, dev, B, L, H, G, dk, dv, io, qv, kv, vv, log_decay.data_ptr(),
          per_token, dk ** -0.5 if scale is None else scale,
          _ptr(state0), ov, _ptr(dstate_final), _ptr(g["dq"]),
          _ptr(g["dk"]), _ptr(g["dv"]), _ptr(g["dlog_decay"]),
          _ptr(g["dstate0"]), _ptr(ws), nbytes)
    return g


def decay_attn_update(state, q, k, v, log_decay, scale=None):
    """One token of decay_attn_fwd; ``state`` (batch, heads, dk, dv) fp32 is
    updated in place.  q, k (batch, key_heads, dk); v (batch, heads, dv);
    log_decay (batch, heads) or (heads,).  Returns o (batch, heads, dv)."""
    dev, G, H, dk, dv = _attn_sizes(q, v, 3)
    B = q.shape[0]
    io, dt = _io_code(q), q.dtype
    _want("state", state, (B, H, dk, dv), _F32, dev)
    qv, kv = _view("q", q, (B, G, dk), dt, dev), _view("k", k, (B, G, dk), dt, dev)
    vv = _view("v", v, (B, H, dv), dt, dev)
    per_token = _per_token(log_decay, (B, H), dev)
    o = torch.empty_like(v, memory_format=torch.contiguous_format)
    _call(_lib.load().ssm_decay_attn_update, dev, B, H, G, dk, dv, io, state.data_ptr(), qv, kv, vv,
          log_decay.data_ptr(), per_token,
          dk ** -0.5 if scale is None else scale,
          o.data_ptr())
    increment_version(state)  # a backward that saved it must not read it
    return o


def _rows(name, t, shape, dtype, dev):
    """(pointer, elements from row to row) of a tensor whose rows are evenly
    spaced: contiguous, or a slice of one along its last dimension."""
    if _is(t, shape, dtype, dev):
        return t.data_ptr(), shape[-1]
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor, got {type(t).__name__}")
    if t.device != dev:
        raise ValueError(f"{name} is on {t.device}, expected {dev}")
    if t.dtype != dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    step, span = None, None
    for n, s in zip(reversed(shape[:-1]), reversed(t.stride()[:-1])):
        if n == 1:
            continue
        if step is None:
            step, span = s, s * n
        elif s != span:
            raise ValueError(f"{name}'s rows are not evenly spaced (strides {t.stride()}); make it contiguous")
        else:
            span = s * n
    step = shape[-1] if step is None else step
    if t.stride(-1) != 1 or step % (4 if dtype is _F32 else 8) or t.data_ptr() % 16:
        raise ValueError(f"{name} must have adjacent elements and 16-byte aligned rows "
                         f"(strides {t.stride()}); make it contiguous")
    return t.data_ptr(), step


def _norm_input(x):
    dev = _gpu("x", x)
    if x.dim() < 1:
        raise ValueError("x must have at least one dimension")
    D = x.shape[-1]
    return dev, _io_code(x), D, x.numel() // max(D, 1)


def _residual_code(residual, x):
    if not isinstance(residual, torch.Tensor):
        raise TypeError(f"the residual must be a torch.Tensor, got {type(residual).__name__}")
    if residual.dtype not in (x.dtype, _F32):
        raise TypeError(f"the residual has dtype {residual.dtype}, expected {x.dtype} or float32")
    return _IO[residual.dtype]


def residual_norm_fwd(x, residual, weight, scale=None, eps=1e-5):
    """The norm before a block: h = residual + scale * x, y = h / rms(h) * weight.

    x (..., dim); residual of the same shape, in x's dtype or fp32; weight and
    scale (dim,) fp32 (scale None = 1).  x may be a slice along the last
    dimension.  Returns (y, h, rstd): h in residual's dtype, rstd (...) fp32."""
    dev, io, D, rows = _norm_input(x)
    xp, xs = _rows("x", x, x.shape, x.dtype, dev)
    ro = _residual_code(residual, x)
    _want("residual", residual, x.shape, residual.dtype, dev)
    _want("weight", weight, (D,), _F32, dev)
    _want_or_none("scale", scale, (D,), _F32, dev)
    y = torch.empty_like(x, memory_format=torch.contiguous_format)
    h = torch.empty_like(residual)
    rstd = torch.empty(x.shape[:-1], dtype=_F32, device=dev)
    _call(_lib.load().ssm_residual_norm_fwd, dev, rows, D, io, ro, xp, xs, residual.data_ptr(),
          weight.data_ptr(), _ptr(scale), eps, y.data_ptr(),
          h.data_ptr(), rstd.data_ptr())
    return y, h, rstd


def residual_norm_bwd(dy, dh, h, rstd, weight, x=None, scale=None):
    """Gradients of residual_norm_fwd given dy and dh (the gradient that reaches
    h by the residual stream; None = 0).  Returns a dict: dx, dresidual (the
    same tensor as dx where they are equal), dweight, dscale (needs x)."""
    dev, io, D, rows = _norm_input(dy)
    ro = _residual_code(h, dy)
    _want("dy", dy, dy.shape, dy.dtype, dev)
    _want("h", h, dy.shape, h.dtype, dev)
    _want_or_none("dh", dh, dy.shape, h.dtype, dev)
    _want("rstd", rstd, dy.shape[:-1], _F32, dev)
    _want("weight", weight, (D,), _F32, dev)
    _want_or_none("scale", scale, (D,), _F32, dev)
    xp, xs = (None, D) if x is None or scale is None else _rows("x", x, dy.shape, dy.dtype, dev)
    dres = torch.empty_like(h)
    same = scale is None and h.dtype == dy.dtype
    dx = dres if same else torch.empty_like(dy)
    dw = torch.empty_like(weight)
    dscale = torch.empty_like(scale) if xp is not None else None
    lib = _lib.load()
    nbytes = lib.ssm_residual_norm_bwd_workspace_bytes(rows, D)
    ws = _workspace(nbytes, dev)
    _call(lib.ssm_residual_norm_bwd, dev, rows, D, io, ro, dy.data_ptr(), _ptr(dh), h.data_ptr(),
          rstd.data_ptr(), weight.data_ptr(), xp, xs, _ptr(scale),
          None if same else dx.data_ptr(), dres.data_ptr(),
          dw.data_ptr(), _ptr(dscale), ws.data_ptr(), nbytes)
    return dict(dx=dx, dresidual=dres, dweight=dw, dscale=dscale)


def gated_norm_fwd(x, z, weight, group=None, eps=1e-5, gate_first=False):
    """The norm after a block's mixing, over groups of ``group`` adjacent
    channels (default: all): y = x / rms(x) * weight * silu(z), or with
    gate_first, t = x * silu(z), y = t / rms(t) * weight.  z None = no gate.

    x, z (..., dim), slices along the last dimension allowed; weight (dim,)
    fp32.  Returns (y, rstd): rstd (..., dim // group) fp32."""
    dev, io, D, rows = _norm_input(x)
    group = D if group is None else int(group)
    xp, xs = _rows("x", x, x.shape, x.dtype, dev)
    zp, zs = (None, D) if z is None else _rows("z", z, x.shape, x.dtype, dev)
    _want("weight", weight, (D,), _F32, dev)
    if group < 1 or D % group:
        raise ValueError(f"{D} channels are not a multiple of group={group}")
    y = torch.empty_like(x, memory_format=torch.contiguous_format)
    rstd = torch.empty((*x.shape[:-1], D // group), dtype=_F32, device=dev)
    _call(_lib.load().ssm_gated_norm_fwd, dev, rows, D, group, io, xp, xs, zp, zs, weight.data_ptr(),
          eps, int(bool(gate_first)), y.data_ptr(),
          rstd.data_ptr())
    return y, rstd


def gated_norm_bwd(dy, x, z, weight, rstd, group=None, gate_first=False):
    """Gradients of gated_norm_fwd.  Returns a dict: dx, dz (None without z), dweight."""
    dev, io, D, rows = _norm_input(x)
    group = D if group is None else int(group)
    xp, xs = _rows("x", x, x.shape, x.dtype, dev)
    zp, zs = (None, D) if z is None else _rows("z", z, x.shape, x.dtype, dev)
    _want("dy", dy, x.shape, x.dtype, dev)
    _want("weight", weight, (D,), _F32, dev)
    if group < 1 or D % group:
        raise ValueError(f"{D} channels are not a multiple of group={group}")
    _want("rstd", rstd, (*x.shape[:-1], D // group), _F32, dev)
    dx = torch.empty(x.shape, dtype=x.dtype, device=dev)
    dz = torch.empty(x.shape, dtype=x.dtype, device=dev) if z is not None else None
    dw = torch.empty_like(weight)
    lib = _lib.load()
    nbytes = lib.ssm_gated_norm_bwd_workspace_bytes(rows, D, group)
    ws = _workspace(nbytes, dev)
    _call(lib.ssm_gated_norm_bwd, dev, rows, D, group, io, dy.data_ptr(), xp, xs, zp, zs,
          weight.data_ptr(), rstd.data_ptr(), int(bool(gate_first)),
          dx.data_ptr(), _ptr(dz), dw.data_ptr(), ws.data_ptr(), nbytes)
    return dict(dx=dx, dz=dz, dweight=dw)


class DecayAttentionFn(torch.autograd.Function):
    """Autograd wrapper of decay attention; the backward recomputes the states."""

    @staticmethod
    def forward(ctx, q, k, v, log_decay, scale=None, state0=None):
        o, final = decay_attn_fwd(q, k, v, log_decay, scale, state0, return_final_state=True)
        ctx.scale = scale
        ctx.set_materialize_grads(False)
        ctx.save_for_backward(q, k, v, log_decay, state0)
        return o, final

    @staticmethod
    @once_differentiable
    def backward(ctx, do, dfinal):
        q, k, v, log_decay, state0 = ctx.saved_tensors
        do = torch.zeros(v.shape, dtype=v.dtype, device=v.device) if do is None else do.contiguous()
        g = decay_attn_bwd(q, k, v, log_decay, do, ctx.scale, state0,
                           None if dfinal is None else dfinal.contiguous(),
                           want_dlog_decay=ctx.needs_input_grad[3],
                           want_dstate0=ctx.needs_input_grad[5])
        return g["dq"], g["dk"], g["dv"], g["dlog_decay"], None, g["dstate0"]


def decay_attention(q, k, v, log_decay, scale=None, state0=None):
    """Differentiable decay attention; returns (o, final state)."""
    return DecayAttentionFn.apply(q, k, v, log_decay, scale, state0)


class ResidualNormFn(torch.autograd.Function):
    """Autograd wrapper of the norm before a block."""

    @staticmethod
    def forward(ctx, x, residual, weight, scale=None, eps=1e-5):
        y, h, rstd = residual_norm_fwd(x, residual, weight, scale, eps)
        ctx.set_materialize_grads(False)
        ctx.save_for_backward(x if scale is not None else None, h, rstd, weight, scale)
        ctx.x_like = (x.shape, x.dtype, x.device)
        return y, h

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, dh):
        x, h, rstd, weight, scale = ctx.saved_tensors
        shape, dtype, dev = ctx.x_like
        dy = torch.zeros(shape, dtype=dtype, device=dev) if dy is None else dy.contiguous()
        g = residual_norm_bwd(dy, None if dh is None else dh.contiguous(), h, rstd, weight, x, scale)
        return g["dx"], g["dresidual"], g["dweight"], g["dscale"], None


def residual_norm(x, residual, weight, scale=None, eps=1e-5):
    """Differentiable norm before a block; returns (y, h)."""
    return ResidualNormFn.apply(x, residual, weight, scale, eps)


class GatedNormFn(torch.autograd.Function):
    """Autograd wrapper of the norm after a block's mixing."""

    @staticmethod
    def forward(ctx, x, z, weight, group=None, eps=1e-5, gate_first=False):
        y, rstd = gated_norm_fwd(x, z, weight, group, eps, gate_first)
        ctx.group, ctx.gate_first = group, gate_first
        ctx.save_for_backward(x, z, weight, rstd)
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        x, z, weight, rstd = ctx.saved_tensors
        g = gated_norm_bwd(dy.contiguous(), x, z, weight, rstd, ctx.group, ctx.gate_first)
        return g["dx"], g["dz"], g["dweight"], None, None, None


def gated_norm(x, z, weight, group=None, eps=1e-5, gate_first=False):
    """Differentiable norm after a block's mixing; returns y."""
    return GatedNormFn.apply(x, z, weight, group, eps, gate_first)

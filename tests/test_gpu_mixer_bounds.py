"""Nothing is written next to an output, a state or a workspace of the gated recurrence,
the causal convolution and the norm and rotation of heads: every tensor that a call
allocates lies between guards, at sizes that end inside tiles, chunks and groups of lanes."""
from __future__ import annotations

import math

import pytest
import torch

from tests import mixer_reference as ref

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
GUARD = 1 << 16  # bytes on either side


@pytest.fixture(scope="module")
def ssm():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import selective_state_space_10_amd as m
    m.load()
    return m


@pytest.fixture
def guards(monkeypatch):
    made = []
    real = torch.empty

    def empty(*shape, dtype=torch.float32, device=None, **kw):
        shape = tuple(shape[0]) if len(shape) == 1 and not isinstance(shape[0], int) else shape
        n = math.prod(shape) * dtype.itemsize
        buf = real(n + 2 * GUARD, dtype=torch.uint8, device=device).fill_(0xA5)
        made.append((buf, n))
        return buf[GUARD:GUARD + n].view(dtype).view(shape)

    def empty_like(t, memory_format=None, **kw):
        return empty(tuple(t.shape), dtype=t.dtype, device=t.device)

    monkeypatch.setattr(torch, "empty", empty)
    monkeypatch.setattr(torch, "empty_like", empty_like)

    def check():
        torch.cuda.synchronize()
        assert made
        for buf, n in made:
            assert bool((buf[:GUARD] == 0xA5).all()) and bool((buf[GUARD + n:] == 0xA5).all()), n
        made.clear()
    return check


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("form", ["power", "logistic"])
@pytest.mark.parametrize("B,L,D", [(1, 1, 8), (2, 3, 72), (1, 17, 136), (2, 127, 64), (1, 129, 200), (3, 200, 40), (1, 300, 1000), (1, 2100, 24)])
@pytest.mark.parametrize("marks", [False, True])
def test_recurrence(ssm, guards, dtype, form, B, L, D, marks):
    print("recurrence", dtype, form, B, L, D, marks, flush=True)
    g = ref.on_gpu(ref.recurrence_inputs(B, L, D, form=form, dtype=dtype, starts=marks, lengths=marks))
    y, f, s = ssm.gated_recurrence_fwd(g["x"], g["decay_gate"], g["input_gate"], g["decay"], g["z"], g["state0"], g["starts"], g["lengths"],
                                       return_final_state=True, save_states=True)
    guards()
    ssm.gated_recurrence_bwd(g["dy"], g["x"], g["decay_gate"], g["input_gate"], g["decay"], g["z"], s, g["starts"], g["lengths"], dstate_final=g["dfinal"])
    guards()
    ssm.gated_recurrence_update(f, g["x"][:, 0].contiguous(), g["decay_gate"][:, 0].contiguous())
    guards()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("K", [1, 2, 3, 4])
@pytest.mark.parametrize("B,L,D", [(1, 1, 8), (2, 2, 72), (1, 17, 136), (2, 61, 64), (1, 62, 200), (3, 130, 520), (1, 300, 1000), (1, 2100, 24)])
def test_conv(ssm, guards, dtype, K, B, L, D):
    print("conv", dtype, K, B, L, D, flush=True)
    for marks in (False, True):
        g = ref.on_gpu(ref.conv_inputs(B, L, D, K, dtype=dtype, starts=marks, lengths=marks))
        ssm.causal_conv_fwd(g["x"], g["weight"], g["bias"], g["state0"], g["starts"], g["lengths"], return_final_state=True)
        guards()
        ssm.causal_conv_bwd(g["dy"], g["x"], g["weight"], g["bias"], g["state0"], g["starts"], g["lengths"], dstate_final=g["dfinal"])
        guards()
    state = torch.empty((B, K - 1, D), dtype=dtype, device="cuda").zero_()
    ssm.causal_conv_update(state, g["x"][:, 0].contiguous(), g["weight"], g["bias"])
    guards()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("weights", ["shared", "per head"])
@pytest.mark.parametrize("B,L,Hq,Hk,d,rot", [(1, 1, 1, 0, 8, 8), (2, 3, 3, 1, 72, 24), (1, 37, 17, 2, 40, 40), (3, 9, 5, 5, 128, 64), (1, 130, 2, 1, 256, 256)])
def test_heads(ssm, guards, dtype, weights, B, L, Hq, Hk, d, rot):
    print("heads", dtype, weights, B, L, Hq, Hk, d, rot, flush=True)
    g = ref.on_gpu(ref.head_inputs(B, L, Hq, Hk, d, rot, dtype=dtype, weights=weights))
    args = [g[n] for n in ("q", "k", "q_weight", "k_weight", "positions", "inv_freq")]
    ssm.head_norm_rotary_fwd(*args)
    guards()
    ssm.head_norm_rotary_bwd(g["dq_out"], g["dk_out"], *args)
    guards()


@pytest.mark.parametrize("weights", ["shared", "per head"])
@pytest.mark.parametrize("B,L,Hq,Hk,d,rot", [(1, 9000, 16, 16, 128, 128), (1, 9000, 20, 5, 80, 40), (1, 70000, 1, 0, 8, 8), (1, 300, 300, 20, 128, 64)])
def test_heads_with_all_workgroups(ssm, guards, weights, B, L, Hq, Hk, d, rot):
    """The workspace of as many workgroups as there are at most, and of blocks of heads beyond that."""
    print("heads", weights, B, L, Hq, Hk, d, rot, flush=True)
    g = ref.on_gpu(ref.head_inputs(B, L, Hq, Hk, d, rot, dtype=BF16, weights=weights))
    ssm.head_norm_rotary_bwd(g["dq_out"], g["dk_out"], *(g[n] for n in ("q", "k", "q_weight", "k_weight", "positions", "inv_freq")))
    guards()


@pytest.mark.parametrize("K,D,B,L,dtype", [(4, 65672, 2, 257, BF16), (3, 32776, 1, 1000, F32), (2, 2056, 8, 500, BF16)])
def test_conv_with_all_workgroups(ssm, guards, K, D, B, L, dtype):
    print("conv", K, D, B, L, dtype, flush=True)
    g = ref.on_gpu(ref.conv_inputs(B, L, D, K, dtype=dtype, starts=True, lengths=True))
    ssm.causal_conv_bwd(g["dy"], g["x"], g["weight"], g["bias"], g["state0"], g["starts"], g["lengths"], dstate_final=g["dfinal"])
    guards()

"""How the gated recurrence, the convolution and the heads are split over workgroups: the plans of the
sizes that the GPU tests of training sizes rest on, so that another rule cannot move those
tests off the paths that they are for.  And the convolution's reference at once against the one step by step."""
from __future__ import annotations

import pytest
import torch

from tests import mixer_plans as plans
from tests import mixer_reference as ref


@pytest.mark.parametrize("K", [1, 2, 4])
@pytest.mark.parametrize("silu", [True, False])
@pytest.mark.parametrize("seed", range(8))
def test_convolution_at_once(K, silu, seed):
    coin = lambda i: bool(seed >> i & 1)  # noqa: E731
    p = ref.conv_inputs(4, 1 + 7 * seed, 8, K, bias=coin(0), state0=coin(1), starts=coin(2), lengths=not coin(0), seed=seed)
    if p["starts"] is not None:
        p["starts"] = torch.rand(p["starts"].shape, generator=torch.Generator().manual_seed(seed)) < 0.3
    y, final, g = ref.conv_at_once(p, silu)
    y1, final1, g1 = ref.conv(p, silu)
    assert torch.allclose(y, y1) and torch.equal(final, final1) and g.keys() == g1.keys()
    assert all(torch.allclose(g[n], g1[n]) for n in g)


# B, L, D, width, bytes of an element: (more than 64 steps of a chunk, several chunks of a wave)
CONV = {(8, 2048, 2048, 4, 2): (True, False), (8, 2048, 2048, 4, 4): (True, False), (2, 257, 65672, 4, 2): (True, True),
        (3, 333, 32776, 4, 4): (True, True), (1, 1000, 32776, 3, 4): (True, True), (1, 700, 65672, 2, 2): (True, True)}


@pytest.mark.parametrize("sizes", CONV, ids=str)
def test_convolution_backward(sizes):
    p = plans.conv_backward(*sizes)
    assert (p["nrow"] > 64, sizes[0] * p["nchunk"] > 4 * p["nruns"]) == CONV[sizes], p


# B, L, D, bytes of an element: chunks per published state, fewer than the sequence has
RECURRENCE = {(8, 515, 2056, 2): 1, (2, 700, 4104, 2): 2, (3, 700, 2056, 2): 4, (2, 1100, 1000, 2): 8, (2, 2100, 520, 2): 16,
              (8, 700, 1000, 4): 1, (4, 700, 1000, 4): 2, (3, 1537, 1000, 4): 4, (2, 1537, 712, 4): 8}


@pytest.mark.parametrize("sizes", RECURRENCE, ids=str)
def test_recurrence(sizes):
    group = plans.recurrence_group(*sizes)
    assert group == RECURRENCE[sizes] and -(-sizes[1] // 128) > group


def test_recurrence_of_the_longest_rows():
    assert (plans.recurrence_group(3, 87500, 8192, 2), plans.recurrence_group(1, 87500, 8192, 2)) == (1, 2)


# B, L, q heads, k heads, dim, bytes of an element: several chunks of tokens per workgroup in the backward
HEADS = {(1, 9000, 16, 16, 128, 2), (3, 3000, 16, 16, 128, 4), (2, 4500, 32, 4, 64, 2), (1, 9000, 20, 5, 80, 4)}


@pytest.mark.parametrize("sizes", sorted(HEADS), ids=str)
def test_heads_backward(sizes):
    B, L, Hq, Hk, d, es = sizes
    p = plans.heads(1, B * L, Hq + Hk, d, d, 1, es)  # (contiguous rows of a batch follow each other as one)
    assert p["nchunk"] > 2 * p["nruns"], p

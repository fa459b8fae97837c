"""The example block: training and serving through the operators together."""
from __future__ import annotations

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,tol", [(torch.float32, 1e-4), (torch.bfloat16, 4e-2)])
def test_block(dtype, tol):
    """Serving differs from the prompt by rounding alone: fp32 products of width
    256 and 512 in another order; in bf16 the projections' roundings of 2^-8 go
    through a product of 512 terms."""
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from examples.decay_attention_block import run
    diff, losses = run(dtype=dtype)
    assert diff <= tol, diff
    assert losses[-1] < losses[0]

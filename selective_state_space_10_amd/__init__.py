"""Selective-SSM scan for AMD MI355X (gfx950).

Hand-written HIP kernels behind a C ABI (``include/ssm_scan.h``), with this
package as a thin torch binding: the forward scan, its backward with
recomputation from chunk-boundary states, and the single-token decode update
of the Mamba selective state-space model (Gu & Dao, arXiv 2312.00752).  Beside
it (``include/ssm_block.h``), linear attention with a decay for each head, and
the norms around a block.
"""
from ._lib import BLOCK_EXPORTS, EXPORTS, LIB_PATH, SSMError, load  # noqa: F401
from .block_ops import (DecayAttentionFn, GatedNormFn, ResidualNormFn, decay_attention,  # noqa: F401
                        decay_attn_bwd, decay_attn_fwd, decay_attn_update, gated_norm,
                        gated_norm_bwd, gated_norm_fwd, residual_norm, residual_norm_bwd,
                        residual_norm_fwd)
from .ops import (ConvScanFn, SelectiveScanFn, affine_scan, bidirectional_scan, chunk_len,  # noqa: F401
                  conv_selective_scan, scan_bwd, scan_bwd_conv, scan_fwd, scan_fwd_conv,
                  scan_fwd_plan, selective_scan, state_update)

__all__ = ["scan_fwd", "scan_bwd", "state_update", "selective_scan", "SelectiveScanFn",
           "bidirectional_scan", "scan_fwd_conv", "scan_bwd_conv", "conv_selective_scan",
           "ConvScanFn", "chunk_len", "scan_fwd_plan", "affine_scan", "decay_attn_fwd",
           "decay_attn_bwd", "decay_attn_update", "decay_attention", "DecayAttentionFn",
           "residual_norm_fwd", "residual_norm_bwd", "residual_norm", "ResidualNormFn",
           "gated_norm_fwd", "gated_norm_bwd", "gated_norm", "GatedNormFn", "load", "SSMError"]

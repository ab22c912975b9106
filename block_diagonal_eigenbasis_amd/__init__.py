"""Dobb optimizer step on MI355X (gfx950): HIP kernels behind a C ABI (libdobb.so).

The method is "Dobb: Shard-Local Preconditioning in Block-Diagonal Eigenbases" (arXiv 2610.39412):
per weight, block-diagonal input-activation second moments (EMA), a complete eigenbasis per block,
and the update sign(M_b Q_b) Q_b^T.  ``_abi`` binds the C entry points one to one; ``optimizer``
drives them with a refresh cadence, as a torch optimizer.  ``_ops`` adds what a training loop runs around
the step: gradient norms and clipping over tensor lists, and captures held in MXFP4.  ``_layers`` adds the
operators of the layers whose weights it trains: layer norm, products of FP8 operands, and captures held in FP8.
"""
from ._abi import (DOBB_BF16, DOBB_F32, DOBB_NORM_COL_L2, DOBB_NORM_IDENTITY, DOBB_NORM_SIGN,  # noqa: F401
                   DOBB_OP_ACCUMULATE, DOBB_OP_REFRESH, DOBB_OP_STEP, DOBB_REFRESH_EXACT,
                   DOBB_REFRESH_ORTH_ITER, DobbError, HParams, Shape, dobb_abi_version,
                   dobb_accumulate_moment, dobb_accumulate_moment_grouped, dobb_profile_enable,
                   dobb_profile_read, dobb_profile_reset, dobb_refresh_basis, dobb_refresh_basis_grouped,
                   dobb_step, dobb_step_grouped, dobb_step_noalloc, dobb_workspace_size, lib, make_hparams,
                   status_string, DOBB_ERR_WORKSPACE, DOBB_NOALLOC_SCRATCH_BYTES, DOBB_WS_BF16_BASIS,
                   DOBB_OP_STEP_G, dobb_step_g, dobb_step_g_grouped, DOBB_REFRESH_ORTH_ITER_CHOLQR)
from ._ops import (MX4_TILE, dobb_accumulate_moment_mx4, dobb_accumulate_moment_mx4_grouped,  # noqa: E402,F401
                   dobb_clip_grad_norm_grouped, dobb_clip_grads_grouped, dobb_grad_norm_grouped,
                   dobb_moment_mx4_workspace_size, dobb_mx4_dequantize, dobb_mx4_quantize, mx4_tiles)
from ._layers import (FP8_TILE, Fp8Capture, Fp8Operand, dobb_accumulate_moment_fp8, dobb_accumulate_moment_fp8_grouped,  # noqa: E402,F401
                      dobb_fp8_dequantize, dobb_fp8_matmul, dobb_fp8_matmul_workspace_size, dobb_fp8_quantize, dobb_layer_norm,
                      dobb_layer_norm_backward, dobb_layer_norm_fp8, dobb_moment_fp8_workspace_size, fp8_tiles)

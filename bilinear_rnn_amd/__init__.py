"""Comba mixer hot path for AMD Instinct MI355X (gfx950).

The chunk-wise parallel forward and the recurrent (decode) step of Comba,
a bilinear RNN with a scalar-plus-low-rank state transition and output
correction, and the operators a recurrent layer needs around it (short causal
convolution, selective state space scan, block norms), as hand-written HIP
kernels behind a C ABI (include/comba.h).
This package is the thin Python binding over that library.
"""
from .api import (CombaError, block_norm, block_norm_bwd, bwd_cached_workspace_size, bwd_workspace_size, check_inputs,  # noqa: F401
                  chunk_bwd, chunk_fwd, chunk_fwd_noalloc,
                  chunk_states_size, lds_probe, lib, library_path,
                  mfma_peak_probe, recurrent_step, segmented_workspace_size, selective_scan, selective_scan_bwd,
                  selective_scan_workspace_size, selective_step, short_conv, short_conv_bwd, short_conv_step,
                  varlen_order, workspace_size)

__all__ = ["chunk_fwd", "chunk_bwd", "bwd_workspace_size", "bwd_cached_workspace_size", "chunk_states_size",
           "recurrent_step", "varlen_order", "workspace_size", "segmented_workspace_size", "mfma_peak_probe",
           "lds_probe", "check_inputs", "short_conv", "short_conv_step", "short_conv_bwd", "selective_scan",
           "selective_step", "selective_scan_bwd", "selective_scan_workspace_size", "block_norm", "block_norm_bwd",
           "CombaError"]

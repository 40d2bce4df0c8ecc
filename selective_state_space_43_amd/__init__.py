"""Thin Python binding over libselscan's C ABI (include/selscan.h).

Argument marshalling only: every step of the scan runs in the HIP kernels of
``libselscan.so``.  PyTorch supplies device memory and the current stream.
There is no CPU fallback: if the library is missing the first call raises.

Entry points carry the C names:

  ssm_selective_scan_fwd(u, delta, A, B, C, D=None, z=None, delta_bias=None,
                         delta_softplus=False, h0=None, bbar="delta",
                         y=None, final_state=None, want_final_state=True,
                         checkpoints=None)
      -> (y, final_state)
  ssm_checkpoint_shape(batch, dim, dstate, seqlen) -> shape of `checkpoints`
  ssm_state_update(state, u, delta, A, B, C, D=None, z=None, delta_bias=None,
                   delta_softplus=False, bbar="delta", y=None) -> y
  ssm_lti_kernel(A, Bv, Cv, delta, L, bbar="delta", K=None) -> K
  ssm_lti_conv(K, u, D=None, y=None, method="direct") -> y  (y = K * u + D u, causal;
                                                              method "direct" or "fft")
  ssm_selective_scan_bwd(u, delta, A, B, C, dy, D=None, z=None, delta_bias=None,
                         delta_softplus=False, h0=None, dfinal_state=None,
                         bbar="delta", workspace=None, checkpoints=None)
      -> dict of gradients
  ssm_causal_conv1d_fwd(x, weight, bias=None, state_in=None, silu=True,
                        out=None, state_out=None, want_state_out=False)
      -> (out, state_out)
  ssm_causal_conv1d_update(x, conv_state, weight, bias=None, silu=True) -> out
  ssm_causal_conv1d_bwd(x, weight, dout, bias=None, state_in=None, silu=True)
      -> dict of gradients
  ssm_ssd_fwd(x, dt, A, B, C, nheads, ngroups, D=None, z=None, dt_bias=None,
              dt_softplus=True, h0=None) -> (y, final_state)      (Mamba-2 scan)
  ssm_ssd_fwd_noalloc(x, dt, A, B, C, nheads, ngroups, y, ...) -> (y, final_state)
      the same with the workspace in the library's static scratch: allocates
      nothing (for callers that cannot allocate; ssm_ssd_scratch_bytes())
  selective_scan_fn(u, delta, A, B, C, D=None, z=None, delta_bias=None,
                    delta_softplus=False, h0=None, bbar="delta")
      -> (y, final_state), differentiable (torch.autograd): the forward's
         checkpoints feed ssm_selective_scan_bwd
  causal_conv1d_fn(x, weight, bias=None, state_in=None, silu=True) -> out,
      differentiable through ssm_causal_conv1d_bwd
  ssm_conv_ssd_fwd(xbc, dt, conv_weight, A, cu_seqlens, headdim, ngroups,
                   conv_bias=None, D=None, z=None, dt_bias=None, dt_softplus=True,
                   slots=None, has_state=None, conv_state=None, ssm_state=None,
                   y=None, workspace=None) -> y
      the Mamba-2 mixer's convolution and scan over packed prompts (rows are
      tokens), the states of each sequence read and written at its slot
  ssm_conv_ssd_update(xbc, dt, conv_state, ssm_state, conv_weight, A, ngroups,
                      ..., slots=None, y=None) -> y       (one token a sequence)
  ssm_group_norm_fwd(x, weight, ngroups, bias=None, z=None, eps=1e-5,
                     center=False, activation="none", gate="none", y=None) -> y
  ssm_group_norm_bwd(dy, x, weight, ngroups, ...) -> dict of gradients
      the norm over groups of a row's channels, with its gate or activation
  group_norm_fn(x, weight, ngroups, ...) -> y, differentiable
  ssm_gated_delta_fwd(q, k, v, dt, beta, A, cu_seqlens, ngroups, dt_bias=None,
                      dt_softplus=True, beta_sigmoid=True, qk_norm=True, eps=1e-6,
                      scale=None, slots=None, has_state=None, ssm_state=None,
                      y=None, workspace=None) -> y
      the gated delta rule over packed prompts, states as for the mixer
  ssm_gated_delta_update(q, k, v, dt, beta, ssm_state, A, ngroups, ...,
                         slots=None, y=None) -> y         (one token a sequence)
  ssm_gated_delta_bwd(dy, q, k, v, dt, beta, A, cu_seqlens, ngroups, ..., h0=None,
                      dfinal_state=None, workspace=None) -> dict of gradients
  gated_delta_fn(q, k, v, dt, beta, A, cu_seqlens, ngroups, ..., h0=None)
      -> (y, final_state), differentiable
  ssm_add_norm_fwd(x, weight, residual=None, eps=1e-5, quant="none", block=0,
                   residual_out=None, y=None, scales=None)
      -> (y, residual_out, scales)
      the residual's addition and the root-mean-square norm of the sum, the
      output in 8 bits with scales for quant="e4m3"
  ssm_add_norm_bwd(dy, r, weight, dresidual_out=None, eps=1e-5, workspace=None)
      -> dict of gradients
  add_norm_fn(x, weight, residual=None, eps=1e-5) -> (y, residual_out),
      differentiable

Layouts: u, delta, z, y [batch, dim, L]; B, C [batch, dstate, L]; A
[dim, dstate]; D, delta_bias [dim]; h0 / final_state / state
[batch, dim, dstate]; the mixer's tensors are [rows, channels] with any row
stride.  Sequence tensors are torch.bfloat16 or torch.float32
(one dtype for all of them); everything else is float32.
"""
from __future__ import annotations

from ._lib import (SSM_ACT_NONE, SSM_ACT_SILU, SSM_GATE_AFTER, SSM_GATE_BEFORE, SSM_GATE_NONE,
                   SSM_QUANT_E4M3, SSM_QUANT_NONE, SSM_BBAR_DELTA_B, SSM_BBAR_ZOH_EXACT, SSM_DTYPE_BF16, SSM_DTYPE_F32,
                   SelscanError, library_path, lib, ssm_abi_version, ssm_last_error,
                   ssm_status_str)
from .binding import (ssm_causal_conv1d_bwd, ssm_causal_conv1d_fwd, ssm_causal_conv1d_update,
                      ssm_checkpoint_shape, ssm_lti_conv, ssm_lti_conv_fft_workspace_size,
                      ssm_lti_kernel,
                      ssm_selective_scan_bwd, ssm_ssd_fwd, ssm_ssd_fwd_noalloc,
                      ssm_ssd_scratch_bytes, ssm_ssd_workspace_size,
                      ssm_selective_scan_bwd_workspace_size, ssm_selective_scan_fwd,
                      ssm_state_update, selective_scan_fn, causal_conv1d_fn,
                      ssm_conv_ssd_fwd, ssm_conv_ssd_update, ssm_conv_ssd_workspace_size,
                      ssm_group_norm_fwd, ssm_group_norm_bwd, ssm_group_norm_bwd_workspace_size,
                      group_norm_fn,
                      ssm_gated_delta_fwd, ssm_gated_delta_update, ssm_gated_delta_bwd,
                      ssm_gated_delta_workspace_size, ssm_gated_delta_bwd_workspace_size,
                      gated_delta_fn, ssm_add_norm_fwd, ssm_add_norm_bwd,
                      ssm_add_norm_bwd_workspace_size, add_norm_fn)

__all__ = [
    "ssm_selective_scan_fwd", "ssm_state_update", "ssm_lti_kernel", "ssm_lti_conv",
    "ssm_lti_conv_fft_workspace_size",
    "ssm_selective_scan_bwd", "ssm_checkpoint_shape", "selective_scan_fn", "causal_conv1d_fn",
    "ssm_selective_scan_bwd_workspace_size", "ssm_causal_conv1d_fwd", "ssm_causal_conv1d_update",
    "ssm_causal_conv1d_bwd", "ssm_ssd_fwd", "ssm_ssd_workspace_size", "ssm_ssd_fwd_noalloc",
    "ssm_ssd_scratch_bytes", "ssm_conv_ssd_fwd", "ssm_conv_ssd_update",
    "ssm_conv_ssd_workspace_size", "ssm_group_norm_fwd", "ssm_group_norm_bwd",
    "ssm_group_norm_bwd_workspace_size", "group_norm_fn",
    "ssm_gated_delta_fwd", "ssm_gated_delta_update", "ssm_gated_delta_bwd",
    "ssm_gated_delta_workspace_size", "ssm_gated_delta_bwd_workspace_size", "gated_delta_fn",
    "ssm_add_norm_fwd", "ssm_add_norm_bwd", "ssm_add_norm_bwd_workspace_size", "add_norm_fn",
    "SSM_QUANT_NONE", "SSM_QUANT_E4M3", "ssm_status_str",
    "ssm_last_error", "ssm_abi_version", "SelscanError", "library_path", "lib",
    "SSM_ACT_NONE", "SSM_ACT_SILU", "SSM_GATE_NONE", "SSM_GATE_BEFORE", "SSM_GATE_AFTER",
    "SSM_DTYPE_F32", "SSM_DTYPE_BF16", "SSM_BBAR_DELTA_B", "SSM_BBAR_ZOH_EXACT",
]

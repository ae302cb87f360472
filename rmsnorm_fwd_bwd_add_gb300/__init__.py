"""GB300-native row-wise RMSNorm hot path.

Two operations, hand-written CUDA for sm_103a behind the C ABI of
include/rmsnorm.h (librmsnorm_gb300.so), with these thin Python bindings:

  rmsnorm_fwd  -- fused residual-add RMSNorm forward with two outputs
                  (out, new_residual), fp32 accumulation, weight_bias scalar.
  rmsnorm_fwd_bind, rmsnorm_vjp_bind -- the same calls with their tensors
                  checked once, for loops over fixed buffers (decode).
  rmsnorm_vjp  -- RMSNorm VJP: gx and an fp32 gw reduced across rows inside
                  the kernels (deterministic, no [rows, D] temporary).
  rmsnorm_fused_vjp -- VJP of the two-output fused op (adds the gradient that
                  reaches new_residual in the same pass).
  rmsnorm_fwd_ex, rmsnorm_vjp_ex -- the same on rows a stride apart, with the
                  forward's per-row scale (rstd) written and reused.
  fp16, bf16 and fp32 tensors.
  rmsnorm_block_fwd, rmsnorm_block_vjp -- the norms before and after a block
                  fused with the block's gate and residual scale.
  fused_add_rmsnorm, rms_norm, block_norm -- torch.autograd wrappers.
  rmsnorm_gated_silu -- the decode loop's gated activation silu(x[:d]) * x[d:].
  rmsnorm_rope_kv_append -- rotary embedding of q and k with the KV-cache append.
  rope_frequencies, rmsnorm_rope, rmsnorm_rope_kv_append_ex, rope -- rotary
                  positions over part of the head, stretched for long contexts,
                  on strided heads: forward, VJP (rope: torch.autograd) and the
                  append.
  rope_sections, rmsnorm_rope_axes -- the same with positions of several axes.
  rmsnorm_fwd_q8 -- the forward with an e4m3 output and its scales.
  rmsnorm_kv_append, rmsnorm_kv_read -- the append into a cache of 8 bits with a
                  scale a head, and tokens read back from it.
  rmsnorm_kv_plan, rmsnorm_kv_release -- block tables and slot maps of a paged
                  cache from the requests' lengths.

PyTorch supplies device memory and streams only.
"""
from .api import (  # noqa: F401
    BoundCall,
    KvPlan,
    rmsnorm_block_fwd,
    rmsnorm_block_vjp,
    rmsnorm_debug_claim_counters,
    rmsnorm_debug_fail_allocs,
    rmsnorm_debug_inject,
    rmsnorm_describe_dispatch,
    rmsnorm_device_status,
    rmsnorm_fused_vjp,
    rmsnorm_fwd,
    rmsnorm_fwd_bind,
    rmsnorm_fwd_ex,
    rmsnorm_fwd_q8,
    rmsnorm_gated_silu,
    rmsnorm_kv_append,
    rmsnorm_kv_plan,
    rmsnorm_kv_read,
    rmsnorm_kv_release,
    rmsnorm_rope,
    rmsnorm_rope_axes,
    rmsnorm_rope_kv_append,
    rmsnorm_rope_kv_append_ex,
    rmsnorm_status_string,
    rmsnorm_vjp,
    rmsnorm_vjp_bind,
    rmsnorm_vjp_ex,
    rmsnorm_vjp_noalloc,
    rmsnorm_vjp_workspace_size,
    rmsnorm_vjp_ws,
    rope_frequencies,
    rope_sections,
)
from ._native import DEVSTATUS_BAD_INDEX, DEVSTATUS_WAIT_TIMEOUT, MAX_D, RmsnormError  # noqa: F401
from .autograd import block_norm, fused_add_rmsnorm, rms_norm, rope  # noqa: F401

__all__ = [
    "rmsnorm_fwd",
    "rmsnorm_vjp",
    "rmsnorm_fwd_bind",
    "rmsnorm_vjp_bind",
    "BoundCall",
    "rmsnorm_fused_vjp",
    "rmsnorm_fwd_ex",
    "rmsnorm_vjp_ex",
    "rmsnorm_block_fwd",
    "rmsnorm_block_vjp",
    "rmsnorm_gated_silu",
    "rmsnorm_rope_kv_append",
    "rope_frequencies",
    "rmsnorm_rope",
    "rope_sections",
    "rmsnorm_rope_axes",
    "rmsnorm_rope_kv_append_ex",
    "rmsnorm_fwd_q8",
    "rmsnorm_kv_append",
    "rmsnorm_kv_read",
    "rmsnorm_kv_plan",
    "rmsnorm_kv_release",
    "KvPlan",
    "rope",
    "fused_add_rmsnorm",
    "rms_norm",
    "block_norm",
    "rmsnorm_vjp_ws",
    "rmsnorm_vjp_noalloc",
    "rmsnorm_vjp_workspace_size",
    "rmsnorm_device_status",
    "rmsnorm_debug_inject",
    "rmsnorm_debug_fail_allocs",
    "rmsnorm_debug_claim_counters",
    "rmsnorm_describe_dispatch",
    "rmsnorm_status_string",
    "RmsnormError",
]

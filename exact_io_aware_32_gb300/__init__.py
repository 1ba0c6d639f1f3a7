"""Exact, IO-aware scaled-dot-product attention for NVIDIA GB300 (sm_103a).

The kernels sit behind the C ABI of ``include/fa.h`` (``libfa.so``); this
package holds the thin ctypes binding (``fa``), the build script, the seeded
input generators and the flop/byte model the benchmark reports against.
"""
from .fa import (  # noqa: F401
    FA_OK, FAError, attention, attention_window, backward, backward_dropout, backward_kv, backward_rope, backward_window,
    fa_bwd, fa_bwd_dropout, fa_bwd_kv, fa_bwd_kv_workspace_bytes, fa_bwd_noalloc, fa_bwd_window,
    fa_bwd_window_workspace_bytes, fa_bwd_workspace_bytes, fa_device_status, fa_fwd, fa_fwd_dropout, fa_fwd_fp8, fa_fwd_kv,
    fa_fwd_kv_workspace_bytes, fa_fwd_paged, fa_fwd_paged_window, fa_fwd_paged_workspace_bytes, fa_fwd_window,
    fa_paged_plan, fa_paged_positions, fa_paged_rope_store, fa_paged_store, fa_rope_bwd, fa_rope_bwd_workspace_bytes,
    fa_rope_fwd, fa_status_string, fa_test_arm_fault, forward, forward_dropout, forward_fp8, forward_kv, forward_paged,
    forward_rope, forward_window, paged_plan, paged_positions, paged_rope_store, paged_store, rope, rope_frequencies,
)

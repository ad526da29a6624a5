"""GB300-native batched draft-verification sampler for speculative decoding.

The computation lives in libspecverify.so (hand-written sm_103a CUDA behind
the C ABI of include/specverify.h); this package is its Python binding.
"""
from ._binding import (ROW_STATUS, SPEC_BF16, SPEC_E4M3, SPEC_F16, SPEC_F32,  # noqa: F401
                       SPEC_GREEDY, SPEC_STOCHASTIC, SpecError, debug_force_wait_timeout,
                       get_wait_timeout_ns, lib, set_wait_timeout_ns, spec_adaptive_tree_policy,
                       spec_drift_residuals, spec_kv_append, spec_kv_compact_pages, spec_kv_compact_tree,
                       spec_kv_entry_bytes, spec_kv_read, spec_page_plan, spec_paged_attention, spec_prefix_attention,
                       spec_rollback_lengths, spec_sample, spec_token_logprobs, spec_verify_chain,
                       spec_verify_tree)

"""GB300-native verification step of speculative decoding.

The compute lives in libspecverify.so (hand-written CUDA for sm_103a, C ABI in
include/spec_verify.h); this package is its thin binding plus the seeded
workload generator used by the tests and the benchmark.
"""
from .api import (AttnCall, Rope, SamplerConfig, SpecError, accept_sample,  # noqa: F401
                  accept_sample_tree, append_block, append_scaled, append_tokens, attn_num_splits,
                  attn_workspace_size, decode_attn, decode_attn_workspace_size, extend_tables,
                  kv_commit, load, logits_penalize, logits_process, new_workspace, read_scaled,
                  release_pages, rotate, sample_workspace_size, tree_prepare, verify_attn,
                  verify_attn_scaled, verify_attn_scaled_workspace_size, workspace_error)

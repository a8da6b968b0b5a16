"""GB300 (sm_103a) paged KV-cache attention: store_kv, paged decode and
extend attention, the log-sum-exp merge, and beside them the append of normed
and rotated q, k, v, decode and extend under score rules, and attention of
drafted token trees, as hand-written CUDA kernels behind the C ABI of
include/pkv.h. This package holds the ctypes binding
(same names as the C entry points), the nvcc build and the seeded
synthetic-input generator used by the tests and the benchmark.
"""
from .binding import (PkvError, pkv_cascade_workspace_size,  # noqa: F401
                      pkv_decode_workspace_size, pkv_extend_workspace_size, pkv_init,
                      pkv_kv_store, pkv_paged_cascade_decode_attn,
                      pkv_merge_lse, pkv_norm_rope_kv_store, pkv_paged_decode_attn,
                      pkv_paged_decode_attn_noalloc, pkv_paged_decode_attn_store,
                      pkv_paged_extend_attn, pkv_paged_extend_attn_store,
                      pkv_paged_tree_attn, pkv_tree_workspace_size,
                      pkv_decode_mod_workspace_size, pkv_extend_mod_workspace_size,
                      pkv_paged_decode_attn_mod,
                      pkv_paged_extend_attn_mod,
                      pkv_read_device_errors)

"""Paged decode/verify attention, KV append and speculative acceptance for
one GB300 GPU (sm_103a), with eviction, page-sparse attention, page assignment
and log probabilities beside them.

The computation lives in libsvp.so (CUDA kernels behind the C ABI declared in
include/svp.h); this package is its thin Python binding.  Importing it loads
nothing; the first call loads the library and raises if it is not built.
"""
from .binding import (  # noqa: F401
    StepRunner,
    SvpError,
    fp4_row_bytes,
    kv_append,
    kv_assign_pages,
    kv_evict,
    kv_gather,
    kv_page_bounds,
    last_launch_count,
    load_library,
    paged_decode_attention,
    paged_page_scores,
    paged_score_update,
    paged_select_pages,
    paged_sparse_attention,
    paged_tree_attention,
    read_device_status,
    spec_accept,
    spec_accept_tree,
    token_logprobs,
    workspace_for,
)

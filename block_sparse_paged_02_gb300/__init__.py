"""block_sparse_paged_02_gb300 -- block-sparse paged decode (MiniMax-M3-style
index top-k + sparse paged attention), draft-tree attention over the same
cache and eviction from it, prompts into it and the sharing of its pages, for
one GB300 (sm_103a).

The compute runs in libmsa.so (CUDA kernels behind the C ABI of include/msa.h,
include/msa_cache.h and include/msa_prompt.h); this package builds it and
marshals torch tensors into it.
"""
from .binding import (MSA_DEV_BAD_LEN, MSA_DEV_BAD_PAGE, MSA_DEV_BAD_TABLE, MSA_DEV_MALFORMED,
                      MSA_DEV_TIMEOUT, MSA_KV_BF16, MSA_KV_FP8_E4M3, MSA_SCALE_NONE,
                      MSA_SCALE_PER_TOKEN_HEAD, MSA_SCALE_SCALAR, MsaError, lib, make_attn_args,
                      make_batch, make_index_cache, make_trace, msa_decode, msa_index_score, msa_kv_insert,
                      msa_sparse_paged_attn, msa_status_string, msa_topk_build_table,
                      msa_workspace_size)
from .binding import make_mla_args, msa_sparse_mla_decode, msa_sparse_mla_workspace_size
from .binding import MSA_CHECK_WAIT_COPY, MSA_CHECK_WAIT_TMEM, msa_check_bounded_wait
from .binding import (make_cache_view, make_kv_pools, make_tree, msa_attn_mass, msa_evict_select,
                      msa_kv_compact, msa_tree_attn, msa_tree_attn_workspace_size)
from .binding import (MSA_DEV_BAD_POS, MSA_DEV_NO_PAGES, make_page_set, make_qkv, make_rope, msa_page_copy,
                      msa_page_fork, msa_prompt_attn, msa_prompt_attn_workspace_size, msa_qk_rope_insert)
from .case import DeviceCase, MlaCase

__all__ = [
    "lib", "make_batch", "make_attn_args", "make_index_cache", "make_trace", "msa_index_score",
    "msa_topk_build_table", "msa_sparse_paged_attn", "msa_decode", "msa_kv_insert",
    "msa_workspace_size",
    "msa_status_string", "MsaError", "DeviceCase", "MlaCase", "make_mla_args",
    "msa_sparse_mla_decode", "msa_sparse_mla_workspace_size", "MSA_KV_BF16", "MSA_KV_FP8_E4M3",
    "MSA_SCALE_NONE", "MSA_SCALE_SCALAR", "MSA_SCALE_PER_TOKEN_HEAD", "MSA_DEV_BAD_PAGE",
    "MSA_DEV_BAD_LEN", "MSA_DEV_MALFORMED", "MSA_DEV_BAD_TABLE", "MSA_DEV_TIMEOUT",
    "make_tree", "msa_tree_attn", "msa_tree_attn_workspace_size", "msa_attn_mass",
    "make_cache_view", "msa_evict_select", "make_kv_pools", "msa_kv_compact",
    "make_rope", "make_qkv", "msa_qk_rope_insert", "msa_prompt_attn", "msa_prompt_attn_workspace_size",
    "make_page_set", "msa_page_fork", "msa_page_copy", "MSA_DEV_BAD_POS", "MSA_DEV_NO_PAGES",
    "msa_check_bounded_wait", "MSA_CHECK_WAIT_TMEM", "MSA_CHECK_WAIT_COPY",
]

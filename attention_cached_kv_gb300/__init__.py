"""GB300 (sm_103a) library for attention of new tokens against a read-only
cached KV segment: gist-compressed items gathered by id, or a paged cache read
through a block table.

The compute lives in ``_lib/libgistattn.so`` (C ABI in include/gist_attn.h);
``binding`` marshals torch tensors into it; ``workloads`` draws seeded
synthetic inputs.  The library is loaded on first use and every call fails
loudly if it has not been built.
"""
from .binding import (FLAG_PREROTATED, GistAttnError, PagedPlan, STATUS_BAD_BLOCK, STATUS_NOT_SERVED, STATUS_RANGE, STATUS_TIMEOUT, gist_attn_fwd,
                      gist_attn_fwd_block_mass, gist_attn_fwd_fp8kv, gist_attn_fwd_gist_mask,
                      gist_attn_fwd_ws, workspace_bytes,
                      gist_attn_paged_fp8kv, gist_kv_append_fp8, gist_paged_plan, paged_workspace_bytes,
                      PagesCompact, PagesFork, PagesFree, gist_attn_paged_decode, gist_out_proj_w4,
                      gist_pages_compact, gist_pages_copy, gist_pages_fork, gist_pages_free,
                      gist_qkv_rope_w4, paged_decode_workspace_bytes,
                      gist_kv_append, gist_kv_store, gist_out_proj, gist_qkv_rope,
                      gist_attn_gather_debug, kv_bytes_batch, kv_bytes_per_item,
                      kv_bytes_per_position, load_library, status_string)

__all__ = ["FLAG_PREROTATED", "GistAttnError", "PagedPlan", "STATUS_NOT_SERVED", "STATUS_BAD_BLOCK", "STATUS_RANGE", "STATUS_TIMEOUT", "gist_attn_fwd", "gist_attn_fwd_fp8kv",
           "gist_attn_fwd_block_mass", "gist_attn_fwd_gist_mask", "gist_attn_fwd_ws", "workspace_bytes",
           "gist_attn_paged_decode", "paged_decode_workspace_bytes", "PagesCompact", "PagesFork", "PagesFree",
           "gist_pages_compact", "gist_pages_copy", "gist_pages_fork", "gist_pages_free",
           "gist_qkv_rope_w4", "gist_out_proj_w4",
           "gist_paged_plan", "gist_kv_append_fp8", "gist_attn_paged_fp8kv", "paged_workspace_bytes",
           "gist_kv_append", "gist_kv_store",
           "gist_qkv_rope", "gist_out_proj",
           "gist_attn_gather_debug", "kv_bytes_batch", "kv_bytes_per_item",
           "kv_bytes_per_position", "load_library", "status_string"]

"""MI355X-native fused MLA query up-projection (GEMM + RoPE/YaRN + MXFP8) and its backward.

The compute lives in libmlaqup.so (hand-written HIP kernels for gfx950, C ABI
in include/mla_qup.h); `binding` marshals torch device tensors into it.
"""
from .binding import (  # noqa: F401
    DTYPE_BF16, DTYPE_FP32, DTYPE_INT8, DTYPE_MXFP8, FMT_BSHD, FMT_SBHD, FMT_THD, FUNCTIONS, LIB_PATH, MlaError,
    lib, mla_qup_bwd, mla_qup_bwd_mxfp8, mla_qup_bwd_noalloc, mla_qup_bwd_mxfp8_workspace_size, mla_qup_bwd_workspace_size,
    mla_kv_rope, mla_qup_fwd, mla_status_str, mxfp8_quantize, mxfp8_quantize_t, rope_cache_build,
    PagePool, mla_draft_accept, mla_kv_rope_paged, mla_pages_compact, mla_pages_copy, mla_pages_fork, mla_pages_free,
    mla_pages_reserve, mla_pages_workspace_size, mla_qup_fwd_w4, mla_tree_attention,
    mla_tree_attention_workspace_size, mxfp4_quantize,
    int8_quantize, mla_attn_bwd, mla_attn_bwd_workspace_size, mla_attn_fwd, mla_attn_fwd_workspace_size, mla_attn_spans,
    mla_qup_fwd_i8, mla_rmsnorm_bwd, mla_rmsnorm_bwd_workspace_size, mla_rmsnorm_fwd)

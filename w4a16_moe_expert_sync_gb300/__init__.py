"""GB300-native W4A16 routed mixture-of-experts layer.

The compute lives in libw4moe.so (hand-written CUDA for sm_103a, C ABI in
include/w4moe.h).  This package is its thin Python binding plus the seeded
synthetic workloads (``workloads``) used by the tests and the benchmark.

    import w4a16_moe_expert_sync_gb300 as w4
    q, s, z = w4.w4_quantize(W_fp32_cuda, group=128)
    ids, w = w4.w4_moe_route(logits, k=8)
    out = w4.w4_moe_layer(x_bf16, ids, w, (gu_q, gu_s, gu_z), (dn_q, dn_s, dn_z))

A decoding step has the layer for a few tokens, a paged cache and attention:

    w4.w4_kv_reserve(table, lens, refs, slots, new_lens, page_size)
    w4.w4_kv_append(k_pages, v_pages, table, lens, k, v, q_offsets)
    o = w4.w4_attn_shared_prefix(q, k_pages, v_pages, table, lens, q_offsets,
                                 group_offsets, shared_lens, max_q=1)
    out, ids, w = w4.w4_moe_layer_few_from_logits(x, logits, 8, gate_up, down)

A step that verifies a tree of drafts has projections for few rows, the rotation on
the way into the cache, attention by ancestors, and keeps the accepted path:

    qkv = w4.w4_w4a16_linear_few(x, *weight)
    q = w4.w4_kv_append_rope(k_pages, v_pages, table, lens, q, k, v, q_offsets, steps,
                             positions=depths)
    o = w4.w4_attn_tree(q, k_pages, v_pages, table, lens, q_offsets, tree, max_q=n)
    w4.w4_kv_keep(pool, table, lens, refs, q_offsets, kept, kept_offsets)
"""
from ._lib import (W4_DEV_BAD_EXPERT_ID, W4_DEV_FP16_RANGE, W4_DEV_OUT_OF_BOUNDS,
                   W4_DEV_PIPELINE_TIMEOUT,
                   W4_DEV_TOO_MANY_JOBS, W4_DEV_BAD_SLOT, W4_DEV_BAD_PAGE, W4_DEV_NO_PAGES,
                   W4Error, header_functions, korder_to_natural, load_library,
                   w4_gather_activations, w4_grouped_gemm_down, w4_moe_align_gather,
                   w4_grouped_gemm_gate_up, w4_moe_align, w4_moe_align_capacity,
                   w4_moe_combine_fixed_order, w4_moe_combine_prepare,
                   w4_grouped_gemm_down_combine, w4_moe_layer, w4_moe_layer_static_scratch,
                   w4_moe_layer_workspace_size, w4_moe_layer_from_logits, w4_moe_layer_host,
                   w4_moe_layer_host_workspace_size,
                   w4_moe_layer_few, w4_moe_layer_few_from_logits,
                   w4_moe_layer_few_workspace_size,
                   w4_attn_shared_prefix, w4_attn_shared_prefix_workspace_size, w4_attn_tree,
                   w4_kv_append, w4_kv_append_rope, w4_kv_compact, w4_kv_copy_pages, w4_kv_fork,
                   w4_kv_free, w4_kv_keep, w4_kv_reserve, w4_kv_workspace_size,
                   w4_qk_norm_rope, w4_rope_steps,
                   w4_moe_route, w4_moe_route_align_gather, w4_quantize, w4_rmsnorm,
                   w4_sample_logits, w4_sample_logits_workspace_size, w4_fused_entropy,
                   w4_gumbel_argmax_sample, w4_w4a16_linear, w4_w4a16_linear_few,
                   w4_w4a16_linear_workspace_size)

__all__ = [
    "W4Error", "load_library", "header_functions", "korder_to_natural", "w4_gather_activations",
    "w4_moe_align_gather",
    "w4_quantize", "w4_moe_route", "w4_moe_align", "w4_moe_align_capacity",
    "w4_grouped_gemm_gate_up", "w4_grouped_gemm_down", "w4_moe_combine_fixed_order",
    "w4_moe_combine_prepare", "w4_grouped_gemm_down_combine",
    "w4_moe_layer", "w4_moe_layer_workspace_size", "w4_moe_layer_static_scratch",
    "w4_moe_layer_host", "w4_moe_layer_host_workspace_size",
    "w4_moe_layer_few", "w4_moe_layer_few_from_logits", "w4_moe_layer_few_workspace_size",
    "w4_moe_route_align_gather", "w4_moe_layer_from_logits", "w4_rmsnorm", "w4_sample_logits",
    "w4_sample_logits_workspace_size", "w4_fused_entropy", "w4_gumbel_argmax_sample",
    "w4_w4a16_linear", "w4_w4a16_linear_few", "w4_w4a16_linear_workspace_size",
    "w4_attn_shared_prefix", "w4_attn_shared_prefix_workspace_size", "w4_attn_tree",
    "w4_kv_reserve", "w4_kv_free", "w4_kv_fork", "w4_kv_copy_pages", "w4_kv_compact",
    "w4_kv_append", "w4_kv_keep", "w4_kv_workspace_size",
    "w4_rope_steps", "w4_qk_norm_rope", "w4_kv_append_rope",
    "W4_DEV_BAD_SLOT", "W4_DEV_BAD_PAGE", "W4_DEV_NO_PAGES",
    "W4_DEV_BAD_EXPERT_ID", "W4_DEV_FP16_RANGE", "W4_DEV_OUT_OF_BOUNDS", "W4_DEV_PIPELINE_TIMEOUT", "W4_DEV_TOO_MANY_JOBS",
]

"""GB300-native block-FP8 (E4M3) Mixture-of-Experts FFN layer.

The layer runs in ``libmoe_fp8.so`` (hand-written sm_103a CUDA kernels behind
the C ABI in ``include/moe_fp8.h``).  This package is its thin Python binding:
``_lib`` (ctypes, one function per C entry point) and ``device`` (weights held
in HBM as PyTorch tensors, plus a forward call).  ``decoder`` holds the
operators of the rest of a decoder layer: expert selection with balance bias
and groups, query/key norms with rotary positions into a paged cache, paged
attention of one new token per sequence or of several drafted ones, latent
attention with its paged cache, and block-FP8 linear layers.  The package never
computes any part of these itself and has no CPU fallback.
"""
from ._lib import (  # noqa: F401
    Dims, Fp8Ffn, Fp8Mat, MoeError, dims, ffn, lib, version, workspace_bytes,
    moe_route, moe_permute, moe_expert_ffn_fp8, moe_combine, moe_layer_forward,
    moe_layer_forward_gated, moe_layer_forward_act8,
    moe_read_device_status, kernel_launches, expert_uses_gemm,
    moe_select_experts, moe_route_select, moe_experts_forward, moe_qk_norm_rope,
    moe_paged_attention, moe_tree_attention, moe_latent_store, moe_latent_attention,
    moe_expanded_attention, moe_linear_fp8,
)

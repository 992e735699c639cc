"""MI355X (gfx950) MoE token dispatch / unpermute-combine.

Top-k routing with a softmax over the selected logits (optionally group-limited), the expert
histogram with its running sum (group_list), the stable expert-major permute (standard,
drop-and-pad, expert-aligned, the two-stage group dispatch, an FP8 E4M3 dispatch), the weighted
unpermute-combine (optional bias) and the per-group local pre-combine, with the backward of the
combine and of the routing softmax; the residual RMS norm that stands before (rows, FP8 rows,
backward), the whole layer for a few tokens, the router's balance loss with its gradient, and rows in
4 bits (MXFP4) with the experts' products of them, as hand-written HIP kernels behind a C ABI
(``include/moe_dispatch.h``, ``libmoe_dispatch.so``). This package is the torch binding.
"""
from .ops import (MoeIndex, add_rmsnorm, add_rmsnorm_backward, add_rmsnorm_fp8, alloc_index, balance_loss,
                  balance_loss_backward, balance_workspace_bytes, build_index, build_index_noalloc, expert_capacity,
                  few_token_experts, few_token_layer, few_token_workspace_bytes, group_precombine,
                  grouped_product_mxfp4, index_rows, permute, permute_grouped, permute_grouped_fp8, permute_scatter,
                  permute_scatter_fp8, quantize_fp8, quantize_mxfp4, rmsnorm_workspace_bytes, route_topk,
                  route_topk_backward, route_topk_index, unpermute_combine, unpermute_combine_backward,
                  workspace_bytes)
from ._capi import MoeError, lib

__all__ = ["MoeError", "MoeIndex", "add_rmsnorm", "add_rmsnorm_backward", "add_rmsnorm_fp8", "alloc_index",
           "balance_loss", "balance_loss_backward", "balance_workspace_bytes", "build_index",
           "build_index_noalloc", "expert_capacity", "few_token_experts", "few_token_layer",
           "few_token_workspace_bytes", "group_precombine", "grouped_product_mxfp4", "index_rows", "lib",
           "permute", "permute_grouped", "permute_grouped_fp8", "permute_scatter", "permute_scatter_fp8",
           "quantize_fp8", "quantize_mxfp4", "rmsnorm_workspace_bytes", "route_topk", "route_topk_backward",
           "route_topk_index", "unpermute_combine", "unpermute_combine_backward", "workspace_bytes"]

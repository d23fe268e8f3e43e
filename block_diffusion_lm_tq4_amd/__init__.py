"""TQ4_1S ("Config-I") dequantize-and-multiply library for AMD MI355X (gfx950).

The kernels live in ``libtq4.so`` (C ABI in ``include/tq4.h``), built in-tree
by ``block_diffusion_lm_tq4_amd.build``.  ``ops`` is the torch-facing binding;
``inputs`` holds the seeded synthetic workloads.
"""

from .ops import (act_int8, act_mxfp4, act_mxfp8, act_rht, codebook, fp8_cache, fp8_cache_experts,  # noqa: F401
                  int8_cache, int8_cache_bf16, int8_cache_experts, int8_cache_size, linear,
                  linear_epilogue, linear_epilogue_bf16, linear_fp8, linear_fp8_quantized,
                  linear_int8, linear_int8_epilogue, linear_int8_epilogue_bf16,
                  linear_int8_quantized, linear_int8_workspace_size, linear_mxfp4,
                  linear_mxfp4_epilogue, linear_mxfp4_epilogue_bf16, linear_mxfp4_quantized,
                  linear_mxfp4_workspace_size, linear_rotated, linear_workspace_size, moe_balance,
                  moe_balance_workspace_size, moe_block, moe_grouped, moe_grouped_fp8,
                  moe_grouped_fp8_workspace_size, moe_grouped_int8,
                  moe_grouped_int8_workspace_size, moe_grouped_mxfp4,
                  moe_grouped_mxfp4_workspace_size, moe_route, moe_router, moe_router_backward,
                  moe_router_scored, moe_workspace_size, mxfp4_cache, mxfp4_cache_bf16,
                  mxfp4_cache_experts, mxfp4_cache_size, mxfp4_values, pack, packed_size)

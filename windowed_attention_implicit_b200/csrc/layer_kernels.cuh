// layer_kernels.cuh -- trace ids and names of the layer operators' kernels
// (layer norm, linear projections, gated feed-forward block).  X(id, name)
#pragma once

#define RIB_LAYER_KERNELS(X)                \
  X(K_LN_FWD, "layer_norm_fwd_kernel")      \
  X(K_LN_BWD, "layer_norm_bwd_kernel")      \
  X(K_ROWS_RED, "reduce_rows_kernel")       \
  X(K_LINEAR, "gemm_kernel (linear)")       \
  X(K_LINEAR_DX, "gemm_kernel (dx)")        \
  X(K_GATED, "gemm_kernel (gated)")         \
  X(K_FFN_FUSED, "ffn_fused_kernel")        \
  X(K_FEW_ROWS, "few_rows_kernel")          \
  X(K_DZ, "dz_kernel")                      \
  X(K_DW, "dw_kernel")                      \
  X(K_DW_RED, "dw_reduce_kernel")           \
  X(K_FFN_BWD, "ffn_bwd_kernel")

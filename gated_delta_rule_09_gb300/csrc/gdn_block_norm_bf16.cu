// Norms around a block: rows of bf16, residual stream of bf16.
#include "gdn_block_norm.cuh"

cudaError_t gdn_block_norm_bf16(const GdnBlockNormArgs &a, cudaStream_t s) { return block_norm<__nv_bfloat16, __nv_bfloat16>(a, s); }

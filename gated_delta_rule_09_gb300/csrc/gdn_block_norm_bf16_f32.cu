// Norms around a block: rows of bf16, residual stream of fp32.
#include "gdn_block_norm.cuh"

cudaError_t gdn_block_norm_bf16_f32(const GdnBlockNormArgs &a, cudaStream_t s) { return block_norm<__nv_bfloat16, float>(a, s); }

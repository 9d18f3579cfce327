// Norms around a block: rows of fp32, residual stream of fp32.
#include "gdn_block_norm.cuh"

cudaError_t gdn_block_norm_f32(const GdnBlockNormArgs &a, cudaStream_t s) { return block_norm<float, float>(a, s); }

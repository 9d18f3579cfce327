// The state space scan over prompts for fp32 inputs.
#include "gdn_ssm_scan.cuh"

cudaError_t gdn_ssm_scan_f32(const GdnSsmArgs &a, cudaStream_t s) { return scan<float>(a, s); }

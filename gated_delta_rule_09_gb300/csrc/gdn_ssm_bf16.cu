// The state space scan over prompts for bf16 inputs.
#include "gdn_ssm_scan.cuh"

cudaError_t gdn_ssm_scan_bf16(const GdnSsmArgs &a, cudaStream_t s) { return scan<__nv_bfloat16>(a, s); }

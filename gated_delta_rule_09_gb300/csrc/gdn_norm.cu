// Group norm of token rows, channels last, with an activation or a gate.
//
// Each run of channels / groups channels of a row is normalised by its own
// mean and variance (or mean square); y = act(u weight + bias) silu(gate).
// Two values are computed per element moved: bound by HBM.
#include "gdn_layer.h"
#include "gdn_layer.cuh"

namespace {

using namespace gdn_layer;

constexpr int kThreads = 128;

__device__ __forceinline__ float block_sum(float v, float *sh)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    __syncthreads();  // sh may still be read from the previous sum
    if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = v;
    __syncthreads();
    v = 0.f;
#pragma unroll
    for (int i = 0; i < kThreads / 32; ++i) v += sh[i];
    return v;
}

// One block per group: three passes over the group's channels (from cache).
template <typename E>
__global__ void __launch_bounds__(kThreads) gdn_group_norm_kernel(const GdnNormArgs a)
{
    __shared__ float sh[kThreads / 32];
    const int width = a.channels / a.groups;
    const int64_t row = blockIdx.x / a.groups;
    const int c0 = (int)(blockIdx.x % a.groups) * width;
    const E *x = static_cast<const E *>(a.x) + row * a.ld_x + c0;
    const E *gate = a.gate ? static_cast<const E *>(a.gate) + row * a.ld_gate + c0 : nullptr;
    E *y = static_cast<E *>(a.y) + row * a.ld_y + c0;
    float mean = 0.f;
    if (!a.rms) {
        float s = 0.f;
        for (int i = threadIdx.x; i < width; i += kThreads) s += to_f(x[i]);
        mean = block_sum(s, sh) / width;
    }
    float q = 0.f;
    for (int i = threadIdx.x; i < width; i += kThreads) {
        const float v = to_f(x[i]) - mean;
        q = fmaf(v, v, q);
    }
    const float rstd = rsqrtf(block_sum(q, sh) / width + a.eps);
    for (int i = threadIdx.x; i < width; i += kThreads) {
        float v = (to_f(x[i]) - mean) * rstd;
        if (a.weight) v *= a.weight[c0 + i];
        if (a.bias) v += a.bias[c0 + i];
        if (a.act == GDN_ACT_SILU) v = silu(v);
        if (gate) v *= silu(to_f(gate[i]));
        y[i] = from_f<E>(v);
    }
}

}  // namespace

cudaError_t gdn_launch_group_norm(const GdnNormArgs &a, cudaStream_t s)
{
    const unsigned blocks = (unsigned)(a.rows * a.groups);
    if (a.dtype == 1)
        gdn_group_norm_kernel<__nv_bfloat16><<<blocks, kThreads, 0, s>>>(a);
    else
        gdn_group_norm_kernel<float><<<blocks, kThreads, 0, s>>>(a);
    return cudaGetLastError();
}

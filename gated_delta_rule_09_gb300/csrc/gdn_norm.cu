// Group norm of token rows, channels last, with an activation or a gate.
//
// Each run of width = channels / groups channels of a row is normalised by its
// own mean and variance (or mean square); y = act(u weight + bias) silu(gate).
// A few operations per element moved: bound by HBM, so every element is read
// once, in 16-byte words where rows allow it, and kept in registers between the
// statistics and the output.  A team of T lanes of a warp (width up to 8 words
// per lane), or a whole block, has one group of kRows rows: their loads are in
// flight together and share the weights.  The variance is taken about the mean
// in a second pass over the registers.
#include "gdn_layer.h"
#include "gdn_layer.cuh"

namespace {

using namespace gdn_layer;

constexpr int kThreads = 256;

// Sum over the team: T lanes of a warp, or the block.
template <bool BLOCK> __device__ __forceinline__ float team_sum(float v, int T, float *sh)
{
    if (!BLOCK) {
        for (int o = T >> 1; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        return v;
    }
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

__device__ __forceinline__ float finish(const GdnNormArgs &a, float u, float w, float b, bool gated, float gate)
{
    u = fmaf(u, w, b);
    if (a.act == GDN_ACT_SILU) u = silu(u);
    return gated ? u * silu(gate) : u;
}

// K words of VEC elements per thread and row, kRows rows per team.
template <typename E, int VEC, int K, int kRows, bool BLOCK>
__global__ void __launch_bounds__(kThreads) gdn_group_norm_kernel(const GdnNormArgs a, int T)
{
    __shared__ float sh[kThreads / 32];
    typedef typename Word<VEC * sizeof(E)>::type Vec;
    const int width = a.channels / a.groups;
    const int64_t teams = ((a.rows + kRows - 1) / kRows) * a.groups;
    const int64_t mine = BLOCK ? blockIdx.x : (int64_t)blockIdx.x * (kThreads / T) + threadIdx.x / T;
    const int64_t team = mine < teams ? mine : teams - 1;  // surplus teams repeat the last, and store nothing
    const int lane = BLOCK ? threadIdx.x : threadIdx.x & (T - 1);
    const int64_t row0 = team / a.groups * kRows;
    const int c0 = (int)(team % a.groups) * width;
    const bool gated = a.gate != nullptr;
    Vec xv[kRows][K], gv[kRows][K];
    int64_t at[kRows];  // rows past the end repeat the last, and store nothing
#pragma unroll
    for (int r = 0; r < kRows; ++r) at[r] = row0 + r < a.rows ? row0 + r : a.rows - 1;
#pragma unroll
    for (int r = 0; r < kRows; ++r)
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int i = (lane + k * T) * VEC;
            if (i >= width) continue;
            xv[r][k] = *reinterpret_cast<const Vec *>(static_cast<const E *>(a.x) + at[r] * a.ld_x + c0 + i);
            if (gated)
                gv[r][k] = *reinterpret_cast<const Vec *>(static_cast<const E *>(a.gate) + at[r] * a.ld_gate + c0 + i);
        }
    const float inv = 1.f / width;
    float mean[kRows], rstd[kRows];
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
        mean[r] = 0.f;
        if (!a.rms) {
#pragma unroll
            for (int k = 0; k < K; ++k) {
                if ((lane + k * T) * VEC >= width) continue;
                float x[VEC];
                widen(xv[r][k], x);
#pragma unroll
                for (int i = 0; i < VEC; ++i) mean[r] += x[i];
            }
            mean[r] = team_sum<BLOCK>(mean[r], T, sh) * inv;
        }
    }
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
        float q = 0.f;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            if ((lane + k * T) * VEC >= width) continue;
            float x[VEC];
            widen(xv[r][k], x);
#pragma unroll
            for (int i = 0; i < VEC; ++i) q = fmaf(x[i] - mean[r], x[i] - mean[r], q);
        }
        rstd[r] = rsqrtf(team_sum<BLOCK>(q, T, sh) * inv + a.eps);
    }
    if (mine >= teams) return;
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int i0 = (lane + k * T) * VEC;
        if (i0 >= width) continue;
        float w[VEC], b[VEC];
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            w[i] = 1.f;
            b[i] = 0.f;
        }
        if (a.weight) ld_vec<float, VEC>(a.weight + c0 + i0, w);
        if (a.bias) ld_vec<float, VEC>(a.bias + c0 + i0, b);
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            if (row0 + r >= a.rows) continue;
            float x[VEC], g[VEC];
            widen(xv[r][k], x);
            if (gated) widen(gv[r][k], g);
#pragma unroll
            for (int i = 0; i < VEC; ++i)
                x[i] = finish(a, (x[i] - mean[r]) * rstd[r], w[i], b[i], gated, gated ? g[i] : 0.f);
            st_vec<E, VEC>(static_cast<E *>(a.y) + at[r] * a.ld_y + c0 + i0, x);
        }
    }
}

// Groups wider than a block's registers: a block per group, three passes over it.
template <typename E>
__global__ void __launch_bounds__(kThreads) gdn_group_norm_wide_kernel(const GdnNormArgs a)
{
    __shared__ float sh[kThreads / 32];
    const int width = a.channels / a.groups;
    const int64_t row = blockIdx.x / a.groups;
    const int c0 = (int)(blockIdx.x % a.groups) * width;
    const E *x = static_cast<const E *>(a.x) + row * a.ld_x + c0;
    const E *gate = a.gate ? static_cast<const E *>(a.gate) + row * a.ld_gate + c0 : nullptr;
    E *y = static_cast<E *>(a.y) + row * a.ld_y + c0;
    float mean = 0.f, q = 0.f;
    if (!a.rms) {
        for (int i = threadIdx.x; i < width; i += kThreads) mean += to_f(x[i]);
        mean = team_sum<true>(mean, 0, sh) / width;
    }
    for (int i = threadIdx.x; i < width; i += kThreads) {
        const float v = to_f(x[i]) - mean;
        q = fmaf(v, v, q);
    }
    const float rstd = rsqrtf(team_sum<true>(q, 0, sh) / width + a.eps);
    for (int i = threadIdx.x; i < width; i += kThreads)
        y[i] = from_f<E>(finish(a, (to_f(x[i]) - mean) * rstd, a.weight ? a.weight[c0 + i] : 1.f,
                                a.bias ? a.bias[c0 + i] : 0.f, gate != nullptr, gate ? to_f(gate[i]) : 0.f));
}

template <typename E, int VEC, int K, int kRows, bool BLOCK>
cudaError_t launch(const GdnNormArgs &a, int T, cudaStream_t s)
{
    const int64_t teams = (a.rows + kRows - 1) / kRows * a.groups, per = BLOCK ? 1 : kThreads / T;
    const int64_t blocks = (teams + per - 1) / per;
    if (blocks > 0x7fffffff) return cudaErrorInvalidConfiguration;
    gdn_group_norm_kernel<E, VEC, K, kRows, BLOCK><<<(unsigned)blocks, kThreads, 0, s>>>(a, T);
    return cudaGetLastError();
}

// The team by the group's words: lanes of a warp up to 8 words each, then a
// block.  Four loads per thread and matrix in flight, from as many rows as that
// takes; few rows are spread one to a team.
template <typename E, int VEC> cudaError_t by_width(const GdnNormArgs &a, cudaStream_t s)
{
    const int words = (a.channels / a.groups + VEC - 1) / VEC;
    const bool few = a.rows * a.groups < 16384;
    if (words <= 32) {
        int T = 1;
        while (T < words) T *= 2;
        return few ? launch<E, VEC, 1, 1, false>(a, T, s) : launch<E, VEC, 1, 4, false>(a, T, s);
    }
    if (words <= 64) return few ? launch<E, VEC, 2, 1, false>(a, 32, s) : launch<E, VEC, 2, 2, false>(a, 32, s);
    if (words <= 128) return launch<E, VEC, 4, 1, false>(a, 32, s);
    if (words <= 256) return launch<E, VEC, 8, 1, false>(a, 32, s);
    if (words <= 512) return launch<E, VEC, 2, 1, true>(a, kThreads, s);
    if (words <= 1024) return launch<E, VEC, 4, 1, true>(a, kThreads, s);
    if (words <= 2048) return launch<E, VEC, 8, 1, true>(a, kThreads, s);
    const int64_t blocks = a.rows * a.groups;
    if (blocks > 0x7fffffff) return cudaErrorInvalidConfiguration;
    gdn_group_norm_wide_kernel<E><<<(unsigned)blocks, kThreads, 0, s>>>(a);
    return cudaGetLastError();
}

template <typename E> cudaError_t by_rows(const GdnNormArgs &a, cudaStream_t s)
{
    constexpr int V = 16 / sizeof(E);
    const bool words = a.channels / a.groups % V == 0 && a.ld_x % V == 0 && a.ld_y % V == 0 &&
                       (!a.gate || a.ld_gate % V == 0) && aligned16(a.x) && aligned16(a.y) && aligned16(a.gate) &&
                       aligned16(a.weight) && aligned16(a.bias);
    return words ? by_width<E, V>(a, s) : by_width<E, 1>(a, s);
}

}  // namespace

cudaError_t gdn_launch_group_norm(const GdnNormArgs &a, cudaStream_t s)
{
    return a.dtype == 1 ? by_rows<__nv_bfloat16>(a, s) : by_rows<float>(a, s);
}

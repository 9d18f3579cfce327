// Short causal depthwise convolution, over prompts and for single tokens.
//
//     y[t, c] = act(bias[c] + sum_j weight[c, j] x[t - (width - 1) + j, c])
//
// 2 width operations per 4 bytes (bf16) moved: bound by HBM.  Channels are
// independent and neighbouring tokens share width - 1 inputs, so a thread owns
// 16 bytes of channels (one wide access per token, a block's threads side by
// side along the row) and walks a tile of tokens with the last width - 1 inputs
// in registers: every input is loaded once, plus the width - 1 rows ahead of
// each tile.
#include "gdn_layer.h"
#include "gdn_layer.cuh"

namespace {

using namespace gdn_layer;

constexpr int kThreads = 128;
constexpr int kUnroll = 8;  // tokens loaded ahead of their use

template <int VEC, int W>
__device__ __forceinline__ void ld_params(const GdnConvArgs &a, int c0, float (&w)[W][VEC],
                                          float (&b)[VEC])
{
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
#pragma unroll
        for (int j = 0; j < W; ++j) w[j][i] = a.weight[(size_t)(c0 + i) * W + j];
        b[i] = a.bias ? a.bias[c0 + i] : 0.f;
    }
}

template <typename E, int VEC, int W>
__global__ void __launch_bounds__(kThreads)
    gdn_conv_fwd_kernel(const GdnConvArgs a, int tl, int tiles)
{
    Span s;
    if (!find_span(a.cu_seqlens, a.N, a.T, tl, blockIdx.x, tiles, a.status, s)) return;
    const int c0 = (blockIdx.y * kThreads + threadIdx.x) * VEC;
    if (c0 >= a.channels) return;
    const E *x = static_cast<const E *>(a.x) + s.row * a.ld_x + c0;
    E *y = static_cast<E *>(a.y) + s.row * a.ld_y + c0;
    const int t0 = s.tile * tl, t1 = min(s.len, t0 + tl);

    float win[W][VEC];  // win[j]: the input j - (W - 1) tokens from the current one; win[W-1] is current
    if (s.tile == 0) {
        // The state is read and written by this thread alone (whichever tile
        // the sequence ends in), so it may be updated in place.
        const int entry = state_entry(a.slots, s.n, a.pool, a.status);
        const E *in = static_cast<const E *>(a.state_in);
        const size_t at = entry < 0 ? 0 : (size_t)entry * (W - 1) * a.channels + c0;
#pragma unroll
        for (int j = 0; j < W - 1; ++j) {
            if (in && entry >= 0) {
                ld_vec<E, VEC>(in + at + (size_t)j * a.channels, win[j]);
            } else {
#pragma unroll
                for (int i = 0; i < VEC; ++i) win[j][i] = 0.f;
            }
        }
        if (a.state_out && entry >= 0) {
            E *out = static_cast<E *>(a.state_out);
#pragma unroll
            for (int j = 0; j < W - 1; ++j) {
                const int p = s.len - (W - 1) + j;
                float v[VEC];
                if (p >= 0) {
                    ld_vec<E, VEC>(x + p * a.ld_x, v);
                } else {  // fewer tokens than taps: the older state moves up
#pragma unroll
                    for (int k = 0; k < W - 1; ++k)
                        if (k == p + W - 1)
#pragma unroll
                            for (int i = 0; i < VEC; ++i) v[i] = win[k][i];
                }
                st_vec<E, VEC>(out + at + (size_t)j * a.channels, v);
            }
        }
    } else {  // a tile is longer than the taps, so these lie in the same sequence
#pragma unroll
        for (int j = 0; j < W - 1; ++j)
            ld_vec<E, VEC>(x + (int64_t)(t0 - (W - 1) + j) * a.ld_x, win[j]);
    }
    if (t0 >= t1) return;

    float w[W][VEC], b[VEC];
    ld_params<VEC, W>(a, c0, w, b);
    for (int t = t0; t < t1; t += kUnroll) {
        Pack<E, VEC> u[kUnroll];
#pragma unroll
        for (int k = 0; k < kUnroll; ++k)
            if (t + k < t1)
                u[k] = *reinterpret_cast<const Pack<E, VEC> *>(x + (int64_t)(t + k) * a.ld_x);
#pragma unroll
        for (int k = 0; k < kUnroll; ++k) {
            if (t + k >= t1) break;
            float r[VEC];
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                win[W - 1][i] = to_f(u[k].v[i]);
                r[i] = b[i];
#pragma unroll
                for (int j = 0; j < W; ++j) r[i] = fmaf(w[j][i], win[j][i], r[i]);
                if (a.act == GDN_ACT_SILU) r[i] = silu(r[i]);
#pragma unroll
                for (int j = 0; j < W - 1; ++j) win[j][i] = win[j + 1][i];
            }
            st_vec<E, VEC>(y + (int64_t)(t + k) * a.ld_y, r);
        }
    }
}

// One token per sequence: the state row group moves on by one input.
template <typename E, int VEC, int W>
__global__ void __launch_bounds__(kThreads) gdn_conv_step_kernel(const GdnConvArgs a)
{
    const int c0 = (blockIdx.y * kThreads + threadIdx.x) * VEC;
    if (c0 >= a.channels) return;
    const int n = blockIdx.x;
    float w[W][VEC], b[VEC], win[W][VEC];
    ld_params<VEC, W>(a, c0, w, b);
    const int entry = state_entry(a.slots, n, a.pool, a.status);
    const E *in = static_cast<const E *>(a.state_in);
    const size_t at = entry < 0 ? 0 : (size_t)entry * (W - 1) * a.channels + c0;
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
        if (in && entry >= 0) {
            ld_vec<E, VEC>(in + at + (size_t)j * a.channels, win[j]);
        } else {
#pragma unroll
            for (int i = 0; i < VEC; ++i) win[j][i] = 0.f;
        }
    }
    ld_vec<E, VEC>(static_cast<const E *>(a.x) + n * a.ld_x + c0, win[W - 1]);
    float r[VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
        r[i] = b[i];
#pragma unroll
        for (int j = 0; j < W; ++j) r[i] = fmaf(w[j][i], win[j][i], r[i]);
        if (a.act == GDN_ACT_SILU) r[i] = silu(r[i]);
    }
    st_vec<E, VEC>(static_cast<E *>(a.y) + n * a.ld_y + c0, r);
    if (entry >= 0) {
        E *out = static_cast<E *>(a.state_out);
#pragma unroll
        for (int j = 0; j < W - 1; ++j)
            st_vec<E, VEC>(out + at + (size_t)j * a.channels, win[j + 1]);
    }
}

template <typename E>
bool vector_rows(const GdnConvArgs &a)
{
    constexpr int V = 16 / sizeof(E);
    return a.channels % V == 0 && a.ld_x % V == 0 && a.ld_y % V == 0 && aligned16(a.x) &&
           aligned16(a.y) && aligned16(a.state_in) && aligned16(a.state_out);
}

template <typename E, int VEC, int W>
cudaError_t fwd(const GdnConvArgs &a, cudaStream_t s)
{
    const int blocks = (a.channels / VEC + (a.channels % VEC != 0) + kThreads - 1) / kThreads;
    const int tl = 32;
    const int tiles = a.T > tl ? (a.T + tl - 1) / tl : 1;
    const int64_t slots = a.cu_seqlens ? (int64_t)a.T / tl + a.N : (int64_t)a.N * tiles;
    gdn_conv_fwd_kernel<E, VEC, W><<<dim3((unsigned)slots, blocks), kThreads, 0, s>>>(a, tl, tiles);
    return cudaGetLastError();
}

template <typename E, int VEC, int W>
cudaError_t step(const GdnConvArgs &a, cudaStream_t s)
{
    const int blocks = (a.channels / VEC + (a.channels % VEC != 0) + kThreads - 1) / kThreads;
    gdn_conv_step_kernel<E, VEC, W><<<dim3(a.N, blocks), kThreads, 0, s>>>(a);
    return cudaGetLastError();
}

template <bool STEP, typename E, int W>
cudaError_t by_vector(const GdnConvArgs &a, cudaStream_t s)
{
    constexpr int V = 16 / sizeof(E);
    if (vector_rows<E>(a)) return STEP ? step<E, V, W>(a, s) : fwd<E, V, W>(a, s);
    return STEP ? step<E, 1, W>(a, s) : fwd<E, 1, W>(a, s);
}

template <bool STEP, typename E>
cudaError_t by_width(const GdnConvArgs &a, cudaStream_t s)
{
    switch (a.width) {
    case 1: return by_vector<STEP, E, 1>(a, s);
    case 2: return by_vector<STEP, E, 2>(a, s);
    case 3: return by_vector<STEP, E, 3>(a, s);
    case 4: return by_vector<STEP, E, 4>(a, s);
    case 5: return by_vector<STEP, E, 5>(a, s);
    case 6: return by_vector<STEP, E, 6>(a, s);
    case 7: return by_vector<STEP, E, 7>(a, s);
    default: return by_vector<STEP, E, 8>(a, s);
    }
}

}  // namespace

cudaError_t gdn_launch_conv_fwd(const GdnConvArgs &a, cudaStream_t s)
{
    return a.dtype == 1 ? by_width<false, __nv_bfloat16>(a, s) : by_width<false, float>(a, s);
}

cudaError_t gdn_launch_conv_step(const GdnConvArgs &a, cudaStream_t s)
{
    return a.dtype == 1 ? by_width<true, __nv_bfloat16>(a, s) : by_width<true, float>(a, s);
}

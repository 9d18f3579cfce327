// Selective state space scan, over prompts and for single tokens.
//
// Per channel c with d_state fp32 states, token by token:
//
//     h[s] = exp(d A[c, s]) h[s] + d B[t, s] x        y = sum_s C[t, s] h[s] + D x
//
// A lane holds four consecutive states of one channel, the LPC = 1..32 lanes of
// a channel (d_state padded to 4 LPC) are neighbours, and their partial sums of
// y meet in a butterfly.  exp is 2^(d A log2 e).
#include "gdn_layer.h"
#include "gdn_layer.cuh"

namespace {

using namespace gdn_layer;

constexpr int kThreads = 128;
constexpr float kLog2e = 1.4426950408889634f;

// Four consecutive states (zeros past the end).
__device__ __forceinline__ void ld_state(const float *p, int s0, int ds, float (&h)[4])
{
#pragma unroll
    for (int j = 0; j < 4; ++j) h[j] = s0 + j < ds ? p[s0 + j] : 0.f;
}

__device__ __forceinline__ void st_state(float *p, int s0, int ds, const float (&h)[4])
{
#pragma unroll
    for (int j = 0; j < 4; ++j)
        if (s0 + j < ds) p[s0 + j] = h[j];
}

template <typename E>
__device__ __forceinline__ void ld_bc(const E *p, int s0, int ds, float (&h)[4])
{
#pragma unroll
    for (int j = 0; j < 4; ++j) h[j] = s0 + j < ds ? to_f(p[s0 + j]) : 0.f;
}

// What a launch over tiles of tokens does.  A call whose sequences are one
// tile each is kWhole.  Cut into pieces, kPieces finds every piece's end state
// (the first from the sequence's own state, the others from zero) and the sum
// of its d, and kOutputs starts each piece from the states chained up to it:
// a run of tokens takes h to exp(A sum d) h + (its end state from zero).  The
// last piece's end state is not needed, and its place keeps the sequence's
// start state instead: kOutputs writes the final state while the first piece
// may still be starting, so in place that piece cannot read it from the pool.
enum Mode { kWhole, kPieces, kOutputs };

template <typename E, int LPC, int MODE>
__global__ void __launch_bounds__(kThreads)
    gdn_ssm_fwd_kernel(const GdnSsmArgs a, int tl, int tiles)
{
    Span s;
    if (!find_span(a.cu_seqlens, a.N, a.T, tl, blockIdx.x, tiles, a.status, s)) return;
    const int pieces = s.len > tl ? (s.len + tl - 1) / tl : 1;
    if (MODE == kPieces && s.tile == pieces - 1) return;
    const int c = blockIdx.y * (kThreads / LPC) + threadIdx.x / LPC;
    const bool live = c < a.channels;
    const int cc = live ? c : a.channels - 1;
    const int s0 = 4 * (threadIdx.x % LPC), ds = a.d_state;
    const int g = cc / (a.channels / a.groups);
    const int entry = state_entry(a.slots, s.n, a.pool, a.status);
    const int64_t slot0 = (int64_t)blockIdx.x - s.tile;  // the sequence's first piece
    float A[4], h[4] = {0.f, 0.f, 0.f, 0.f};
    ld_state(a.A + (size_t)cc * ds, s0, ds, A);
#pragma unroll
    for (int j = 0; j < 4; ++j) A[j] *= kLog2e;
    const size_t at = ((size_t)(entry < 0 ? 0 : entry) * a.channels + cc) * ds;
    auto piece = [&](int64_t slot) { return a.piece_state + ((size_t)slot * a.channels + cc) * ds; };
    if (MODE == kOutputs && pieces > 1) {
        ld_state(piece(s.tile == 0 ? slot0 + pieces - 1 : slot0), s0, ds, h);
        for (int k = 1; k < s.tile; ++k) {
            const float sum = a.piece_delta[(size_t)(slot0 + k) * a.channels + cc];
            float e[4];
            ld_state(piece(slot0 + k), s0, ds, e);
#pragma unroll
            for (int j = 0; j < 4; ++j) h[j] = fmaf(ex2(sum * A[j]), h[j], e[j]);
        }
    } else if (s.tile == 0 && a.state_in && entry >= 0) {
        ld_state(a.state_in + at, s0, ds, h);
    }
    if (MODE == kPieces && s.tile == 0 && live) st_state(piece(slot0 + pieces - 1), s0, ds, h);
    const float bias = a.delta_bias ? a.delta_bias[cc] : 0.f, D = a.D ? a.D[cc] : 0.f;
    const int t0 = s.tile * tl, t1 = min(s.len, t0 + tl);
    float sum = 0.f;
    for (int t = t0; t < t1; ++t) {
        const int64_t r = s.row + t;
        float d = to_f(static_cast<const E *>(a.delta)[r * a.ld_delta + cc]) + bias;
        if (a.softplus) d = softplus(d);
        sum += d;
        const float x = to_f(static_cast<const E *>(a.x)[r * a.ld_x + cc]);
        float B[4], C[4], y = 0.f;
        ld_bc(static_cast<const E *>(a.Bm) + r * a.ld_b + (size_t)g * ds, s0, ds, B);
        ld_bc(static_cast<const E *>(a.Cm) + r * a.ld_c + (size_t)g * ds, s0, ds, C);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            h[j] = fmaf(ex2(d * A[j]), h[j], d * x * B[j]);
            y = fmaf(C[j], h[j], y);
        }
        if (MODE == kPieces) continue;
#pragma unroll
        for (int o = 1; o < LPC; o <<= 1) y += __shfl_xor_sync(0xffffffffu, y, o);
        if (live && threadIdx.x % LPC == 0) {
            y = fmaf(D, x, y);
            if (a.z) y *= silu(to_f(static_cast<const E *>(a.z)[r * a.ld_z + cc]));
            static_cast<E *>(a.y)[r * a.ld_y + cc] = from_f<E>(y);
        }
    }
    if (!live) return;
    if (MODE == kPieces) {
        st_state(piece(blockIdx.x), s0, ds, h);
        if (threadIdx.x % LPC == 0) a.piece_delta[(size_t)blockIdx.x * a.channels + cc] = sum;
    } else if (s.tile == pieces - 1 && a.state_out && entry >= 0) {
        st_state(a.state_out + at, s0, ds, h);
    }
}

template <typename E, int LPC>
__global__ void __launch_bounds__(kThreads) gdn_ssm_step_kernel(const GdnSsmArgs a)
{
    const int c = blockIdx.y * (kThreads / LPC) + threadIdx.x / LPC;
    const bool live = c < a.channels;
    const int cc = live ? c : a.channels - 1, n = blockIdx.x;
    const int s0 = 4 * (threadIdx.x % LPC), ds = a.d_state;
    const int g = cc / (a.channels / a.groups);
    const int entry = state_entry(a.slots, n, a.pool, a.status);
    float A[4], h[4] = {0.f, 0.f, 0.f, 0.f}, B[4], C[4], y = 0.f;
    ld_state(a.A + (size_t)cc * ds, s0, ds, A);
    const size_t at = ((size_t)(entry < 0 ? 0 : entry) * a.channels + cc) * ds;
    if (a.state_in && entry >= 0) ld_state(a.state_in + at, s0, ds, h);
    float d = to_f(static_cast<const E *>(a.delta)[n * a.ld_delta + cc]) +
              (a.delta_bias ? a.delta_bias[cc] : 0.f);
    if (a.softplus) d = softplus(d);
    const float x = to_f(static_cast<const E *>(a.x)[n * a.ld_x + cc]);
    ld_bc(static_cast<const E *>(a.Bm) + n * a.ld_b + (size_t)g * ds, s0, ds, B);
    ld_bc(static_cast<const E *>(a.Cm) + n * a.ld_c + (size_t)g * ds, s0, ds, C);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        h[j] = fmaf(ex2(d * (A[j] * kLog2e)), h[j], d * x * B[j]);
        y = fmaf(C[j], h[j], y);
    }
#pragma unroll
    for (int o = 1; o < LPC; o <<= 1) y += __shfl_xor_sync(0xffffffffu, y, o);
    if (live && threadIdx.x % LPC == 0) {
        y = fmaf(a.D ? a.D[cc] : 0.f, x, y);
        if (a.z) y *= silu(to_f(static_cast<const E *>(a.z)[n * a.ld_z + cc]));
        static_cast<E *>(a.y)[n * a.ld_y + cc] = from_f<E>(y);
    }
    if (entry >= 0 && live) st_state(a.state_out + at, s0, ds, h);
}

template <bool STEP, typename E, int LPC>
cudaError_t launch(const GdnSsmArgs &a, cudaStream_t s)
{
    const int per = kThreads / LPC, blocks = (a.channels + per - 1) / per;
    if (STEP) {
        gdn_ssm_step_kernel<E, LPC><<<dim3(a.N, blocks), kThreads, 0, s>>>(a);
    } else if (a.segment) {
        const int tiles = (a.T + a.segment - 1) / a.segment;
        const dim3 grid((unsigned)a.pieces, blocks);
        gdn_ssm_fwd_kernel<E, LPC, kPieces><<<grid, kThreads, 0, s>>>(a, a.segment, tiles);
        gdn_ssm_fwd_kernel<E, LPC, kOutputs><<<grid, kThreads, 0, s>>>(a, a.segment, tiles);
    } else {
        const int tl = a.T > 0 ? a.T : 1;
        const dim3 grid(a.cu_seqlens ? a.T / tl + a.N : a.N, blocks);
        gdn_ssm_fwd_kernel<E, LPC, kWhole><<<grid, kThreads, 0, s>>>(a, tl, 1);
    }
    return cudaGetLastError();
}

template <bool STEP, typename E>
cudaError_t by_state(const GdnSsmArgs &a, cudaStream_t s)
{
    if (a.d_state <= 4) return launch<STEP, E, 1>(a, s);
    if (a.d_state <= 8) return launch<STEP, E, 2>(a, s);
    if (a.d_state <= 16) return launch<STEP, E, 4>(a, s);
    if (a.d_state <= 32) return launch<STEP, E, 8>(a, s);
    if (a.d_state <= 64) return launch<STEP, E, 16>(a, s);
    return launch<STEP, E, 32>(a, s);
}

}  // namespace

void gdn_ssm_plan(int N, int T, int channels, int d_state, bool packed, int asked, int *segment,
                  int64_t *piece_slots)
{
    *segment = 0;
    *piece_slots = 0;
    if (asked <= 0) return;
    const int64_t seg = ((int64_t)asked + 63) / 64 * 64;
    if (seg >= T) return;
    *segment = (int)seg;
    *piece_slots = packed ? T / seg + N : N * ((T + seg - 1) / seg);
}

cudaError_t gdn_launch_ssm_fwd(const GdnSsmArgs &a, cudaStream_t s, int *launches)
{
    *launches = a.segment ? 2 : 1;
    return a.dtype == 1 ? by_state<false, __nv_bfloat16>(a, s) : by_state<false, float>(a, s);
}

cudaError_t gdn_launch_ssm_step(const GdnSsmArgs &a, cudaStream_t s)
{
    return a.dtype == 1 ? by_state<true, __nv_bfloat16>(a, s) : by_state<true, float>(a, s);
}

// Norms around a block in one pass: the norm after it, its gate and scale, the
// residual sum, and the norm before the next block.
//
//     u = y                          or norm(y) post_weight + post_bias
//     r = residual_scale residual + scale u act(gate)       -> residual_out
//     h = norm(r) pre_weight + pre_bias                     -> h
//
// Bound by HBM: y, gate and residual are read once, r and h written once; r stays
// in registers, in fp32, for the second norm.  A team of T lanes of a warp, or a
// whole block, keeps to one row at a time (kRows of them for fewer barriers) and
// walks down the rows with the next ones in flight.  Variances are taken about
// the mean in a second pass over the registers.  The parameters, up to five fp32
// arrays, would cost 40 registers a word: they are read for each turn instead,
// from L1, which keeps them for all teams of an SM.
#pragma once

#include "gdn_layer.cuh"
#include "gdn_layer.h"
#include "gdn_team.cuh"

namespace {

using namespace gdn_layer;

constexpr int kTeams = 256;  // threads of a block of teams

template <int VEC> struct Pairs {
    static constexpr int P = VEC > 1 ? VEC / 2 : 1;  // a lone element is half a pair
    f32x2 v[P];

    __device__ __forceinline__ void set(const float (&f)[VEC])
    {
#pragma unroll
        for (int i = 0; i < P; ++i) v[i] = pack2(f[VEC > 1 ? 2 * i : 0], VEC > 1 ? f[VEC > 1 ? 2 * i + 1 : 0] : 0.f);
    }
    __device__ __forceinline__ void get(float (&f)[VEC]) const
    {
#pragma unroll
        for (int i = 0; i < P; ++i) {
            float lo, hi;
            unpack2(v[i], lo, hi);
            f[VEC > 1 ? 2 * i : 0] = lo;
            if (VEC > 1) f[VEC > 1 ? 2 * i + 1 : 0] = hi;
        }
    }
    __device__ __forceinline__ float sum() const
    {
        f32x2 s = v[0];
#pragma unroll
        for (int i = 1; i < P; ++i) s = add2(s, v[i]);
        float lo, hi;
        unpack2(s, lo, hi);
        return VEC > 1 ? lo + hi : lo;
    }
    __device__ __forceinline__ float squares() const
    {
        f32x2 s = mul2(v[0], v[0]);
#pragma unroll
        for (int i = 1; i < P; ++i) s = fma2(v[i], v[i], s);
        float lo, hi;
        unpack2(s, lo, hi);
        return VEC > 1 ? lo + hi : lo;
    }
};

// VEC elements as they lie in memory: loads that are still in flight keep to the
// registers that the bytes need.
template <typename T, int VEC> struct Raw {
    static constexpr int N = VEC * sizeof(T) > 16 ? 2 : 1, PER = VEC / N;
    typedef typename Word<PER * sizeof(T)>::type W;
    W w[N];

    __device__ __forceinline__ void load(const T *p)
    {
#pragma unroll
        for (int i = 0; i < N; ++i) w[i] = *reinterpret_cast<const W *>(p + i * PER);
    }
    __device__ __forceinline__ void to(Pairs<VEC> &v) const
    {
        float f[VEC];
#pragma unroll
        for (int i = 0; i < N; ++i) {
            float x[PER];
            widen(w[i], x);
#pragma unroll
            for (int j = 0; j < PER; ++j) f[i * PER + j] = x[j];
        }
        v.set(f);
    }
};

// A gate's factor: sigmoid(g) or g sigmoid(g).
__device__ __forceinline__ float gate_of(float g, int act)
{
    const float s = rcp(1.f + ex2(-kLog2e * g));
    return act == GDN_ACT_SILU ? g * s : act == GDN_ACT_SIGMOID ? s : g;
}

// E: type of y, gate and h; R: of the residual stream.
template <typename E, typename R, int VEC, int K, int kRows, int BLOCK>
__global__ void __launch_bounds__(BLOCK ? BLOCK : kTeams) gdn_block_norm_kernel(const GdnBlockNormArgs a, int T, int walkers)
{
    __shared__ __align__(16) float sh[BLOCK ? 2 : 1][kRows][kTeamWarps];
    TeamSum<BLOCK, kRows> team_sum = {sh, 0};
    typedef Pairs<VEC> V;
    constexpr int P = V::P;
    const int width = a.channels;
    const int64_t mine = BLOCK ? blockIdx.x : (int64_t)blockIdx.x * (kTeams / T) + threadIdx.x / T;
    const bool live = mine < walkers;  // surplus teams walk with the first, and store nothing
    const int64_t team = live ? mine : 0;
    const int lane = BLOCK ? threadIdx.x : threadIdx.x & (T - 1);
    const E *y = static_cast<const E *>(a.y), *gate = static_cast<const E *>(a.gate);
    const R *res = static_cast<const R *>(a.residual);
    Raw<E, VEC> yv[kRows][K], gv[kRows][K];
    Raw<R, VEC> rv[kRows][K];
    int at[K];
    bool has[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
        at[k] = (lane + k * T) * VEC;
        has[k] = at[k] < width;
    }
#pragma unroll
    for (int r = 0; r < kRows; ++r)
#pragma unroll
        for (int k = 0; k < K; ++k) {
            yv[r][k] = gv[r][k] = Raw<E, VEC>();
            rv[r][k] = Raw<R, VEC>();
        }
    auto load = [&](int64_t row) {
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            if (row + r >= a.rows) break;
#pragma unroll
            for (int k = 0; k < K; ++k) {
                if (!has[k]) continue;
                yv[r][k].load(y + (row + r) * a.ld_y + at[k]);
                if (gate) gv[r][k].load(gate + (row + r) * a.ld_gate + at[k]);
                if (res) rv[r][k].load(res + (row + r) * a.ld_residual + at[k]);
            }
        }
    };
    const float inv = 1.f / width;
    // (x - mean) / sqrt(var + eps) of the rows, zeros past the width
    auto normalise = [&](V (&c)[kRows][K]) {
        float s[kRows];
        if (!a.rms) {
#pragma unroll
            for (int r = 0; r < kRows; ++r) {
                s[r] = 0.f;
#pragma unroll
                for (int k = 0; k < K; ++k) s[r] += c[r][k].sum();
            }
            team_sum(s, T);
#pragma unroll
            for (int r = 0; r < kRows; ++r)
#pragma unroll
                for (int k = 0; k < K; ++k)
                    if (has[k])
#pragma unroll
                        for (int i = 0; i < P; ++i) c[r][k].v[i] = add2(c[r][k].v[i], pack2(-s[r] * inv, VEC > 1 ? -s[r] * inv : 0.f));
        }
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            s[r] = 0.f;
#pragma unroll
            for (int k = 0; k < K; ++k) s[r] += c[r][k].squares();
        }
        team_sum(s, T);
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            const f32x2 f = dup2(rsqrtf(s[r] * inv + a.eps));
#pragma unroll
            for (int k = 0; k < K; ++k)
#pragma unroll
                for (int i = 0; i < P; ++i) c[r][k].v[i] = mul2(c[r][k].v[i], f);
        }
    };
    // c weight + bias, either of them optional
    auto affine = [&](V (&c)[kRows][K], const float *weight, const float *bias) {
#pragma unroll
        for (int k = 0; k < K; ++k) {
            if (!has[k]) continue;
            float f[VEC];
            V w;
            if (weight) {
                ld_vec<float, VEC>(weight + at[k], f);
                w.set(f);
#pragma unroll
                for (int r = 0; r < kRows; ++r)
#pragma unroll
                    for (int i = 0; i < P; ++i) c[r][k].v[i] = mul2(c[r][k].v[i], w.v[i]);
            }
            if (bias) {
                ld_vec<float, VEC>(bias + at[k], f);
                w.set(f);
#pragma unroll
                for (int r = 0; r < kRows; ++r)
#pragma unroll
                    for (int i = 0; i < P; ++i) c[r][k].v[i] = add2(c[r][k].v[i], w.v[i]);
            }
        }
    };
    const int64_t stride = (int64_t)walkers * kRows;
    load(team * kRows);
    // the same number of turns for every team: teams of a warp shuffle together
    int64_t row = team * kRows;
    for (int64_t ahead = a.rows; ahead > 0; ahead -= stride, row += stride) {
        V c[kRows][K], g[kRows][K], x[kRows][K];
#pragma unroll
        for (int r = 0; r < kRows; ++r)
#pragma unroll
            for (int k = 0; k < K; ++k) {
                yv[r][k].to(c[r][k]);
                gv[r][k].to(g[r][k]);
                rv[r][k].to(x[r][k]);
            }
        load(row + stride);
        if (a.post) {
            normalise(c);
            affine(c, a.post_weight, a.post_bias);
        }
        affine(c, a.scale, nullptr);
#pragma unroll
        for (int r = 0; r < kRows; ++r)
#pragma unroll
            for (int k = 0; k < K; ++k) {
                if (gate) {
                    float f[VEC];
                    g[r][k].get(f);
#pragma unroll
                    for (int i = 0; i < VEC; ++i) f[i] = gate_of(f[i], a.gate_act);
                    g[r][k].set(f);
#pragma unroll
                    for (int i = 0; i < P; ++i) c[r][k].v[i] = mul2(c[r][k].v[i], g[r][k].v[i]);
                }
                if (res)
#pragma unroll
                    for (int i = 0; i < P; ++i) c[r][k].v[i] = fma2(x[r][k].v[i], dup2(a.residual_scale), c[r][k].v[i]);
                if (live && row + r < a.rows && has[k]) {
                    float f[VEC];
                    c[r][k].get(f);
                    st_vec<R, VEC>(static_cast<R *>(a.residual_out) + (row + r) * a.ld_residual_out + at[k], f);
                }
            }
        if (!a.h) continue;
        normalise(c);
        affine(c, a.pre_weight, a.pre_bias);
#pragma unroll
        for (int r = 0; r < kRows; ++r)
#pragma unroll
            for (int k = 0; k < K; ++k)
                if (live && row + r < a.rows && has[k]) {
                    float f[VEC];
                    c[r][k].get(f);
                    st_vec<E, VEC>(static_cast<E *>(a.h) + (row + r) * a.ld_h + at[k], f);
                }
    }
}

// Rows wider than a block's registers: a block per row, the sum formed anew for
// each of the passes over it, the later ones from L1 and L2.  Only the last one
// writes, each element after it has been read: outputs may be inputs.
template <typename E, typename R>
__global__ void __launch_bounds__(512) gdn_block_norm_wide_kernel(const GdnBlockNormArgs a)
{
    constexpr int kThreads = 512;
    __shared__ __align__(16) float sh[2][1][kTeamWarps];
    TeamSum<kThreads, 1> team_sum = {sh, 0};
    const int width = a.channels;
    const int64_t row = blockIdx.x;
    const E *y = static_cast<const E *>(a.y) + row * a.ld_y;
    const E *gate = a.gate ? static_cast<const E *>(a.gate) + row * a.ld_gate : nullptr;
    const R *res = a.residual ? static_cast<const R *>(a.residual) + row * a.ld_residual : nullptr;
    R *out = static_cast<R *>(a.residual_out) + row * a.ld_residual_out;
    E *h = a.h ? static_cast<E *>(a.h) + row * a.ld_h : nullptr;
    auto moments = [&](auto value, float &mean, float &rstd) {
        float s[1] = {0.f};
        mean = 0.f;
        if (!a.rms) {
            for (int i = threadIdx.x; i < width; i += kThreads) s[0] += value(i);
            team_sum(s, kThreads);
            mean = s[0] / width;
        }
        s[0] = 0.f;
        for (int i = threadIdx.x; i < width; i += kThreads) {
            const float v = value(i) - mean;
            s[0] = fmaf(v, v, s[0]);
        }
        team_sum(s, kThreads);
        rstd = rsqrtf(s[0] / width + a.eps);
    };
    float mean = 0.f, rstd = 1.f;
    if (a.post) moments([&](int i) { return to_f(y[i]); }, mean, rstd);
    auto sum = [&](int i) {
        float u = to_f(y[i]);
        if (a.post) u = (u - mean) * rstd * (a.post_weight ? a.post_weight[i] : 1.f) + (a.post_bias ? a.post_bias[i] : 0.f);
        if (a.scale) u *= a.scale[i];
        if (gate) u *= gate_of(to_f(gate[i]), a.gate_act);
        return res ? fmaf(to_f(res[i]), a.residual_scale, u) : u;
    };
    float pmean = 0.f, prstd = 1.f;
    if (h) moments(sum, pmean, prstd);
    for (int i = threadIdx.x; i < width; i += kThreads) {
        const float r = sum(i);
        out[i] = from_f<R>(r);
        if (h) h[i] = from_f<E>((r - pmean) * prstd * (a.pre_weight ? a.pre_weight[i] : 1.f) + (a.pre_bias ? a.pre_bias[i] : 0.f));
    }
}

template <typename E, typename R, int VEC, int K, int kRows, int BLOCK>
cudaError_t launch(const GdnBlockNormArgs &a, int T, cudaStream_t s)
{
    // As many teams as are resident at once, or as there are rows for.
    static int fit = 0;  // blocks of this kind at once; the same for every caller
    constexpr int threads = BLOCK ? BLOCK : kTeams;
    const int per = threads / T;
    if (!fit) {
        int blocks = 0;
        const cudaError_t e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(
            &blocks, gdn_block_norm_kernel<E, R, VEC, K, kRows, BLOCK>, threads, 0);
        if (e != cudaSuccess) return e;
        fit = gdn_ssm_sms() * (blocks > 0 ? blocks : 1);
    }
    const int64_t turns = (a.rows + kRows - 1) / kRows;
    int64_t walkers = (int64_t)fit * per;
    if (walkers > turns) walkers = turns;
    // equal shares: the last turn is as full as the others
    const int64_t each = (turns + walkers - 1) / walkers;
    walkers = (turns + each - 1) / each;
    const int64_t blocks = (walkers + per - 1) / per;
    gdn_block_norm_kernel<E, R, VEC, K, kRows, BLOCK><<<(unsigned)blocks, threads, 0, s>>>(a, T, (int)walkers);
    return cudaGetLastError();
}

// The team by the row's words.  us, bf16, gated and scaled, both norms, a team of T
// threads, K words each, R rows at a time as T x K x R.
// 16-byte words: 16 384 rows of 4096 256 x 2 x 1 119 (5.6 TB/s), 128 x 4 x 1 125, 512 x
// 1 x 2 133, 256 x 2 x 2 148; 32 768 rows of 1024 128 x 1 x 2 57 (5.9 TB/s), 64 x 2 x 1
// 57; 8192 rows of 8192 512 x 2 x 1 145, 256 x 4 x 1 189; 5000 rows of 12 288 512 x 3 x 1
// 142, element by element from memory 521.  8192 rows of 2048 with an fp32 stream, mean
// and variance: 256 x 1 x 2 45 (4.5 TB/s), 256 x 1 x 1 47, 128 x 2 x 1 47.
// Single elements, 16 384 rows: of 1925 512 x 4 x 1 229, 256 x 8 x 1 262; of 4093 from
// memory 448, 512 x 8 x 1 545 (issue slots).
template <typename E, typename R, int VEC> cudaError_t by_width(const GdnBlockNormArgs &a, cudaStream_t s)
{
    const int words = (a.channels + VEC - 1) / VEC;
    if (words <= 32) {
        int T = 1;
        while (T < words) T *= 2;
        return launch<E, R, VEC, 1, 2, 0>(a, T, s);
    }
    if (words <= 64) return launch<E, R, VEC, 1, 2, 64>(a, 64, s);
    if (words <= 128) return launch<E, R, VEC, 1, 2, 128>(a, 128, s);
    if (words <= 256) return launch<E, R, VEC, 1, 2, 256>(a, 256, s);
    if (words <= 512) return launch<E, R, VEC, 2, 1, 256>(a, 256, s);
    if (words <= 1024) return launch<E, R, VEC, 2, 1, 512>(a, 512, s);
    if (words <= 1536) return launch<E, R, VEC, 3, 1, 512>(a, 512, s);
    if (words <= 2048) return launch<E, R, VEC, 4, 1, 512>(a, 512, s);
    if (a.rows > 0x7fffffff) return cudaErrorInvalidConfiguration;
    gdn_block_norm_wide_kernel<E, R><<<(unsigned)a.rows, 512, 0, s>>>(a);
    return cudaGetLastError();
}

// Whether all rows and the parameters can be read in words of V elements.
template <typename E, typename R> bool words_of(const GdnBlockNormArgs &a, int V)
{
    const size_t al = V * sizeof(E), ar = V * sizeof(R) > 16 ? 16 : V * sizeof(R), ap = V == 2 ? 8 : 16;
    return a.channels % V == 0 && a.ld_y % V == 0 && (!a.gate || a.ld_gate % V == 0) &&
           (!a.residual || a.ld_residual % V == 0) && a.ld_residual_out % V == 0 && (!a.h || a.ld_h % V == 0) &&
           aligned_to(a.y, al) && aligned_to(a.gate, al) && aligned_to(a.h, al) && aligned_to(a.residual, ar) &&
           aligned_to(a.residual_out, ar) && aligned_to(a.post_weight, ap) && aligned_to(a.post_bias, ap) &&
           aligned_to(a.pre_weight, ap) && aligned_to(a.pre_bias, ap) && aligned_to(a.scale, ap);
}

template <typename E, typename R> cudaError_t block_norm(const GdnBlockNormArgs &a, cudaStream_t s)
{
    constexpr int V = 16 / sizeof(E);
    return words_of<E, R>(a, V)   ? by_width<E, R, V>(a, s)
           : words_of<E, R>(a, 2) ? by_width<E, R, 2>(a, s)
                                  : by_width<E, R, 1>(a, s);
}

}  // namespace

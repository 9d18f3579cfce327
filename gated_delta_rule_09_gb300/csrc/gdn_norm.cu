// Group norm of token rows, channels last, with an activation or a gate.
//
// Each run of width = channels / groups channels of a row is normalised by its
// own mean and variance (or mean square); y = act(u weight + bias) silu(gate).
// A few operations per element moved: bound by HBM, so every element is read
// once, in words of 16 bytes, of two elements or of one as rows allow, and kept in
// registers between the statistics and the output.  A team of T lanes of a warp,
// or a whole block, keeps to one group, whose weights it holds, and walks down
// the rows, kRows at a time; the next rows are in flight while these are
// normalised.  The variance is taken about the mean in a second pass over the
// registers.
//
// Measured, bf16, gated, 16 384 rows of 2048 channels: 16 groups 34 us, 2 groups
// 34 us, one group 35 us (5.7 to 6.0 TB/s); fp32 62 us, 6.4 TB/s.  16 groups with
// the butterflies in a loop over the team's size and row offsets multiplied out
// for each access: 37 us, 72 % of the issue slots.  Heads of 130 (words of two)
// 53 us; heads of 129, element by element, 81 us: issue slots.
#include "gdn_layer.h"
#include "gdn_layer.cuh"

namespace {

using namespace gdn_layer;

constexpr int kThreads = 256;

// Sums over the team, T lanes of a warp or the block, of R values at a time.  A
// block's warps meet in one of two buffers: by the time one is filled again, the
// barrier of the sum between has seen everybody through reading it.
template <int BLOCK, int R> struct TeamSum {
    float (*sh)[R][kThreads / 32];
    int turn;

    __device__ __forceinline__ void operator()(float (&v)[R], int T)
    {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            if (!BLOCK && o >= T) continue;
#pragma unroll
            for (int r = 0; r < R; ++r) v[r] += __shfl_xor_sync(0xffffffffu, v[r], o);
        }
        if constexpr (BLOCK != 0) {
            if ((threadIdx.x & 31) == 0)
#pragma unroll
                for (int r = 0; r < R; ++r) sh[turn][r][threadIdx.x >> 5] = v[r];
            __syncthreads();
#pragma unroll
            for (int r = 0; r < R; ++r) {
                v[r] = 0.f;
#pragma unroll
                for (int i = 0; i < BLOCK / 32; ++i) v[r] += sh[turn][r][i];
            }
            turn ^= 1;
        }
    }
};

// K words of VEC elements per thread and row, kRows rows at a time.  `walkers`
// teams share the rows of a group.
template <typename E, int VEC, int K, int kRows, int BLOCK>
__global__ void __launch_bounds__(BLOCK ? BLOCK : kThreads) gdn_group_norm_kernel(const GdnNormArgs a, int T, int walkers)
{
    __shared__ __align__(16) float sh[BLOCK ? 2 : 1][kRows][kThreads / 32];
    TeamSum<BLOCK, kRows> team_sum = {sh, 0};
    typedef typename Word<VEC * sizeof(E)>::type Vec;
    constexpr int P = VEC > 1 ? VEC / 2 : 1;  // pairs, for packed arithmetic; a lone element is half a pair
    const int width = a.channels / a.groups;
    const int64_t mine = BLOCK ? blockIdx.x : (int64_t)blockIdx.x * (kThreads / T) + threadIdx.x / T;
    const bool live = mine < (int64_t)walkers * a.groups;  // surplus teams walk with the first, and store nothing
    const int64_t team = live ? mine : 0;
    const int lane = BLOCK ? threadIdx.x : threadIdx.x & (T - 1);
    const int c0 = (int)(team % a.groups) * width;
    const bool gated = a.gate != nullptr;
    const E *x = static_cast<const E *>(a.x) + c0 + lane * VEC, *gate = static_cast<const E *>(a.gate) + c0 + lane * VEC;
    E *y = static_cast<E *>(a.y) + c0 + lane * VEC;
    bool has[K];
    f32x2 w[K][P], b[K][P];
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int at = (lane + k * T) * VEC;
        float f[VEC], g[VEC];
        has[k] = at < width;
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            f[i] = 1.f;
            g[i] = 0.f;
        }
        if (a.weight && has[k]) ld_vec<float, VEC>(a.weight + c0 + at, f);
        if (a.bias && has[k]) ld_vec<float, VEC>(a.bias + c0 + at, g);
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const int lo = VEC > 1 ? 2 * i : 0, hi = VEC > 1 ? 2 * i + 1 : 0;
            w[k][i] = pack2(f[lo], f[hi]);
            b[k][i] = pack2(g[lo], g[hi]);
        }
    }
    auto pairs = [](const Vec &u, f32x2 (&v)[P]) {
        float f[VEC];
        widen(u, f);
#pragma unroll
        for (int i = 0; i < P; ++i) v[i] = pack2(f[VEC > 1 ? 2 * i : 0], VEC > 1 ? f[VEC > 1 ? 2 * i + 1 : 0] : 0.f);
    };
    auto both = [](f32x2 v) {
        float lo, hi;
        unpack2(v, lo, hi);
        return VEC > 1 ? lo + hi : lo;
    };
    Vec xv[kRows][K], gv[kRows][K];
#pragma unroll
    for (int r = 0; r < kRows; ++r)
#pragma unroll
        for (int k = 0; k < K; ++k) xv[r][k] = gv[r][k] = Vec();
    const float inv = 1.f / width;
    const int64_t first = team / a.groups * kRows, stride = (int64_t)walkers * kRows;
    x += first * a.ld_x;
    gate += first * a.ld_gate;
    y += first * a.ld_y;
    auto load = [&](int64_t left) {  // the next rows; past the last the values stay, and are not stored
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            if (r >= left) break;
#pragma unroll
            for (int k = 0; k < K; ++k) {
                if (!has[k]) continue;
                xv[r][k] = *reinterpret_cast<const Vec *>(x + r * a.ld_x + k * T * VEC);
                if (gated) gv[r][k] = *reinterpret_cast<const Vec *>(gate + r * a.ld_gate + k * T * VEC);
            }
        }
        x += stride * a.ld_x;
        gate += stride * a.ld_gate;
    };
    int64_t left = a.rows - first;
    load(left);
    // the same number of turns for every team: teams of a warp shuffle together
    for (int64_t ahead = a.rows; ahead > 0; ahead -= stride, left -= stride, y += stride * a.ld_y) {
        f32x2 c[kRows][K][P];  // about the mean
        Vec gn[kRows][K];
#pragma unroll
        for (int r = 0; r < kRows; ++r)
#pragma unroll
            for (int k = 0; k < K; ++k) {
                pairs(xv[r][k], c[r][k]);  // zeros past the width
                gn[r][k] = gv[r][k];
            }
        load(left - stride);
        float mean[kRows], rstd[kRows];
#pragma unroll
        for (int r = 0; r < kRows; ++r) mean[r] = 0.f;
        if (!a.rms) {
#pragma unroll
            for (int r = 0; r < kRows; ++r) {
                f32x2 sum = 0;
#pragma unroll
                for (int k = 0; k < K; ++k)
#pragma unroll
                    for (int i = 0; i < P; ++i) sum = add2(sum, c[r][k][i]);
                mean[r] = both(sum);
            }
            team_sum(mean, T);
        }
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            const f32x2 off = dup2(-mean[r] * inv);
            f32x2 sq = 0;
#pragma unroll
            for (int k = 0; k < K; ++k) {
                if (!has[k]) continue;
#pragma unroll
                for (int i = 0; i < P; ++i) {
                    c[r][k][i] = add2(c[r][k][i], off);
                    sq = fma2(c[r][k][i], c[r][k][i], sq);
                }
            }
            rstd[r] = both(sq);
        }
        team_sum(rstd, T);
#pragma unroll
        for (int r = 0; r < kRows; ++r) rstd[r] = rsqrtf(rstd[r] * inv + a.eps);
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            if (!live || r >= left) break;
#pragma unroll
            for (int k = 0; k < K; ++k) {
                if (!has[k]) continue;
                f32x2 u[P];
#pragma unroll
                for (int i = 0; i < P; ++i) u[i] = fma2(mul2(c[r][k][i], dup2(rstd[r])), w[k][i], b[k][i]);
                if (a.act == GDN_ACT_SILU)
#pragma unroll
                    for (int i = 0; i < P; ++i) u[i] = silu2(u[i]);
                if (gated) {
                    f32x2 g[P];
                    pairs(gn[r][k], g);
#pragma unroll
                    for (int i = 0; i < P; ++i) u[i] = mul2(u[i], silu2(g[i]));
                }
                float out[VEC];
#pragma unroll
                for (int i = 0; i < P; ++i) {
                    float lo, hi;
                    unpack2(u[i], lo, hi);
                    out[VEC > 1 ? 2 * i : 0] = lo;
                    if (VEC > 1) out[VEC > 1 ? 2 * i + 1 : 0] = hi;
                }
                st_vec<E, VEC>(y + r * a.ld_y + k * T * VEC, out);
            }
        }
    }
}

// Groups wider than a block's registers: a block per group, three passes over it,
// the later ones from L1 (single elements of 2051 channels: 94 us; held in
// registers by a block of 544 threads, 145).
template <typename E>
__global__ void __launch_bounds__(kThreads) gdn_group_norm_wide_kernel(const GdnNormArgs a)
{
    __shared__ __align__(16) float sh[2][1][kThreads / 32];
    TeamSum<kThreads, 1> team_sum = {sh, 0};
    const int width = a.channels / a.groups;
    const int64_t row = blockIdx.x / a.groups;
    const int c0 = (int)(blockIdx.x % a.groups) * width;
    const E *x = static_cast<const E *>(a.x) + row * a.ld_x + c0;
    const E *gate = a.gate ? static_cast<const E *>(a.gate) + row * a.ld_gate + c0 : nullptr;
    E *y = static_cast<E *>(a.y) + row * a.ld_y + c0;
    float sum[1] = {0.f}, q[1] = {0.f};
    if (!a.rms) {
        for (int i = threadIdx.x; i < width; i += kThreads) sum[0] += to_f(x[i]);
        team_sum(sum, kThreads);
    }
    const float mean = sum[0] / width;
    for (int i = threadIdx.x; i < width; i += kThreads) {
        const float v = to_f(x[i]) - mean;
        q[0] = fmaf(v, v, q[0]);
    }
    team_sum(q, kThreads);
    const float rstd = rsqrtf(q[0] / width + a.eps);
    for (int i = threadIdx.x; i < width; i += kThreads) {
        float u = fmaf((to_f(x[i]) - mean) * rstd, a.weight ? a.weight[c0 + i] : 1.f, a.bias ? a.bias[c0 + i] : 0.f);
        if (a.act == GDN_ACT_SILU) u = silu(u);
        y[i] = from_f<E>(gate ? u * silu(to_f(gate[i])) : u);
    }
}

template <typename E, int VEC, int K, int kRows, int BLOCK>
cudaError_t launch(const GdnNormArgs &a, int T, cudaStream_t s)
{
    // As many teams as are resident at once, or as there are rows for.
    static int fit = 0;  // blocks per device of this kind; the same for every caller
    constexpr int threads = BLOCK ? BLOCK : kThreads;
    const int per = threads / T;
    if (!fit) {
        int dev = 0, sms = 0, blocks = 0;
        cudaError_t e = cudaGetDevice(&dev);
        if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
        if (e == cudaSuccess)
            e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(
                &blocks, gdn_group_norm_kernel<E, VEC, K, kRows, BLOCK>, threads, 0);
        if (e != cudaSuccess) return e;
        fit = sms * (blocks > 0 ? blocks : 1);
    }
    const int64_t turns = (a.rows + kRows - 1) / kRows;
    int64_t walkers = ((int64_t)fit * per + a.groups - 1) / a.groups;
    if (walkers > turns) walkers = turns;
    // equal shares: the last turn is as full as the others
    const int64_t each = (turns + walkers - 1) / walkers;
    walkers = (turns + each - 1) / each;
    const int64_t blocks = (walkers * a.groups + per - 1) / per;
    if (blocks > 0x7fffffff) return cudaErrorInvalidConfiguration;
    gdn_group_norm_kernel<E, VEC, K, kRows, BLOCK><<<(unsigned)blocks, threads, 0, s>>>(a, T, (int)walkers);
    return cudaGetLastError();
}

// The team by the group's words: as many lanes of a warp as there are words, then
// what was fastest at each width.  us per 16 384 rows of about 2048 channels, bf16,
// gated (a team of T threads, K words each, R rows at a time as T x K x R).
// 16-byte words: heads of 128 16 x 1 x 2 34, x 3 34, x 1 36; of 512 64 x 1 x 2 33,
// 32 x 2 x 1 37, 32 x 2 x 2 48; of 1024 128 x 1 x 2 34, 32 x 4 x 1 43, 256 x 1 x 2
// 55; of 2048 256 x 1 x 2 35, 32 x 8 x 1 62.
// Single elements: heads of 129 32 x 5 x 2 81, 32 x 5 x 1 87, 64 x 3 x 2 100; of 189
// 32 x 6 x 1 74, 64 x 3 x 2 82, 32 x 6 x 2 109; of 255 64 x 4 x 2 66, 128 x 2 x 3 78,
// 128 x 2 x 2 83; of 293 128 x 3 x 2 87, 32 x 10 x 1 95, 128 x 4 x 2 140; of 405
// 64 x 8 x 1 85, 256 x 2 x 2 102, 128 x 4 x 2 110; of 679 256 x 4 x 2 95, x 1 135.
template <typename E, int VEC> cudaError_t by_width(const GdnNormArgs &a, cudaStream_t s)
{
    const int words = (a.channels / a.groups + VEC - 1) / VEC;
    if (words <= 32) {
        int T = 1;
        while (T < words) T *= 2;
        return launch<E, VEC, 1, 2, 0>(a, T, s);
    }
    if constexpr (VEC <= 2) {
        if (words <= 64) return launch<E, VEC, 2, 2, 0>(a, 32, s);
        if (words <= 96) return launch<E, VEC, 3, 2, 0>(a, 32, s);
        if (words <= 128) return launch<E, VEC, 4, 2, 0>(a, 32, s);
        if (words <= 160) return launch<E, VEC, 5, 2, 0>(a, 32, s);
        if (words <= 192) return launch<E, VEC, 6, 1, 0>(a, 32, s);
        if (words <= 256) return launch<E, VEC, 4, 2, 64>(a, 64, s);
        if (words <= 384) return launch<E, VEC, 3, 2, 128>(a, 128, s);
        if (words <= 512) return launch<E, VEC, 8, 1, 64>(a, 64, s);
        if (words <= 1024) return launch<E, VEC, 4, 2, 256>(a, 256, s);
    } else {
        if (words <= 64) return launch<E, VEC, 1, 2, 64>(a, 64, s);
        if (words <= 128) return launch<E, VEC, 1, 2, 128>(a, 128, s);
        if (words <= 256) return launch<E, VEC, 1, 2, 256>(a, 256, s);
        if (words <= 512) return launch<E, VEC, 2, 1, 256>(a, 256, s);
        if (words <= 1024) return launch<E, VEC, 4, 1, 256>(a, 256, s);
    }
    const int64_t blocks = a.rows * a.groups;
    if (blocks > 0x7fffffff) return cudaErrorInvalidConfiguration;
    gdn_group_norm_wide_kernel<E><<<(unsigned)blocks, kThreads, 0, s>>>(a);
    return cudaGetLastError();
}

// Whether all rows of all groups, and the weights, can be read in words of V elements.
template <typename E> bool words_of(const GdnNormArgs &a, int V)
{
    const size_t al = V * sizeof(E);
    return a.channels / a.groups % V == 0 && a.ld_x % V == 0 && a.ld_y % V == 0 && (!a.gate || a.ld_gate % V == 0) &&
           aligned_to(a.x, al) && aligned_to(a.y, al) && aligned_to(a.gate, al) &&
           aligned_to(a.weight, V == 2 ? 8 : 16) && aligned_to(a.bias, V == 2 ? 8 : 16);
}

template <typename E> cudaError_t by_rows(const GdnNormArgs &a, cudaStream_t s)
{
    constexpr int V = 16 / sizeof(E);
    return words_of<E>(a, V) ? by_width<E, V>(a, s) : words_of<E>(a, 2) ? by_width<E, 2>(a, s) : by_width<E, 1>(a, s);
}

}  // namespace

cudaError_t gdn_launch_group_norm(const GdnNormArgs &a, cudaStream_t s)
{
    return a.dtype == 1 ? by_rows<__nv_bfloat16>(a, s) : by_rows<float>(a, s);
}

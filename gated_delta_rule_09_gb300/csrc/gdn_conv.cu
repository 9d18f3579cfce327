// Short causal depthwise convolution, over prompts and for single tokens.
//
//     y[t, c] = act(bias[c] + sum_j weight[c, j] x[t - (width - 1) + j, c])
//
// 2 width operations per 4 bytes (bf16) moved: bound by HBM.  Channels are
// independent and neighbouring tokens share width - 1 inputs, so a thread owns
// 16 bytes of channels (one wide access per token, a block's threads side by
// side along the row) and walks a tile of tokens with the last width - 1 inputs
// in registers: every input is loaded once, plus the width - 1 rows ahead of
// each tile.  What keeps HBM busy is bytes on their way: a thread has 8 to 12
// tokens in flight through shared memory, whose columns no two threads share, so
// that no barrier is needed.  Rows that 16 bytes do not divide are read in words
// of two elements, and odd ones element by element.
//
// Measured, four taps, bf16: 4 x 4096 tokens x 6144 channels 68 us, 5.9 TB/s (a
// copy of the same tensors takes 64; the next four tokens held in registers
// instead of shared memory: 75); x 6142 channels, words of two, 85 us (159
// element by element with one channel per thread); x 6143 channels 99 us.  fp32,
// 6144 channels 130 us, 6.2 TB/s (a copy 122).
// 27 610 packed tokens x 1023 channels in fp32, three taps: 45 us, 5.0 TB/s.
// A token of 256 sequences x 6144 channels: 7.7 us.
#include <type_traits>

#include "gdn_layer.h"
#include "gdn_layer.cuh"

namespace {

using namespace gdn_layer;

constexpr int kThreads = 128;
constexpr int kGroup = 4;   // tokens loaded at a time
constexpr int kStages = 3;  // groups held or on their way

// Arithmetic on VEC channels, in pairs.
template <int VEC> struct Lanes {
    static constexpr int N = VEC / 2;
    f32x2 v[N];
};

// A thread's VEC channels are neighbours in one word, or, where rows are not
// aligned for that (SPLIT, VEC = 2), two single elements kThreads apart: both
// accesses of a warp are then contiguous, and arithmetic stays in pairs.  The two
// stay in registers of their own until they are used: packing them would wait
// for their loads.
template <typename E, int VEC, bool SPLIT> struct Access {
    typedef typename std::conditional<SPLIT, uint2, typename Word<VEC * sizeof(E)>::type>::type Vec;
    typedef typename Word<sizeof(E)>::type One;
    int c0;  // first channel
    int hi;  // where the second element is; 0 without one (the first is read again and not stored)

    __device__ __forceinline__ explicit Access(int channels)
    {
        c0 = block_of() * kThreads * VEC + threadIdx.x * (SPLIT ? 1 : VEC);
        hi = c0 + kThreads < channels ? kThreads : 0;
    }
    __device__ __forceinline__ Vec load(const E *p) const
    {
        if constexpr (SPLIT) {
            const One *u = reinterpret_cast<const One *>(p);
            return make_uint2(u[0], u[hi]);
        } else {
            return *reinterpret_cast<const Vec *>(p);
        }
    }
    __device__ __forceinline__ void store(E *p, const Vec &v) const
    {
        if constexpr (SPLIT) {
            One *u = reinterpret_cast<One *>(p);
            u[0] = (One)v.x;
            if (hi) u[hi] = (One)v.y;
        } else {
            *reinterpret_cast<Vec *>(p) = v;
        }
    }
    __device__ __forceinline__ static Lanes<VEC> get(const Vec &v)
    {
        float x[VEC];
        if constexpr (SPLIT) {
            const int up = sizeof(E) == 2 ? 16 : 0;
            x[0] = __uint_as_float(v.x << up);
            x[1] = __uint_as_float(v.y << up);
        } else {
            widen(v, x);
        }
        Lanes<VEC> l;
#pragma unroll
        for (int i = 0; i < VEC; i += 2) l.v[i / 2] = pack2(x[i], x[i + 1]);
        return l;
    }
    __device__ __forceinline__ static Vec put(const Lanes<VEC> &l)
    {
        float x[VEC];
#pragma unroll
        for (int i = 0; i < VEC; i += 2) unpack2(l.v[i / 2], x[i], x[i + 1]);
        typename Word<VEC * sizeof(E)>::type u;
        narrow(u, x);
        if constexpr (SPLIT && sizeof(E) == 2)
            return make_uint2(u & 0xffff, u >> 16);
        else
            return u;
    }
};

// Taps and bias of the thread's channels.
template <typename E, int VEC, bool SPLIT, int W> struct Taps {
    Lanes<VEC> w[W], b;

    __device__ __forceinline__ Taps(const GdnConvArgs &a, const Access<E, VEC, SPLIT> &at)
    {
        float f[VEC * W], bias[VEC];
        const float *weight = a.weight + (size_t)at.c0 * W;
        if constexpr (SPLIT) {
#pragma unroll
            for (int j = 0; j < W; ++j) {
                f[j] = weight[j];
                f[W + j] = weight[at.hi * W + j];
            }
        } else {  // VEC W and c0 W are multiples of the words' elements
            constexpr int V = VEC > 2 ? 4 : 2;
#pragma unroll
            for (int i = 0; i < VEC * W; i += V) {
                float t[V];
                ld_vec<float, V>(weight + i, t);
#pragma unroll
                for (int j = 0; j < V; ++j) f[i + j] = t[j];
            }
        }
#pragma unroll
        for (int i = 0; i < VEC; ++i) bias[i] = a.bias ? a.bias[at.c0 + (SPLIT ? i * at.hi : i)] : 0.f;
#pragma unroll
        for (int i = 0; i < VEC; i += 2) {
#pragma unroll
            for (int j = 0; j < W; ++j) w[j].v[i / 2] = pack2(f[i * W + j], f[(i + 1) * W + j]);
            b.v[i / 2] = pack2(bias[i], bias[i + 1]);
        }
    }

    // y of the token whose input is win[W - 1]
    __device__ __forceinline__ typename Access<E, VEC, SPLIT>::Vec apply(const Lanes<VEC> (&win)[W], int act) const
    {
        Lanes<VEC> r = b;
#pragma unroll
        for (int i = 0; i < Lanes<VEC>::N; ++i) {
#pragma unroll
            for (int j = 0; j < W; ++j) r.v[i] = fma2(w[j].v[i], win[j].v[i], r.v[i]);
            if (act == GDN_ACT_SILU) r.v[i] = silu2(r.v[i]);
        }
        return Access<E, VEC, SPLIT>::put(r);
    }
};

template <typename E, int VEC, bool SPLIT, int W>
__global__ void __launch_bounds__(kThreads)
    gdn_conv_fwd_kernel(const GdnConvArgs a, int tl, int tiles)
{
    typedef typename Access<E, VEC, SPLIT>::Vec Vec;
    extern __shared__ __align__(16) unsigned char smem[];
    Span s;
    if (!find_span(a.cu_seqlens, a.N, a.T, tl, blockIdx.x, tiles, a.status, s)) return;
    const Access<E, VEC, SPLIT> mine(a.channels);
    const int c0 = mine.c0;
    if (c0 >= a.channels) return;
    const E *x = static_cast<const E *>(a.x) + s.row * a.ld_x + c0;
    E *y = static_cast<E *>(a.y) + s.row * a.ld_y + c0;
    const int t0 = s.tile * tl, t1 = min(s.len, t0 + tl);
    auto input = [&](int64_t t) { return mine.load(x + t * a.ld_x); };

    Lanes<VEC> win[W];  // win[j]: the input j - (W - 1) tokens from the current one
    if (s.tile == 0) {
        // The state is read and written by this thread alone (whichever tile
        // the sequence ends in), so it may be updated in place.
        const int entry = state_entry(a.slots, s.n, a.pool, a.status);
        const E *in = static_cast<const E *>(a.state_in);
        const size_t at = entry < 0 ? 0 : (size_t)entry * (W - 1) * a.channels + c0;
        Vec kept[W];
#pragma unroll
        for (int j = 0; j < W - 1; ++j) {
            kept[j] = Vec();
            if (in && entry >= 0) kept[j] = mine.load(in + at + (size_t)j * a.channels);
            win[j] = mine.get(kept[j]);
        }
        if (a.state_out && entry >= 0) {
            E *out = static_cast<E *>(a.state_out);
#pragma unroll
            for (int j = 0; j < W - 1; ++j) {
                const int p = s.len - (W - 1) + j;
                Vec v = Vec();
                if (p >= 0) {
                    v = input(p);
                } else {  // fewer tokens than taps: the older state moves up
#pragma unroll
                    for (int k = 0; k < W - 1; ++k)
                        if (k == p + W - 1) v = kept[k];
                }
                mine.store(out + at + (size_t)j * a.channels, v);
            }
        }
    } else {  // a tile is longer than the taps, so these lie in the same sequence
#pragma unroll
        for (int j = 0; j < W - 1; ++j) win[j] = mine.get(input(t0 - (W - 1) + j));
    }
    if (t0 >= t1) return;

    const Taps<E, VEC, SPLIT, W> taps(a, mine);
    auto token = [&](int t, const Vec &u) {
        win[W - 1] = mine.get(u);
        mine.store(y + (int64_t)t * a.ld_y, taps.apply(win, a.act));
#pragma unroll
        for (int j = 0; j < W - 1; ++j) win[j] = win[j + 1];
    };
    auto use = [&](const Vec (&u)[kGroup], int t) {
        if (t + kGroup <= t1) {
#pragma unroll
            for (int k = 0; k < kGroup; ++k) token(t + k, u[k]);
        } else {
#pragma unroll
            for (int k = 0; k < kGroup; ++k)
                if (t + k < t1) token(t + k, u[k]);
        }
    };
    if constexpr (sizeof(Vec) == 16) {
        // A column of shared memory per thread, filled and read by it alone.
        Vec *ring = reinterpret_cast<Vec *>(smem) + threadIdx.x;
        auto fetch = [&](int t, int stage) {
#pragma unroll
            for (int k = 0; k < kGroup; ++k)
                if (t + k < t1)
                    copy_async<sizeof(Vec)>(ring + (stage * kGroup + k) * kThreads, x + (int64_t)(t + k) * a.ld_x);
            copy_commit();
        };
#pragma unroll
        for (int i = 0; i < kStages - 1; ++i) fetch(t0 + i * kGroup, i);
        int at = 0, to = kStages - 1;
#pragma unroll 1
        for (int t = t0; t < t1; t += kGroup) {
            fetch(t + (kStages - 1) * kGroup, to);
            copy_wait<kStages - 1>();
            Vec u[kGroup];
#pragma unroll
            for (int k = 0; k < kGroup; ++k) u[k] = ring[(at * kGroup + k) * kThreads];
            use(u, t);
            to = at;  // what was read is filled next
            at = at + 1 == kStages ? 0 : at + 1;
        }
    } else {  // small words, and so few registers: more threads fit, and the next tokens stay in registers
        Vec u[2][kGroup];
        auto load = [&](Vec (&v)[kGroup], int t) {  // past the end: the last token again, not used
#pragma unroll
            for (int k = 0; k < kGroup; ++k) v[k] = input(min(t + k, t1 - 1));
        };
        load(u[0], t0);
        for (int t = t0; t < t1; t += 2 * kGroup) {
            load(u[1], t + kGroup);
            use(u[0], t);
            if (t + 2 * kGroup < t1) load(u[0], t + 2 * kGroup);
            use(u[1], t + kGroup);
        }
    }
}

// One token per sequence: the state moves on by one input.  A thread takes its
// channels of kRows sequences, whose loads are in flight together and share the
// taps (64 bytes per tap and thread, more than a sequence's own).
template <typename E, int VEC, bool SPLIT, int W, int kRows>
__global__ void __launch_bounds__(kThreads) gdn_conv_step_kernel(const GdnConvArgs a)
{
    typedef typename Access<E, VEC, SPLIT>::Vec Vec;
    const Access<E, VEC, SPLIT> mine(a.channels);
    const int c0 = mine.c0;
    if (c0 >= a.channels) return;
    const int n0 = blockIdx.x * kRows;
    const E *in = static_cast<const E *>(a.state_in), *x = static_cast<const E *>(a.x) + n0 * a.ld_x + c0;
    int entry[kRows];
    Vec u[kRows][W];
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
        const int n = n0 + r;
        entry[r] = n < a.N ? state_entry(a.slots, n, a.pool, a.status) : -1;
        u[r][W - 1] = Vec();
        if (n < a.N) u[r][W - 1] = mine.load(x + r * a.ld_x);
    }
#pragma unroll
    for (int r = 0; r < kRows; ++r)
#pragma unroll
        for (int j = 0; j < W - 1; ++j) {
            u[r][j] = Vec();
            if (in && entry[r] >= 0)
                u[r][j] = mine.load(in + ((size_t)entry[r] * (W - 1) + j) * a.channels + c0);
        }
    const Taps<E, VEC, SPLIT, W> taps(a, mine);
    E *y = static_cast<E *>(a.y) + n0 * a.ld_y + c0;
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
        if (n0 + r >= a.N) break;
        Lanes<VEC> win[W];
#pragma unroll
        for (int j = 0; j < W; ++j) win[j] = mine.get(u[r][j]);
        mine.store(y + r * a.ld_y, taps.apply(win, a.act));
        if (entry[r] < 0) continue;
        E *out = static_cast<E *>(a.state_out) + (size_t)entry[r] * (W - 1) * a.channels + c0;
#pragma unroll
        for (int j = 0; j < W - 1; ++j) mine.store(out + (size_t)j * a.channels, u[r][j + 1]);
    }
}

// Whether rows, states and taps can be read in words of V elements.
template <typename E> bool words_of(const GdnConvArgs &a, int V)
{
    const size_t al = V * sizeof(E);
    return a.channels % V == 0 && a.ld_x % V == 0 && a.ld_y % V == 0 && aligned_to(a.x, al) && aligned_to(a.y, al) &&
           aligned_to(a.state_in, al) && aligned_to(a.state_out, al) && aligned_to(a.weight, V == 2 ? 8 : 16);
}

template <typename E, int VEC, bool SPLIT, int W>
cudaError_t fwd(const GdnConvArgs &a, cudaStream_t s)
{
    const int blocks = (a.channels + kThreads * VEC - 1) / (kThreads * VEC);
    // The tile length of at least 16 tokens that takes the fewest token times: blocks run in
    // waves of what is resident at once, and a tile reads width - 1 rows ahead of its own.
    constexpr size_t smem = VEC <= 2 ? 0 : kStages * kGroup * kThreads * VEC * sizeof(E);
    static int resident = 0;  // blocks per device of this kind; the same for every caller
    if (!resident) {
        int dev = 0, sms = 0, n = 0;
        cudaError_t e = cudaGetDevice(&dev);
        if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(gdn_conv_fwd_kernel<E, VEC, SPLIT, W>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e == cudaSuccess)
            e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, gdn_conv_fwd_kernel<E, VEC, SPLIT, W>, kThreads, smem);
        if (e != cudaSuccess) return e;
        resident = sms * (n > 0 ? n : 1);
    }
    int tl = 16;
    int64_t best = INT64_MAX;
    for (int t = 16; t <= 128; t += 8) {
        const int64_t n = (a.cu_seqlens ? (int64_t)a.T / t + a.N : (int64_t)a.N * ((a.T + t - 1) / t)) * blocks;
        const int64_t cost = (n + resident - 1) / resident * (t + W - 1);
        if (cost <= best) {
            best = cost;
            tl = t;
        }
    }
    const int tiles = a.T > tl ? (a.T + tl - 1) / tl : 1;
    const int64_t slots = a.cu_seqlens ? (int64_t)a.T / tl + a.N : (int64_t)a.N * tiles;
    if (slots > 0x7fffffff) return cudaErrorInvalidConfiguration;
    gdn_conv_fwd_kernel<E, VEC, SPLIT, W><<<grid_of((unsigned)slots, blocks), kThreads, smem, s>>>(a, tl, tiles);
    return cudaGetLastError();
}

template <typename E, int VEC, bool SPLIT, int W>
cudaError_t step(const GdnConvArgs &a, cudaStream_t s)
{
    const int blocks = (a.channels + kThreads * VEC - 1) / (kThreads * VEC);
    // Four sequences per thread once enough blocks are left for the SMs.  bf16, four taps, us with
    // one against four, 6 blocks per sequence (16-byte words): 32 sequences 3.3 : 3.6, 64 4.9 : 4.3,
    // 256 11.4 : 7.7.  24 blocks (single elements): 16 sequences 2.1 : 2.6, 256 9.1 : 8.3.
    if ((int64_t)a.N * blocks >= (SPLIT ? 1024 : 384))
        gdn_conv_step_kernel<E, VEC, SPLIT, W, 4><<<grid_of((a.N + 3) / 4, blocks), kThreads, 0, s>>>(a);
    else
        gdn_conv_step_kernel<E, VEC, SPLIT, W, 1><<<grid_of(a.N, blocks), kThreads, 0, s>>>(a);
    return cudaGetLastError();
}

template <bool STEP, typename E, int W>
cudaError_t by_vector(const GdnConvArgs &a, cudaStream_t s)
{
    constexpr int V = 16 / sizeof(E);
    if (words_of<E>(a, V)) return STEP ? step<E, V, false, W>(a, s) : fwd<E, V, false, W>(a, s);
    if (words_of<E>(a, 2)) return STEP ? step<E, 2, false, W>(a, s) : fwd<E, 2, false, W>(a, s);
    return STEP ? step<E, 2, true, W>(a, s) : fwd<E, 2, true, W>(a, s);
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

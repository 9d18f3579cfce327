// Linear attention with a decay for each head on the tensor cores: bf16 in and
// out, fp32 sums and states.
//
// A block takes one (sequence or piece, head, 64 columns of v) and walks it in
// chunks of 128 tokens.  With b the sum of log decays up to and with a token of
// the chunk, and S^T (d_k x 64) the state before it:
//
//   P   = Lower(Q K^T e^{b_i - b_j})                  [128 x 128]
//   O   = scale (e^{b_i} Q S^T + P V)                 [128 x 64]
//   U   = K^T (V e^{b_n - b_j})                       [d_k x 64]
//   S^T <- e^{b_n} S^T + U
//
// Only the last line is serial, and it is 64 fused multiply-adds a thread: the
// state stays in the registers of four warps, fp32, for the whole walk, and none
// of the products waits for more than the one before it.  Q, K and V enter as they
// are (products of bf16 are exact in fp32); what is formed on the way, P, S and
// the decayed V, enters as two bf16 parts whose sum keeps 16 bits and more, so that
// the final states are right to 2e-6 and the outputs but for their own rounding.
//
// Roles: warps 0-3 form P (tensor memory to tensor memory, a row per thread),
// warps 4-7 keep the state and write its parts for the next chunk, warps 8-11 sum
// the decays and form the decayed V, warps 12-15 write the outputs, warp 16 issues
// the products, warp 17 the tensor copies into a ring of two stages.
//
// Every wait is bounded: on timeout the block raises GDN_DEV_WAIT_TIMEOUT, issues
// no more copies and winds down with waits of 50 us, enough for what is in flight.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <mutex>

#include "gdn_linattn.cuh"
#include "sm100_ptx.cuh"

namespace {

using namespace gdn_linattn;
using namespace sm100;

constexpr int kC = 128;     // tokens per chunk
constexpr int kDVT = 64;    // columns of v per block
constexpr int kThreads = 18 * 32;
constexpr float kPlain = 120.f;  // decays of a block of 32, log 2, that go as products of two factors
constexpr uint64_t kWaitLimitNs = 2000000000ull;
constexpr uint64_t kDrainNs = 50000;  // a wait's bound once the block has given up on one

// Shared memory: tiles of 128-byte rows, 128-byte swizzle.
constexpr int kTile = kC * 128;           // 128 rows
constexpr int kOffQ = 0;                  // 2 stages x 2 halves of d_k
constexpr int kOffK = kOffQ + 4 * kTile;
constexpr int kOffV = kOffK + 4 * kTile;  // 2 stages
constexpr int kOffW = kOffV + 2 * kTile;  // decayed V: high and low parts
constexpr int kOffS = kOffW + 2 * kTile;  // S^T: high and low parts
constexpr int kOffSmall = kOffS + 2 * kTile;

struct Small {
    // decays of two chunks: sums up to and with a token within its block of 32, their
    // inverse factors 2^-in, and the blocks' sums
    float in[2][kC], inverse[2][kC], total[2][4];
    unsigned mask[2][4];
    int odd[2];             // V has infinities or NaN
    uint64_t full[2], kq_free[2], v_free[2], dec_ready[2], dec_free[2], w_ready[2];
    uint64_t qk_full, p_ready, p_free, u_full, u_free, s_ready, o_full, o_free;
    uint32_t tmem;
    int abort_flag;
};
constexpr int kSmemBytes = kOffSmall + (int)sizeof(Small);
static_assert(kSmemBytes <= 232448, "shared memory per block");

// Tensor memory, 512 columns: Q K^T | parts of P | Q S^T x 2 | P V | U.
constexpr uint32_t kColQK = 0, kColP = 128, kColI = 256, kColO = 384, kColU = 448;

__device__ __noinline__ bool wait_long(uint64_t *bar, uint32_t parity, volatile int *abort_flag, unsigned int *status)
{
    if (mbar_wait(bar, parity, *abort_flag ? kDrainNs : kWaitLimitNs)) return true;
    *abort_flag = 1;
    atomicOr(status, GDN_DEV_WAIT_TIMEOUT);
    return false;
}

struct Waiter {
    volatile int *abort_flag;
    unsigned int *status;
    __device__ __forceinline__ void operator()(uint64_t *bar, int phase) const
    {
        if (!mbar_test_wait(bar, phase & 1)) wait_long(bar, phase & 1, abort_flag, status);
    }
};

__device__ __forceinline__ uint32_t lane_addr(uint32_t tbase, int quad, uint32_t col)
{
    return tbase + (static_cast<uint32_t>(quad * 32) << 16) + col;
}

// Waits for this thread's loads from tensor memory; v is not looked at before.
template <int N> __device__ __forceinline__ void landed(float (&v)[N])
{
    tmem_ld_wait();
#pragma unroll
    for (int i = 0; i < N; ++i) asm volatile("" : "+f"(v[i]));
}

__device__ __forceinline__ uint32_t tmem_ld1(uint32_t taddr)
{
    uint32_t v;
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];" : "=r"(v) : "r"(taddr));
    return v;
}

// Two values as two bf16 pairs, the first rounded, the second what that leaves.
// `sign` becomes NaN where a value is infinite or NaN, whose second part then is NaN.
__device__ __forceinline__ void split(f32x2 v, uint32_t &hi, uint32_t &lo, f32x2 &sign)
{
    float x, y;
    unpack2(v, x, y);
    hi = narrow_pair(x, y);
    const f32x2 d = fma2(pack2(__uint_as_float(hi << 16), __uint_as_float(hi & 0xffff0000u)), dup2(-1.f), v);
    sign = fma2(d, dup2(0.f), sign);
    unpack2(d, x, y);
    lo = narrow_pair(x, y);
}

__device__ __forceinline__ bool is_odd(f32x2 sign)
{
    float x, y;
    unpack2(sign, x, y);
    return x + y != 0.f;
}

// Second parts where the first is infinite or NaN: zero.
template <int N> __device__ __forceinline__ void mend(const uint32_t (&hi)[N], uint32_t (&lo)[N])
{
#pragma unroll
    for (int i = 0; i < N; ++i) {
        if ((hi[i] & 0x7f80u) == 0x7f80u) lo[i] &= 0xffff0000u;
        if ((hi[i] & 0x7f800000u) == 0x7f800000u) lo[i] &= 0xffffu;
    }
}

// 8 values into 16-byte column c of row r of two tiles.
__device__ __forceinline__ void st_parts(uint8_t *tiles, int r, int c, const f32x2 (&x)[4])
{
    uint32_t hi[4], lo[4];
    f32x2 sign = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) split(x[i], hi[i], lo[i], sign);
    if (is_odd(sign)) mend(hi, lo);
    const uint32_t at = sw128(r, c);
    *reinterpret_cast<uint4 *>(tiles + at) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
    *reinterpret_cast<uint4 *>(tiles + kTile + at) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
}

// P of one row in the cases that the plain path leaves: tokens that forget, blocks
// that decay by more than 2^120, and products that are infinite or NaN.
__device__ __noinline__ void odd_decays(uint32_t tbase, int quad, int lane, const float *in, const float *total,
                                        const unsigned *mask)
{
    const float mine = in[32 * quad + lane];
    float sum = mine;
    bool cut = mask[quad] & (0xffffffffu >> (31 - lane));
    const int first = first_seen(mask[quad], lane);
#pragma unroll 1
    for (int J = quad; J >= 0; --J) {
        float x[32];
        tmem_ld32(lane_addr(tbase, quad, kColQK + 32 * J), x);
        landed(x);
        uint32_t hi[16], lo[16];
        f32x2 sign = 0;
#pragma unroll
        for (int j = 0; j < 32; ++j) {
            const float w = in[32 * J + j];
            const bool seen = J == quad ? j <= lane && j >= first : !cut && !(mask[J] & (0xfffffffeu << j));
            const float f = decay_of(J == quad ? mine - w : sum + (total[J] - w));
            x[j] = seen && f != 0.f ? x[j] * f : 0.f;
        }
#pragma unroll
        for (int j = 0; j < 16; ++j) split(pack2(x[2 * j], x[2 * j + 1]), hi[j], lo[j], sign);
        mend(hi, lo);
        __syncwarp();
        tmem_st16(lane_addr(tbase, quad, kColP + 16 * J), hi);
        tmem_st16(lane_addr(tbase, quad, kColP + 64 + 16 * J), lo);
        if (J < quad) {
            sum += total[J];
            cut = cut || mask[J];
        }
    }
}

// P V of one row and 32 columns for a chunk whose V is infinite or NaN somewhere: a
// token must see nothing of those behind it, and zero times infinity is NaN.
__device__ __noinline__ void odd_row(uint32_t tbase, int quad, int i, int first, const uint8_t *V, int half, float (&acc)[32])
{
#pragma unroll
    for (int d = 0; d < 32; ++d) acc[d] = 0.f;
#pragma unroll 1
    for (int w = 0; w < 16 * (quad + 1); ++w) {
        __syncwarp();
        uint32_t hi = tmem_ld1(lane_addr(tbase, quad, kColP + w)), lo = tmem_ld1(lane_addr(tbase, quad, kColP + 64 + w));
        tmem_ld_wait();
        asm volatile("" : "+r"(hi), "+r"(lo));
#pragma unroll 1
        for (int e = 0; e < 2; ++e) {
            const int j = 2 * w + e;
            const float p = e ? __uint_as_float(hi & 0xffff0000u) + __uint_as_float(lo & 0xffff0000u)
                              : __uint_as_float(hi << 16) + __uint_as_float(lo << 16);
            if (j > i || j < first) continue;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                float v[8];
                widen(*reinterpret_cast<const uint4 *>(V + sw128(j, half * 4 + q)), v);
#pragma unroll
                for (int d = 0; d < 8; ++d) acc[q * 8 + d] = fmaf(p, v[d], acc[q * 8 + d]);
            }
        }
    }
}

__global__ void __launch_bounds__(kThreads, 1)
gdn_linattn_tc_kernel(const GdnLinattnArgs a, int tiles, int states_only, const __grid_constant__ CUtensorMap tm_q,
                      const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v)
{
    extern __shared__ __align__(1024) uint8_t sm[];
    Small &s = *reinterpret_cast<Small *>(sm + kOffSmall);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, quad = warp & 3, t = tid & 127;
    const int64_t unit = blockIdx.x;
    const int v0 = (int)(unit % tiles) * kDVT, h = (int)(unit / tiles % a.heads);
    Unit u;
    if (!find_unit(a, unit / tiles / a.heads, h, states_only, u)) return;
    const int chunks = (int)(((int64_t)u.len + kC - 1) / kC), dk = a.dk;

    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s.full[i], 1);
            mbar_init(&s.kq_free[i], 1);
            mbar_init(&s.v_free[i], 1);
            mbar_init(&s.dec_ready[i], 128);
            mbar_init(&s.dec_free[i], states_only ? 128 : 384);
            mbar_init(&s.w_ready[i], 128);
        }
        mbar_init(&s.qk_full, 1);
        mbar_init(&s.p_ready, 128);
        mbar_init(&s.p_free, 1);
        mbar_init(&s.u_full, 1);
        mbar_init(&s.u_free, 128);
        mbar_init(&s.s_ready, 128);
        mbar_init(&s.o_full, 1);
        mbar_init(&s.o_free, 128);
        s.abort_flag = 0;
        fence_mbar_init();
        prefetch_tensormap(&tm_q);
        prefetch_tensormap(&tm_k);
        prefetch_tensormap(&tm_v);
    }
    if (warp == 0) {
        tmem_alloc(&s.tmem, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tbase = s.tmem;
    volatile int *abort_flag = &s.abort_flag;
    const Waiter wait = {abort_flag, a.status};

    if (warp < 4) {
        // ---- P
        if (!states_only && chunks > 0) {
            const uint32_t zero[16] = {};
            for (int J = quad + 1; J < 4; ++J) {  // blocks above the diagonal stay zero
                tmem_st16(lane_addr(tbase, quad, kColP + 16 * J), zero);
                tmem_st16(lane_addr(tbase, quad, kColP + 64 + 16 * J), zero);
            }
            tmem_st_wait();
        }
        for (int c = 0; c < chunks && !states_only; ++c) {
            const int st = c & 1;
            wait(&s.dec_ready[st], c >> 1);
            // The factor of tokens i and j is 2^(in_i + the blocks between) 2^(total_J) 2^-in_j, where J, the block
            // of j, decays by less than 2^120; within a block without the middle factor.
            const float in = s.in[st][t];
            bool plain = true;
            for (int J = 0; J <= quad; ++J) plain = plain && s.mask[st][J] == 0 && fabsf(s.total[st][J]) < kPlain;
            wait(&s.qk_full, c);
            if (c > 0) wait(&s.p_free, c - 1);
            __syncwarp();
            tc_fence_after();
            float sum = in;
            bool odd = false;
#pragma unroll 1
            for (int J = quad; J >= 0 && plain; --J) {
                float x[32];
                tmem_ld32(lane_addr(tbase, quad, kColQK + 32 * J), x);
                if (J < quad) sum += s.total[st][J];
                const f32x2 f = dup2(decay_of(sum));
                const float4 *inverse = reinterpret_cast<const float4 *>(&s.inverse[st][32 * J]);
                landed(x);
                if (J == quad) {
#pragma unroll
                    for (int j = 0; j < 32; ++j) x[j] = j <= lane ? x[j] : 0.f;
                }
                uint32_t hi[16], lo[16];
                f32x2 sign = 0;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float4 w = inverse[j];
                    split(mul2(pack2(x[4 * j], x[4 * j + 1]), mul2(f, pack2(w.x, w.y))), hi[2 * j], lo[2 * j], sign);
                    split(mul2(pack2(x[4 * j + 2], x[4 * j + 3]), mul2(f, pack2(w.z, w.w))), hi[2 * j + 1],
                          lo[2 * j + 1], sign);
                }
                odd |= is_odd(sign);
                tmem_st16(lane_addr(tbase, quad, kColP + 16 * J), hi);
                tmem_st16(lane_addr(tbase, quad, kColP + 64 + 16 * J), lo);
            }
            if (__any_sync(0xffffffffu, odd || !plain)) odd_decays(tbase, quad, lane, s.in[st], s.total[st], s.mask[st]);
            mbar_arrive(&s.dec_free[st]);
            tmem_st_wait();
            tc_fence_before();
            mbar_arrive(&s.p_ready);
        }
    } else if (warp < 8) {
        // ---- the state: row t of S^T
        f32x2 S[kDVT / 2];
        const int64_t at = (int64_t)v0 * dk + t;
        const int nv = min(kDVT, a.dv - v0);
#pragma unroll
        for (int d = 0; d < kDVT; d += 2) {
            const bool is = u.in && t < dk;
            S[d / 2] = pack2(is && d < nv ? u.in[at + (int64_t)d * dk] : 0.f,
                             is && d + 1 < nv ? u.in[at + (int64_t)(d + 1) * dk] : 0.f);
        }
        auto hand_over = [&] {
#pragma unroll
            for (int q = 0; q < 8; ++q) {
                const f32x2 x[4] = {S[4 * q], S[4 * q + 1], S[4 * q + 2], S[4 * q + 3]};
                st_parts(sm + kOffS, t, q, x);
            }
            fence_async_smem();
            mbar_arrive(&s.s_ready);
        };
        if (chunks > 0 && !states_only) hand_over();
        for (int c = 0; c < chunks; ++c) {
            const int st = c & 1;
            wait(&s.dec_ready[st], c >> 1);
            const float4 total = *reinterpret_cast<const float4 *>(s.total[st]);
            const uint4 mask = *reinterpret_cast<const uint4 *>(s.mask[st]);
            const float all = mask.x | mask.y | mask.z | mask.w ? 0.f : decay_of(total.x + total.y + total.z + total.w);
            mbar_arrive(&s.dec_free[st]);
            if (all == 0.f)
#pragma unroll
                for (int d = 0; d < kDVT / 2; ++d) S[d] = 0;  // forgotten, infinite or not
            wait(&s.u_full, c);
            __syncwarp();
            tc_fence_after();
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                float x[32];
                tmem_ld32(lane_addr(tbase, quad, kColU + 32 * half), x);
                landed(x);
#pragma unroll
                for (int d = 0; d < 16; ++d) S[16 * half + d] = fma2(dup2(all), S[16 * half + d], pack2(x[2 * d], x[2 * d + 1]));
            }
            tc_fence_before();
            mbar_arrive(&s.u_free);
            if (c + 1 < chunks && !states_only) {
                wait(&s.kq_free[st], c >> 1);  // Q S^T of this chunk has read the parts
                hand_over();
            }
        }
        if (u.out && !*abort_flag)
#pragma unroll
            for (int d = 0; d < kDVT; d += 2) {
                float x, y;
                unpack2(S[d / 2], x, y);
                if (t < dk && d < nv) u.out[at + (int64_t)d * dk] = x;
                if (t < dk && d + 1 < nv) u.out[at + (int64_t)(d + 1) * dk] = y;
            }
    } else if (warp < 12) {
        // ---- decays, and V times the decay to the chunk's end
        const float *decay = a.log_decay + (u.row + t) * a.ld_decay + h;
        float next = t < u.len ? *decay : 0.f;
        for (int c = 0; c < chunks; ++c) {
            const int st = c & 1, n = min(kC, u.len - c * kC);
            Decays d;
            d.scan(next);
            next = t + (int64_t)(c + 1) * kC < u.len ? decay[(int64_t)(c + 1) * kC * a.ld_decay] : 0.f;
            if (c > 1) wait(&s.dec_free[st], (c - 2) >> 1);
            s.in[st][t] = d.in;
            s.inverse[st][t] = ex2(-d.in);
            if (lane == 0) {
                s.total[st][quad] = d.total;
                s.mask[st][quad] = d.mask;
            }
            if (t == 0) s.odd[st] = 0;
            mbar_arrive(&s.dec_ready[st]);
            named_sync(1, 128);
            bool cut = d.cut_behind(lane);
            float sum = d.after;
#pragma unroll
            for (int J = 1; J < 4; ++J)
                if (J > quad) {
                    cut = cut || s.mask[st][J];
                    sum += s.total[st][J];
                }
            const float w = cut ? 0.f : decay_of(sum);
            wait(&s.full[st], c >> 1);
            if (c > 0) wait(&s.u_full, c - 1);  // the product has read the last chunk's
            uint8_t *V = sm + kOffV + st * kTile, *W = sm + kOffW;
            if (t < n) {
                f32x2 sign = 0;
#pragma unroll 2
                for (int q = 0; q < 8; ++q) {
                    float f[8];
                    widen(*reinterpret_cast<const uint4 *>(V + sw128(t, q)), f);
                    f32x2 x[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        x[e] = pack2(f[2 * e], f[2 * e + 1]);
                        sign = fma2(x[e], dup2(0.f), sign);
                        x[e] = w == 0.f ? 0 : mul2(x[e], dup2(w));
                    }
                    st_parts(W, t, q, x);
                }
                if (is_odd(sign)) s.odd[st] = 1;
            } else {  // rows past the end may be another sequence's
                const uint4 zero = make_uint4(0, 0, 0, 0);
                uint8_t *K = sm + kOffK + st * 2 * kTile;
                for (int q = 0; q < 8; ++q) {
                    const uint32_t off = sw128(t, q);
                    *reinterpret_cast<uint4 *>(V + off) = zero;
                    *reinterpret_cast<uint4 *>(W + off) = zero;
                    *reinterpret_cast<uint4 *>(W + kTile + off) = zero;
                    *reinterpret_cast<uint4 *>(K + off) = zero;
                    if (dk > 64) *reinterpret_cast<uint4 *>(K + kTile + off) = zero;
                }
            }
            fence_async_smem();
            mbar_arrive(&s.w_ready[st]);
        }
    } else if (warp < 16) {
        // ---- outputs: row t
        __nv_bfloat16 *o = static_cast<__nv_bfloat16 *>(a.o) + (u.row + t) * a.ld_o + (int64_t)h * a.dv + v0;
        const int nv = min(kDVT, a.dv - v0);
        for (int c = 0; c < chunks && !states_only; ++c, o += kC * a.ld_o) {
            const int st = c & 1, n = min(kC, u.len - c * kC);
            wait(&s.dec_ready[st], c >> 1);
            const unsigned mask = s.mask[st][quad];
            float sum = s.in[st][t];
            bool cut = mask & (0xffffffffu >> (31 - lane));
            int first = 32 * quad + first_seen(mask, lane);
#pragma unroll
            for (int J = 2; J >= 0; --J)
                if (J < quad) {
                    if (!cut) first = 32 * J + (s.mask[st][J] ? 31 - __clz(s.mask[st][J]) : 0);
                    cut = cut || s.mask[st][J];
                    sum += s.total[st][J];
                }
            const float start = cut ? 0.f : a.scale * decay_of(sum);
            wait(&s.w_ready[st], c >> 1);
            const bool odd = s.odd[st];
            mbar_arrive(&s.dec_free[st]);
            wait(&s.o_full, c);
            tc_fence_after();
            if (!odd && t == 0) {
                mbar_arrive(&s.v_free[st]);
                mbar_arrive(&s.p_free);
            }
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                float x[32], y[32];
                __syncwarp();
                tmem_ld32(lane_addr(tbase, quad, kColI + 64 * st + 32 * half), x);
                if (odd)
                    odd_row(tbase, quad, t, first, sm + kOffV + st * kTile, half, y);
                else
                    tmem_ld32(lane_addr(tbase, quad, kColO + 32 * half), y);
                landed(x);
                landed(y);
                if (half == 1) {
                    tc_fence_before();
                    mbar_arrive(&s.o_free);
                }
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    uint32_t f[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int i = 8 * q + 2 * e;
                        const f32x2 w = mul2(pack2(y[i], y[i + 1]), dup2(a.scale));
                        float lo, hi;
                        unpack2(start == 0.f ? w : fma2(pack2(x[i], x[i + 1]), dup2(start), w), lo, hi);
                        f[e] = narrow_pair(lo, hi);
                    }
                    if (t < n && 32 * half + 8 * q < nv) 
                        *reinterpret_cast<uint4 *>(o + 32 * half + 8 * q) = make_uint4(f[0], f[1], f[2], f[3]);
                }
            }
            if (odd) {
                named_sync(2, 128);
                if (t == 0) {
                    mbar_arrive(&s.v_free[st]);
                    mbar_arrive(&s.p_free);
                }
            }
        }
    } else if (warp == 16) {
        // ---- products
        if (lane == 0 && chunks > 0) {
            const uint32_t base = smem_u32(sm);
            const int steps = (dk + 15) / 16;  // of d_k
            const uint32_t id_qk = idesc_bf16_f32(128, 128, 0, 0), id_s = idesc_bf16_f32(128, 64, 0, 1),
                           id_u = idesc_bf16_f32(128, 64, 1, 1);
            auto k_step = [](int k) { return (uint32_t)(((k >> 2) * kTile + (k & 3) * 32) >> 4); };
            auto mn_step = [](int k) { return (uint32_t)(k * 2048 >> 4); };
            auto qk = [&](int st) {
                const uint64_t q = sdesc_sw128(base + kOffQ + st * 2 * kTile, 16, 1024);
                const uint64_t k = sdesc_sw128(base + kOffK + st * 2 * kTile, 16, 1024);
                for (int i = 0; i < steps; ++i) mma_f16kind(tbase + kColQK, q + k_step(i), k + k_step(i), id_qk, i > 0);
                mma_commit(&s.qk_full);
            };
            auto add = [&](int st) {
                const uint64_t k = sdesc_sw128(base + kOffK + st * 2 * kTile, kTile, 1024);
                for (int part = 0; part < 2; ++part) {
                    const uint64_t w = sdesc_sw128(base + kOffW + part * kTile, kTile, 1024);
                    for (int i = 0; i < 8; ++i)
                        mma_f16kind(tbase + kColU, k + mn_step(i), w + mn_step(i), id_u, part + i > 0);
                }
                mma_commit(&s.u_full);
            };
            auto inter = [&](int st) {
                const uint64_t q = sdesc_sw128(base + kOffQ + st * 2 * kTile, 16, 1024);
                for (int part = 0; part < 2; ++part) {
                    const uint64_t S = sdesc_sw128(base + kOffS + part * kTile, kTile, 1024);
                    for (int i = 0; i < steps; ++i)
                        mma_f16kind(tbase + kColI + 64 * st, q + k_step(i), S + mn_step(i), id_s, part + i > 0);
                }
                mma_commit(&s.kq_free[st]);
            };
            auto intra = [&](int st) {
                const uint64_t v = sdesc_sw128(base + kOffV + st * kTile, kTile, 1024);
                for (int part = 0; part < 2; ++part)
                    for (int i = 0; i < 8; ++i)
                        mma_f16kind_ts(tbase + kColO, tbase + kColP + 64 * part + 8 * i, v + mn_step(i), id_s, part + i > 0);
                mma_commit(&s.o_full);
            };
            if (states_only) {
                for (int c = 0; c < chunks; ++c) {
                    const int st = c & 1;
                    wait(&s.full[st], c >> 1);
                    wait(&s.w_ready[st], c >> 1);
                    if (c > 0) wait(&s.u_free, c - 1);
                    tc_fence_after();
                    add(st);
                    mma_commit(&s.kq_free[st]);
                    mma_commit(&s.v_free[st]);
                }
            } else {
                auto ahead = [&](int c) {  // what chunk c needs beside P
                    const int st = c & 1;
                    wait(&s.w_ready[st], c >> 1);
                    if (c > 0) wait(&s.u_free, c - 1);
                    tc_fence_after();
                    add(st);
                    wait(&s.s_ready, c);
                    tc_fence_after();
                    inter(st);
                };
                wait(&s.full[0], 0);
                tc_fence_after();
                qk(0);
                ahead(0);
                for (int c = 0; c < chunks; ++c) {
                    const int st = c & 1;
                    wait(&s.p_ready, c);
                    if (c + 1 < chunks) {
                        wait(&s.full[st ^ 1], (c + 1) >> 1);
                        tc_fence_after();
                        qk(st ^ 1);
                    }
                    if (c > 0) wait(&s.o_free, c - 1);
                    tc_fence_after();
                    intra(st);
                    if (c + 1 < chunks) ahead(c + 1);
                }
            }
        }
    } else if (warp == 17 && lane == 0) {
        // ---- tensor copies
        const int g = h / (a.heads / a.groups), halves = dk > 64 ? 2 : 1;
        const uint32_t bytes = (uint32_t)(halves * (states_only ? 1 : 2) + 1) * kTile;
        for (int c = 0; c < chunks; ++c) {
            const int st = c & 1, row = (int)(u.row + (int64_t)c * kC);
            if (c > 1) {
                wait(&s.kq_free[st], (c - 2) >> 1);
                wait(&s.v_free[st], (c - 2) >> 1);
            }
            if (*abort_flag) break;
            mbar_arrive_expect_tx(&s.full[st], bytes);
            for (int i = 0; i < halves; ++i) {
                tma_load_3d(sm + kOffK + (st * 2 + i) * kTile, &tm_k, &s.full[st], 64 * i, g, row);
                if (!states_only) tma_load_3d(sm + kOffQ + (st * 2 + i) * kTile, &tm_q, &s.full[st], 64 * i, g, row);
            }
            tma_load_3d(sm + kOffV + st * kTile, &tm_v, &s.full[st], v0, h, row);
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc(tbase, 512);
    }
}

PFN_cuTensorMapEncodeTiled_v12000 encoder()
{
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        cudaDriverEntryPointQueryResult q;
        void *p = nullptr;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    });
    return fn;
}

// [rows][heads][width] bf16 with a row stride, in boxes of 128 rows x 1 head x 64.
bool make_map(CUtensorMap *m, const void *base, int64_t rows, int heads, int width, int64_t ld)
{
    const cuuint64_t dim[3] = {(cuuint64_t)width, (cuuint64_t)heads, (cuuint64_t)rows};
    const cuuint64_t stride[2] = {(cuuint64_t)width * 2, (cuuint64_t)ld * 2};
    const cuuint32_t box[3] = {64, 1, (cuuint32_t)kC}, es[3] = {1, 1, 1};
    return encoder()(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dim, stride, box, es,
                     CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

bool gdn_linattn_tc_supported(const GdnLinattnArgs &a)
{
    const int64_t rows = a.cu_seqlens ? a.T : (int64_t)a.N * a.T;
    // tensor copies take strides that are multiples of 16 bytes, below 2^40
    return a.dtype == 1 && a.dk % 8 == 0 && a.dv % 8 == 0 && (a.ld_q | a.ld_k | a.ld_v | a.ld_o) % 8 == 0 &&
           a.ld_q < ((int64_t)1 << 38) && a.ld_k < ((int64_t)1 << 38) && a.ld_v < ((int64_t)1 << 38) && rows > 0 &&
           rows < ((int64_t)1 << 31) - 2 * kC && aligned16(a.q) && aligned16(a.k) && aligned16(a.v) && aligned16(a.o) &&
           encoder();
}

cudaError_t gdn_linattn_tc(const GdnLinattnArgs &a, bool states_only, cudaStream_t s)
{
    const int64_t rows = a.cu_seqlens ? a.T : (int64_t)a.N * a.T;
    const int tiles = (a.dv + kDVT - 1) / kDVT;
    const int64_t blocks = (a.segment ? a.pieces : a.N) * a.heads * tiles;
    if (blocks > 0x7fffffff) return cudaErrorInvalidConfiguration;
    CUtensorMap q, k, v;
    if (!make_map(&q, a.q, rows, a.groups, a.dk, a.ld_q) || !make_map(&k, a.k, rows, a.groups, a.dk, a.ld_k) ||
        !make_map(&v, a.v, rows, a.heads, a.dv, a.ld_v))
        return cudaErrorInvalidValue;
    const cudaError_t e = cudaFuncSetAttribute(gdn_linattn_tc_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
    if (e != cudaSuccess) return e;
    gdn_linattn_tc_kernel<<<(unsigned)blocks, kThreads, kSmemBytes, s>>>(a, tiles, states_only, q, k, v);
    return cudaGetLastError();
}

// Linear attention with a decay for each head on the tensor cores: bf16 in and
// out, fp32 sums and states.
//
// A block takes one (sequence or piece, head, 64 columns of v) and walks it in
// chunks of 128 tokens.  With b the sum of log decays up to and with a token of
// the chunk, and S^T (d_k x 64) the state before it:
//
//   P   = scale Lower(Q K^T e^{b_i - b_j})            [128 x 128]
//   O   = scale e^{b_i} Q S^T + P V                   [128 x 64]
//   U   = K^T (V e^{b_n - b_j})                       [d_k x 64]
//   S^T <- e^{b_n} S^T + U
//
// Only the last line is serial, and it is 64 fused multiply-adds a thread: the
// state stays in the registers of four warps, fp32, for the whole walk, and none
// of the products waits for more than the one before it.  Q, K and V enter as they
// are (products of bf16 are exact in fp32), and sums are fp32.  The decayed V enters
// as three bf16 parts, whose sum is the value to fp32: final states are 3e-7 to 6e-7 off
// in the 2-norm (two parts: 2.0e-6).  P and the state enter the outputs' products as two
// bf16 parts each, which leave 2^-16: outputs are off by their own rounding, 1.7e-3 (one
// part each: 2.3e-3).
//
// 4 x 4096 tokens x 16 heads of 128: 98.6 us, 2.8 TB/s, 41 % of the HBM copy rate; a chunk
// takes 2.6 us.  No one thing bounds it: with the tensor pipe busy for 49 % of the time on
// the multiprocessors that have a block, each scheduler issues in 45 % of its cycles and
// shared memory moves some 510 KB a chunk, most of what 128 bytes a cycle are.  Left out, P's
// second parts gave back 4 us, the outputs' half 5, the copies of Q 4.  Both parts of S^T as
// one product of 128 columns, Q read once, took 96 us where this took 94: its sums then have
// one stage.  Larger loops took 108: warps waited for instructions 1.9 times an issue, now 0.8.
//
// Roles, in groups of four warps: forming P (tensor memory to tensor memory, a row per
// thread), keeping the state and writing its parts for the next chunk, summing the
// decays and forming the decayed V, writing the outputs; then single warps that issue
// P V, K^T V, Q S^T and Q K^T, and the tensor copies into rings of two stages (K and V)
// and one (Q, whose next tile comes after Q S^T: the second part of S^T has the room),
// with later chunks fetched to L2 ahead.  All loops over chunks are kept small, rare paths
// in functions of their own: together they have to stay in the instruction cache.
//
// Every wait is bounded: on timeout the block raises GDN_DEV_WAIT_TIMEOUT, issues no more
// copies and winds down with waits of 50 us, enough for what is in flight; who issued
// products or copies waits for the last of them.
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
// Warps: four that form P, kSG groups of four that keep the state (kDVT / kSG columns
// each), and so on.
constexpr int kSG = 1;
constexpr int kWarpS = 4, kWarpW = kWarpS + 4 * kSG, kWarpO = kWarpW + 4, kWarpIssue = kWarpO + 4;
constexpr int kThreads = (kWarpIssue + 4) * 32;
constexpr int kParts = 3;   // of the decayed V
constexpr int kHalves = 2;  // parts of P and of the state
constexpr int kRing = 3;    // stages of V, which the outputs take over: two of them wait for each other (98 us, three 94)
constexpr int kAhead = 3;   // chunks that are fetched to L2 ahead of the one that is copied
// Sums of decays within a block of 32, log 2, that go as products of two factors: from
// -kFall to kRise.  The factors are 2^-in_j 2^-kShift and 2^(sum up to i) 2^kShift, so that
// neither leaves what fp32 holds before their product is below 2^(kFall - 222).
constexpr float kFall = 90.f, kRise = 24.f, kShift = 96.f, kTwoShift = 7.9228162514264338e28f;
#ifndef GDN_WAIT_TEST
constexpr uint64_t kWaitLimitNs = 2000000000ull;
constexpr bool kWaitTest = false;
#else
// Test build: 5 ms per wait, and one warp that keeps the state withholds one arrival in the
// first block, the one that the state before chunk 1 is written.
constexpr uint64_t kWaitLimitNs = 5000000ull;
constexpr bool kWaitTest = true;
#endif
constexpr uint64_t kDrainNs = 50000;  // a wait's bound once the block has given up on one

// Shared memory: tiles of 128-byte rows, 128-byte swizzle.
constexpr int kTile = kC * 128;           // 128 rows
constexpr int kOffQ = 0;                  // 2 halves of d_k
constexpr int kOffK = kOffQ + 2 * kTile;  // 2 stages of them
constexpr int kOffV = kOffK + 4 * kTile;  // kRing stages
constexpr int kOffW = kOffV + kRing * kTile;  // decayed V in parts
constexpr int kOffS = kOffW + kParts * kTile;  // S^T in parts
constexpr int kOffSmall = kOffS + kHalves * kTile;

struct Small {
    // decays of two chunks: sums up to and with a token within its block of 32, their
    // inverse factors 2^(-in - kShift), for steep tokens and those behind them what the sum's
    // rounding leaves out, and the blocks' sums
    float in[2][kC], inverse[2][kC], total[2][4];
    unsigned mask[2][4], steep[2][4];  // tokens that forget; whose sum is beyond kFall or kRise
    unsigned odd[2][4];     // tokens whose V has infinities or NaN
    uint64_t k_full[2], v_full[kRing], k_free[2], v_free[kRing], dec_ready[2], dec_free[2], w_ready[2], o_free[2], qk_full[2],
        p_ready[2], p_free[2], o_staged[kRing], i_full[2], w_half[2], w_gone[2];
    uint64_t drained[3], odd_read, q_full, q_free, u_full, u_free, s_ready, o_full;
    uint32_t tmem;
    int abort_flag;
};
constexpr int kSmemBytes = kOffSmall + (int)sizeof(Small);
static_assert(kSmemBytes <= 232448, "shared memory per block");

// Tensor memory, 512 columns: Q K^T, then P in its place, x 2 | Q S^T x 2 | P V | U.
// The parts of P of 16 tokens take the columns of their 16 products: 8 and 8.
constexpr uint32_t kColP = 0, kColI = 256, kColO = 384, kColU = 448;

// A wait suspends the warp for as long as the hardware lets it; the clock is looked at
// now and then.
__device__ __noinline__ void wait_long(uint64_t *bar, uint32_t parity, volatile int *abort_flag, unsigned int *status)
{
    const uint64_t limit = *abort_flag ? kDrainNs : kWaitLimitNs;
    uint64_t from = 0;
    for (unsigned i = 0;; ++i) {
        if (mbar_try_wait(bar, parity)) return;
        if (i % 16 == 0) {
            const uint64_t now = globaltimer_ns();
            if (i == 0) from = now;
            if (now - from > limit) break;
        }
    }
    *abort_flag = 1;
    atomicOr(status, GDN_DEV_WAIT_TIMEOUT);
}

// Products in place in rare branches: as statements of their own they stay there, where the
// compiler would form them beside the old values, and registers do not hold both.
__device__ __forceinline__ void mul_here(float &x, float f) { asm volatile("mul.rn.f32 %0, %0, %1;" : "+f"(x) : "f"(f)); }
__device__ __forceinline__ void opaque(float &x) { asm volatile("" : "+f"(x)); }  // no path of its own for each value
__device__ __forceinline__ void mul2_here(f32x2 &x, f32x2 f) { asm volatile("mul.rn.f32x2 %0, %0, %1;" : "+l"(x) : "l"(f)); }

// One arrival for the warp, after all of its lanes.
__device__ __forceinline__ void arrive_warp(uint64_t *bar)
{
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}

// This thread's products have ended before tensor memory is freed, also where the waits for
// them gave up.
__device__ __noinline__ void drain(uint64_t *bar, volatile int *abort_flag, unsigned int *status)
{
    mma_commit(bar);
    if (!mbar_try_wait(bar, 0)) wait_long(bar, 0, abort_flag, status);
}

struct Waiter {
    volatile int *abort_flag;
    unsigned int *status;
    __device__ __forceinline__ void operator()(uint64_t *bar, int phase) const
    {
        if (!mbar_try_wait(bar, phase & 1)) wait_long(bar, phase & 1, abort_flag, status);
    }
};

__device__ __forceinline__ uint32_t lane_addr(uint32_t tbase, int quad, uint32_t col)
{
    return tbase + (static_cast<uint32_t>(quad * 32) << 16) + col;
}

// One thread of the warp, the same each time: products and tensor copies are issued by
// one thread, and the compiler has to know that it is one.
__device__ __forceinline__ bool elect_one()
{
    uint32_t is;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(is));
    return is != 0;
}

__device__ __forceinline__ void fetch_l2(const CUtensorMap *map, int x, int y, int z)
{
    asm volatile("cp.async.bulk.prefetch.tensor.3d.L2.global.tile [%0, {%1, %2, %3}];" ::"l"(map), "r"(x), "r"(y), "r"(z)
                 : "memory");
}

// Columns of this thread's lane.  A load and its wait are one statement: nothing the
// compiler does with the registers, a move or a spill, comes between them.
__device__ __forceinline__ void ld_cols(uint32_t taddr, float (&v)[32])
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31},\n\t[%32];\n\ttcgen05.wait::ld.sync.aligned;"
        : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]),
          "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15]),
          "=f"(v[16]), "=f"(v[17]), "=f"(v[18]), "=f"(v[19]), "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23]),
          "=f"(v[24]), "=f"(v[25]), "=f"(v[26]), "=f"(v[27]), "=f"(v[28]), "=f"(v[29]), "=f"(v[30]), "=f"(v[31])
        : "r"(taddr));
}

__device__ __forceinline__ void ld_cols(uint32_t taddr, float (&v)[16])
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n\ttcgen05.wait::ld.sync.aligned;"
        : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]),
          "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15])
        : "r"(taddr));
}

__device__ __forceinline__ void ld_cols(uint32_t ta, uint32_t tb, float (&v)[16], float (&w)[16])
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%32];\n\t"
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%33];\n\ttcgen05.wait::ld.sync.aligned;"
        : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]),
          "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15]),
          "=f"(w[0]), "=f"(w[1]), "=f"(w[2]), "=f"(w[3]), "=f"(w[4]), "=f"(w[5]), "=f"(w[6]), "=f"(w[7]),
          "=f"(w[8]), "=f"(w[9]), "=f"(w[10]), "=f"(w[11]), "=f"(w[12]), "=f"(w[13]), "=f"(w[14]), "=f"(w[15])
        : "r"(ta), "r"(tb));
}

__device__ __forceinline__ uint32_t ld_col(uint32_t taddr)
{
    uint32_t v;
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];\n\ttcgen05.wait::ld.sync.aligned;" : "=r"(v) : "r"(taddr));
    return v;
}

// What the rounding of two values to a pair of bf16 leaves.
__device__ __forceinline__ f32x2 rest_of(f32x2 v, uint32_t part)
{
    return fma2(pack2(__uint_as_float(part << 16), __uint_as_float(part & 0xffff0000u)), dup2(-1.f), v);
}

__device__ __forceinline__ uint32_t narrow2(f32x2 v)
{
    float x, y;
    unpack2(v, x, y);
    return narrow_pair(x, y);
}

// Two values as pairs of three bf16 parts, each the rounded rest of those before it: their
// sum is the value to 2^-24.  `sign` becomes NaN where a value is infinite or NaN, whose
// other parts then are NaN.
__device__ __forceinline__ void split3(f32x2 v, uint32_t (&part)[kParts], f32x2 &sign)
{
    part[0] = narrow2(v);
    v = rest_of(v, part[0]);
    sign = fma2(v, dup2(0.f), sign);
    part[1] = narrow2(v);
    part[2] = narrow2(rest_of(v, part[1]));
}

// The same as two parts, to 2^-16, for outputs.  The second of an infinite value would be
// NaN: the greater of it and -2^112 is that number, which its products with the other
// factor do not bring up to the first's infinity.  (Values beyond 2^120 lose their second part
// to it at worst.)
__device__ __forceinline__ void split2(f32x2 v, uint32_t &hi, uint32_t &lo)
{
    hi = narrow2(v);
    asm("max.bf16x2 %0, %1, %2;" : "=r"(lo) : "r"(narrow2(rest_of(v, hi))), "r"(0xf780f780u));
}

__device__ __forceinline__ bool is_odd(f32x2 sign)
{
    float x, y;
    unpack2(sign, x, y);
    return x + y != 0.f;
}

// Other parts where the first is infinite or NaN: zero.
__device__ __forceinline__ uint32_t mend(uint32_t hi, uint32_t lo)
{
    if ((hi & 0x7f80u) == 0x7f80u) lo &= 0xffff0000u;
    if ((hi & 0x7f800000u) == 0x7f800000u) lo &= 0xffffu;
    return lo;
}

__device__ __noinline__ void mend_row(uint8_t *tiles, int r)
{
#pragma unroll 1
    for (int w = 0; w < 32; ++w) {
        const uint32_t at = sw128(r, w / 4) + w % 4 * 4;
        for (int p = 1; p < kParts; ++p) {
            uint32_t *lo = reinterpret_cast<uint32_t *>(tiles + p * kTile + at);
            *lo = mend(*reinterpret_cast<const uint32_t *>(tiles + at), *lo);
        }
    }
}

// The decayed row where the decay is zero but no token forgets: the infinities and NaN of V stay.
__device__ __noinline__ void keep_odd_row(uint8_t *tiles, const uint8_t *V, int r)
{
#pragma unroll 1
    for (int w = 0; w < 32; ++w) {
        const uint32_t at = sw128(r, w / 4) + w % 4 * 4;
        uint32_t hi = *reinterpret_cast<const uint32_t *>(V + at);
        if ((hi & 0x7f80u) != 0x7f80u) hi &= 0xffff0000u;
        if ((hi & 0x7f800000u) != 0x7f800000u) hi &= 0xffffu;
        for (int p = 0; p < kParts; ++p) *reinterpret_cast<uint32_t *>(tiles + p * kTile + at) = p ? 0u : hi;
    }
}

__device__ __noinline__ void zero_row(uint8_t *tiles, int r)
{
#pragma unroll 1
    for (int c = 0; c < 8 * kParts; ++c)
        *reinterpret_cast<uint4 *>(tiles + (c >> 3) * kTile + sw128(r, c & 7)) = make_uint4(0, 0, 0, 0);
}

// Whether a row of K, in `halves` tiles, has infinities or NaN; and zeros in its place.
__device__ __noinline__ bool odd_k_row(const uint8_t *K, int r, int halves)
{
    bool odd = false;
#pragma unroll 1
    for (int c = 0; c < 8 * halves; ++c) {
        const uint4 x = *reinterpret_cast<const uint4 *>(K + (c >> 3) * kTile + sw128(r, c & 7));
        for (uint32_t w : {x.x, x.y, x.z, x.w}) odd |= (w & 0x7f80u) == 0x7f80u || (w & 0x7f800000u) == 0x7f800000u;
    }
    return odd;
}

__device__ __noinline__ void zero_k_row(uint8_t *K, int r, int halves)
{
#pragma unroll 1
    for (int c = 0; c < 8 * halves; ++c)
        *reinterpret_cast<uint4 *>(K + (c >> 3) * kTile + sw128(r, c & 7)) = make_uint4(0, 0, 0, 0);
}

// 8 values into 16-byte column c of row r, in parts into tiles one after another.
__device__ __forceinline__ void st_parts(uint8_t *tiles, int r, int c, const f32x2 (&x)[4], f32x2 &sign)
{
    uint32_t w[4][kParts];
#pragma unroll
    for (int i = 0; i < 4; ++i) split3(x[i], w[i], sign);
    const uint32_t at = sw128(r, c);
#pragma unroll
    for (int p = 0; p < kParts; ++p)
        *reinterpret_cast<uint4 *>(tiles + p * kTile + at) = make_uint4(w[0][p], w[1][p], w[2][p], w[3][p]);
}

// The column of P's first part of token pair w; of the second, 8 more.
__device__ __forceinline__ int pair_at(int w) { return w / 8 * 16 + w % 8; }

// P of 16 tokens as parts, in place of the products.
__device__ __forceinline__ void st_p(uint32_t at, const float (&x)[16])
{
    uint32_t w[16];
#pragma unroll
    for (int j = 0; j < 8; ++j) split2(pack2(x[2 * j], x[2 * j + 1]), w[j], w[8 + j]);
    tmem_st16(at, w);
}

// The factor of a row whose sum of decays is x, and of the scale, times 2^kShift.  The
// exponent is shifted only where that costs none of its digits.
__device__ __forceinline__ float row_factor(float x, float scale)
{
    const bool far = x < -64.f;
    const float f = decay_of(far ? x + kShift : x) * scale;
    return far ? f : f * kTwoShift;
}

// P of one row in the cases that the plain path leaves: tokens that forget, and sums of
// decays beyond kFall and kRise, over blocks too.  An exponential an entry: 309 us where the
// plain path takes 98, if every block of 32 goes this way.  Rows that come before any such
// token (`own` false) have the plain path's factors: the same bits, whatever comes later.
__device__ __noinline__ void odd_decays(uint32_t p, int quad, int I, int lane, bool own, float scale, const float *in,
                                        const float *inverse, const float *total, const unsigned *mask, const unsigned *steep)
{
    auto rest = [&](int J, int j) { return (mask[J] | steep[J]) & (0xffffffffu >> (31 - j)) ? inverse[32 * J + j] : 0.f; };
    const float mine = in[32 * I + lane], mine_rest = rest(I, lane);
    float sum = mine;
    bool cut = mask[I] & (0xffffffffu >> (31 - lane));
    const int first = first_seen(mask[I], lane);
#pragma unroll 1
    for (int J = I; J >= 0; --J) {
        const float last = in[32 * J + 31], last_rest = rest(J, 31), plain = row_factor(J == I ? sum : sum + total[J], scale);
#pragma unroll 1
        for (int from = 0; from < 32; from += 16) {
            float x[16];
            ld_cols(lane_addr(p, quad, 32 * J + from), x);
            const unsigned late = (mask[J] | steep[J]) ? ~0u << (__ffs(mask[J] | steep[J]) - 1) : 0;  // tokens with a rest
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                const int j = from + e;
                const float w = in[32 * J + j], other = inverse[32 * J + j], left = late >> j & 1 ? other : 0.f;
                const bool seen = J == I ? j <= lane && j >= first : !cut && !(mask[J] & (0xfffffffeu << j));
                const float f = own ? decay_of(J == I ? mine - w + (mine_rest - left) : sum + (last - w + (last_rest - left))) * scale
                                    : plain * other;
                x[e] = !seen ? 0.f : f != 0.f ? x[e] * f : copysignf(0.f, x[e] * copysignf(1.f, f));  // zeros keep their sign
            }
            __syncwarp();
            st_p(lane_addr(p, quad, 32 * J + from), x);
        }
        if (J < I) {
            sum += total[J];
            cut = cut || mask[J];
        }
    }
}

// A row of V that has infinities or NaN, as P V gets it: in their place the smallest
// numbers there are, one for each kind, which are lost in any sum.  A token must see
// nothing of those behind it, and zero times infinity is NaN; who sees the row gets its
// infinities from odd_row.
__device__ __noinline__ void code_row(uint8_t *V, int r)
{
#pragma unroll 1
    for (int w = 0; w < 32; ++w) {
        uint32_t *at = reinterpret_cast<uint32_t *>(V + sw128(r, w / 4) + w % 4 * 4);
        uint32_t out = 0;
#pragma unroll
        for (int e = 0; e < 32; e += 16) {
            const uint32_t h = *at >> e & 0xffffu, m = h & 0x7fffu;
            out |= (m > 0x7f80u ? 2u : m == 0x7f80u ? (h & 0x8000u) | 1u : m < 3u ? 0u : h) << e;
        }
        *at = out;
    }
}

// What the coded rows of V add to P V of a token that sees them, tokens `first` to i: to the
// columns at o.
__device__ __noinline__ void odd_row(uint32_t p, uint32_t o, int quad, int i, int first, const unsigned *rows, const uint8_t *V)
{
#pragma unroll 1
    for (int part = 0; part < 4; ++part) {
        float acc[16];
        ld_cols(lane_addr(o, quad, 16 * part), acc);
#pragma unroll 1
        for (int j = 0; j < kC; ++j) {
            if (!(rows[j >> 5] >> (j & 31) & 1)) continue;
            __syncwarp();
            const uint32_t hi = ld_col(lane_addr(p, quad, pair_at(j >> 1))), lo = ld_col(lane_addr(p, quad, pair_at(j >> 1) + 8));
            if (j > i || j < first) continue;
            const float h = __uint_as_float(j & 1 ? hi & 0xffff0000u : hi << 16);
            const float f = h == 0.f ? copysignf(1.f, h) : h + __uint_as_float(j & 1 ? lo & 0xffff0000u : lo << 16);
#pragma unroll
            for (int d = 0; d < 16; ++d) {
                const uint32_t v = *reinterpret_cast<const unsigned short *>(V + sw128(j, part * 2 + d / 8) + d % 8 * 2);
                if ((v & 0x7fffu) - 1u < 2u) acc[d] = fmaf(f, __uint_as_float(v == 2u ? 0x7fc00000u : (v & 0x8000u) << 16 | 0x7f800000u), acc[d]);
            }
        }
        __syncwarp();
        uint32_t out[16];
#pragma unroll
        for (int d = 0; d < 16; ++d) out[d] = __float_as_uint(acc[d]);
        tmem_st16(lane_addr(o, quad, 16 * part), out);
        tmem_st_wait();
    }
}

__device__ __noinline__ float exact_sum(Decays &d, float log_decay) { return d.exact(log_decay); }

// The 32 tokens of a chunk whose rows of Q, P and O are in the lanes of a quarter of
// tensor memory, which only every fourth warp, those of one scheduler, can reach.  The
// last tokens have four blocks of P to form, the first one: they change places in every
// other chunk.
__device__ __forceinline__ int row_block(int quad, int chunk) { return chunk & 1 ? 3 - quad : quad; }

// Descriptor steps of 16 along K, K-major (64 to a row) and MN-major (rows).
__device__ __forceinline__ constexpr uint32_t k_step(int k) { return ((k >> 2) * kTile + (k & 3) * 32) >> 4; }
__device__ __forceinline__ constexpr uint32_t mn_step(int k) { return k * 2048 >> 4; }

// kStates: what pieces add to the state, without outputs.  KS: steps of 16 over d_k
// (up to there tiles are filled up with zeros).
template <bool kStates, int KS>
__global__ void __launch_bounds__(kThreads, 1)
gdn_linattn_tc_kernel(const GdnLinattnArgs a, int tiles, const __grid_constant__ CUtensorMap tm_q,
                      const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                      const __grid_constant__ CUtensorMap tm_o)
{
    extern __shared__ __align__(1024) uint8_t sm[];
    Small &s = *reinterpret_cast<Small *>(sm + kOffSmall);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, quad = warp & 3, t = tid & 127;
    const int64_t unit = blockIdx.x;
    const int v0 = (int)(unit % tiles) * kDVT, h = (int)(unit / tiles % a.heads);
    Unit u;
    if (!find_unit(a, unit / tiles / a.heads, h, kStates, u)) return;
    const int chunks = (int)(((int64_t)u.len + kC - 1) / kC), dk = a.dk;

    // Tensor copies of a chunk's K or Q, to shared memory or ahead to L2, and of its V.
    const int g = h / (a.heads / a.groups), halves = dk > 64 ? 2 : 1;
    auto row = [&](int c) { return (int)(u.row + (int64_t)c * kC); };
    auto load_k = [&](int c, bool ahead) {
        uint64_t *bar = &s.k_full[c & 1];
        if (!ahead) mbar_arrive_expect_tx(bar, (uint32_t)halves * kTile);
#pragma unroll 1
        for (int i = 0; i < halves; ++i)
            if (ahead) fetch_l2(&tm_k, 64 * i, g, row(c));
            else tma_load_3d(sm + kOffK + ((c & 1) * 2 + i) * kTile, &tm_k, bar, 64 * i, g, row(c));
    };
    auto load_q = [&](int c, bool ahead) {
        if (!ahead) mbar_arrive_expect_tx(&s.q_full, (uint32_t)halves * kTile);
#pragma unroll 1
        for (int i = 0; i < halves; ++i)
#pragma unroll 1
            for (int b = 0; b < 4; ++b) {
                const int from = row(c) + 32 * row_block(b, c);
                if (ahead) fetch_l2(&tm_q, 64 * i, g, from);
                else tma_load_3d(sm + kOffQ + i * kTile + b * (kTile / 4), &tm_q, &s.q_full, 64 * i, g, from);
            }
    };
    auto load_v = [&](int c) {
        mbar_arrive_expect_tx(&s.v_full[c % kRing], kTile);
        tma_load_3d(sm + kOffV + c % kRing * kTile, &tm_v, &s.v_full[c % kRing], v0, h, row(c));
        if (c + kAhead < chunks) fetch_l2(&tm_v, v0, h, row(c + kAhead));
    };
    if (warp == kWarpIssue + 3 && elect_one()) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s.k_full[i], 1);
            mbar_init(&s.k_free[i], kStates ? 1 : 2);
            mbar_init(&s.p_free[i], 1);
            mbar_init(&s.dec_ready[i], 4);
            mbar_init(&s.dec_free[i], 4 * (kStates ? kSG : kSG + 2) + (kStates ? 0 : 1));
            mbar_init(&s.w_ready[i], 4);
            mbar_init(&s.o_free[i], 4);
            mbar_init(&s.qk_full[i], 1);
            mbar_init(&s.i_full[i], 1);
            mbar_init(&s.w_half[i], 2);
            mbar_init(&s.w_gone[i], 1);
            mbar_init(&s.p_ready[i], 4);
        }
        for (int i = 0; i < kRing; ++i) {
            mbar_init(&s.v_full[i], 1);
            mbar_init(&s.v_free[i], 1);
            mbar_init(&s.o_staged[i], 4);
        }
        for (int i = 0; i < 3; ++i) mbar_init(&s.drained[i], 1);
        mbar_init(&s.odd_read, 4);
        mbar_init(&s.q_full, 1);
        mbar_init(&s.q_free, 1);
        mbar_init(&s.u_full, 1);
        mbar_init(&s.u_free, 4 * kSG);
        mbar_init(&s.s_ready, 4 * kSG);
        mbar_init(&s.o_full, 1);
        s.abort_flag = 0;
        fence_mbar_init();
        fence_async_smem();
        // the first chunks are on their way while tensor memory is allocated
#pragma unroll 1
        for (int c = 0; c < 2 && c < chunks; ++c) load_k(c, false);
        if (!kStates && chunks > 0) load_q(0, false);
#pragma unroll 1
        for (int c = 0; c < kRing && c < chunks; ++c) load_v(c);
#pragma unroll 1
        for (int c = 1; c < 2 + kAhead && c < chunks; ++c) {
            if (c > 1) load_k(c, true);
            if (!kStates && c < 1 + kAhead) load_q(c, true);
        }
        prefetch_tensormap(&tm_o);
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

    if (warp < kWarpS) {
        // ---- P, in the place of Q K^T: a row per thread, blocks of 32 columns up to its own
        if constexpr (!kStates) {
            const float limit = 28.f - log2f(fabsf(a.scale));  // row_factor stays below 2^124
#pragma unroll 1
            for (int c = 0; c < chunks; ++c) {
                const int st = c & 1, I = row_block(quad, c);
                const uint32_t p = tbase + kColP + 128 * st;
                wait(&s.dec_ready[st], c >> 1);
                // The factor of tokens i and j is 2^(in_i + the blocks between + total_J) 2^-in_j, where J is the
                // block of j; within a block without the other sums.
                float sum = s.in[st][32 * I + lane];
                const unsigned here = s.mask[st][I] | s.steep[st][I];
                bool own = here & (0xffffffffu >> (31 - lane));
                float most = sum;
#pragma unroll 1
                for (int J = I; J >= 0; --J) {
                    if (J < I) most += s.total[st][J], own |= s.mask[st][J] || s.steep[st][J];
                    own |= !(most <= limit);
                }
                const bool odd = __any_sync(0xffffffffu, own);
                wait(&s.qk_full[st], c >> 1);
                __syncwarp();
                tc_fence_after();
                if (odd) odd_decays(p, quad, I, lane, own, a.scale, s.in[st], s.inverse[st], s.total[st], s.mask[st], s.steep[st]);
#pragma unroll 1
                for (int J = I; J >= 0 && !odd; --J) {
                    const f32x2 f = dup2(row_factor(sum, a.scale));
#pragma unroll 1
                    for (int from = 0; from < 32; from += 16) {
                        const uint32_t at = lane_addr(p, quad, 32 * J + from);
                        const float4 *inverse = reinterpret_cast<const float4 *>(&s.inverse[st][32 * J + from]);
                        float x[16];
                        ld_cols(at, x);
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const float4 w = inverse[j];
                            unpack2(mul2(pack2(x[4 * j], x[4 * j + 1]), mul2(f, pack2(w.x, w.y))), x[4 * j], x[4 * j + 1]);
                            unpack2(mul2(pack2(x[4 * j + 2], x[4 * j + 3]), mul2(f, pack2(w.z, w.w))), x[4 * j + 2], x[4 * j + 3]);
                        }
                        if (J == I) {  // the factor of a token behind may be infinite: a rise, then a fall
#pragma unroll
                            for (int j = 0; j < 16; ++j) x[j] = from + j <= lane ? x[j] : 0.f;
                        }
                        st_p(at, x);
                    }
                    if (J > 0) sum += s.total[st][J - 1];
                }
                const float zero[32] = {};
#pragma unroll 1
                for (int J = I + 1; J < 4; ++J) tmem_st32(lane_addr(p, quad, 32 * J), zero);
                tmem_st_wait();
                tc_fence_before();
                arrive_warp(&s.dec_free[st]);
                arrive_warp(&s.p_ready[st]);
            }
        }
    } else if (warp < kWarpW) {
        // ---- the state: kCols columns of row t of S^T
        constexpr int kCols = kDVT / kSG;
        const int c0 = (warp - kWarpS) / 4 * kCols;
        f32x2 S[kCols / 2];
        const bool mine = 32 * quad < dk;  // the others' rows are not part of S
        const int64_t at = (int64_t)(v0 + c0) * dk + t;
        const int cols = t < dk ? a.dv - v0 - c0 : 0;
        {
            const float *p = u.in + at;
            const int n = u.in ? cols : 0;
#pragma unroll
            for (int d = 0; d < kCols; d += 2) {
                const float x = d < n ? *p : 0.f;
                p += dk;
                S[d / 2] = pack2(x, d + 1 < n ? *p : 0.f);
                p += dk;
            }
        }
        PieceDecay piece;
#pragma unroll 1
        for (int c = -1; c < chunks; ++c) {
            const int st = c & 1;
            if (c >= 0) {
                wait(&s.dec_ready[st], c >> 1);
                const float4 total = *reinterpret_cast<const float4 *>(s.total[st]);
                const uint4 mask = *reinterpret_cast<const uint4 *>(s.mask[st]);
                const float sum = total.x + total.y + total.z + total.w;
                const unsigned cut = mask.x | mask.y | mask.z | mask.w;
                if (kStates && t == 0) piece.add(sum, cut);
                arrive_warp(&s.dec_free[st]);
                float all = cut ? 0.f : chained_decay_of(once(sum)), again = is_far(sum) ? all : 1.f;
                opaque(all), opaque(again);
                if (all == 0.f)
#pragma unroll
                    for (int d = 0; d < kCols / 2; ++d) S[d] = 0;  // forgotten, infinite or not
                if (again != 1.f) {
#pragma unroll
                    for (int d = 0; d < kCols / 2; ++d) mul2_here(S[d], dup2(again));
                }
                wait(&s.u_full, c);
                __syncwarp();
                tc_fence_after();
#pragma unroll
                for (int q = 0; q < kCols && mine; q += 16) {
                    float x[16];
                    ld_cols(lane_addr(tbase, quad, kColU + c0 + q), x);
#pragma unroll
                    for (int d = 0; d < 8; ++d)
                        S[q / 2 + d] = fma2(dup2(all), S[q / 2 + d], pack2(x[2 * d], x[2 * d + 1]));
                }
                tc_fence_before();
                arrive_warp(&s.u_free);
            }
            if (!kStates && c + 1 < chunks) {
                if (c >= 0) wait(&s.i_full[st], c >> 1);  // Q S^T of this chunk has read it
#pragma unroll
                for (int q = 0; q < kCols / 8 && (t < dk || c < 0); ++q) {  // the rows past d_k stay zero
                    uint32_t hi[4], lo[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) split2(S[4 * q + e], hi[e], lo[e]);
                    uint8_t *at = sm + kOffS + sw128(t, c0 / 8 + q);
                    *reinterpret_cast<uint4 *>(at) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                    *reinterpret_cast<uint4 *>(at + kTile) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
                }
                fence_async_smem();
                if (!(kWaitTest && blockIdx.x == 0 && c == 0 && warp == kWarpS)) arrive_warp(&s.s_ready);
            }
        }
        if (kStates && v0 + c0 == 0 && t == 0) a.piece_decay[unit / tiles] = piece.all();
        if (u.out && !*abort_flag) {
            float *p = u.out + at;
#pragma unroll
            for (int d = 0; d < kCols; d += 2) {
                float x, y;
                unpack2(S[d / 2], x, y);
                if (d < cols) *p = x;
                p += dk;
                if (d + 1 < cols) *p = y;
                p += dk;
            }
        }
    } else if (warp < kWarpO) {
        // ---- decays, and V times the decay to the chunk's end
        const float *decay = a.log_decay + (u.row + t) * a.ld_decay + h;
        float next = t < u.len ? *decay : 0.f;
#pragma unroll 1
        for (int c = 0; c < chunks; ++c) {
            const int st = c & 1, n = min(kC, u.len - c * kC);
            Decays d;
            const float now = next;
            d.scan(now);
            next = t + (int64_t)(c + 1) * kC < u.len ? decay[(int64_t)(c + 1) * kC * a.ld_decay] : 0.f;
            if (c > 1) wait(&s.dec_free[st], (c - 2) >> 1);
            const unsigned steep = __ballot_sync(0xffffffffu, !(d.in > -kFall && d.in < kRise));
            float inverse = ex2(-d.in) * (1.f / kTwoShift);
            if (steep || d.mask) {
                const float rest = exact_sum(d, now);
                if ((steep | d.mask) & (0xffffffffu >> (31 - lane))) inverse = rest;
            }
            s.in[st][t] = d.in;
            s.inverse[st][t] = inverse;
            if (lane == 0) {
                s.total[st][quad] = d.total;
                s.mask[st][quad] = d.mask;
                s.steep[st][quad] = steep;
                s.odd[st][quad] = 0;
            }
            arrive_warp(&s.dec_ready[st]);
            named_sync(1, 128);
            bool cut = d.cut_behind(lane);
            float sum = d.after;
#pragma unroll 1
            for (int J = quad + 1; J < 4; ++J) {
                cut = cut || s.mask[st][J];
                sum += s.total[st][J];
            }
            const float w = cut ? 0.f : decay_of(sum);
            wait(&s.v_full[c % kRing], c / kRing);
            if (n < kC) wait(&s.k_full[st], c >> 1);  // K's rows past the end, below
            if (c > 0) wait(&s.w_gone[quad >> 1], c - 1);  // the product has read the last chunk's
            uint8_t *V = sm + kOffV + c % kRing * kTile, *W = sm + kOffW, *K = sm + kOffK + st * 2 * kTile;
            if (t < n) {
                f32x2 sign = 0;
#pragma unroll 1
                for (int q = 0; q < 8; ++q) {
                    float f[8];
                    widen(*reinterpret_cast<const uint4 *>(V + sw128(t, q)), f);
                    f32x2 x[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) x[e] = mul2(pack2(f[2 * e], f[2 * e + 1]), dup2(w));
                    st_parts(W, t, q, x, sign);
                }
                if (is_odd(sign)) {  // infinite or NaN, decayed or not
                    if (cut) zero_row(W, t);  // what comes after has forgotten it
                    else if (w == 0.f) keep_odd_row(W, V, t);
                    else mend_row(W, t);
                    if (!kStates) {
                        atomicOr(&s.odd[st][quad], 1u << lane);
                        code_row(V, t);
                    }
                }
            } else {  // rows past the end may be another sequence's
                zero_row(W, t);
                zero_k_row(V, t, 1);
                zero_k_row(K, t, halves);
            }
            if (__any_sync(0xffffffffu, cut)) {  // an infinite K that is forgotten meets zeros of W: NaN
                wait(&s.k_full[st], c >> 1);
                const bool odd = cut && t < n && odd_k_row(K, t, halves);
                if (!kStates && __any_sync(0xffffffffu, odd)) wait(&s.qk_full[st], c >> 1);
                if (odd) zero_k_row(K, t, halves);
            }
            fence_async_smem();
            arrive_warp(&s.w_half[quad >> 1]);
            arrive_warp(&s.w_ready[st]);
        }
    } else if (warp < kWarpIssue) {
        // ---- outputs: a row per thread
        if constexpr (!kStates) {
            __nv_bfloat16 *o = static_cast<__nv_bfloat16 *>(a.o) + u.row * a.ld_o + (int64_t)h * a.dv + v0;
            const int nv = min(kDVT, a.dv - v0);
#pragma unroll 1
            for (int c = 0; c < chunks; ++c, o += kC * a.ld_o) {
                const int st = c & 1, n = min(kC, u.len - c * kC), I = row_block(quad, c), i = 32 * I + lane;
                wait(&s.dec_ready[st], c >> 1);
                const unsigned mask = s.mask[st][I];
                float sum = s.in[st][i];
                bool cut = mask & (0xffffffffu >> (31 - lane));
                int first = 32 * I + first_seen(mask, lane);  // the first token this one sees
#pragma unroll 1
                for (int J = I - 1; J >= 0; --J) {
                    if (!cut) first = 32 * J + first_seen(s.mask[st][J], 31);
                    cut = cut || s.mask[st][J];
                    sum += s.total[st][J];
                }
                const float from = decay_of(once(sum, -60.f));
                float again = is_far(sum, -60.f) ? from : 1.f;
                opaque(again);
                const f32x2 start = dup2(a.scale * from);
                wait(&s.w_ready[st], c >> 1);
                const uint4 odd = *reinterpret_cast<const uint4 *>(s.odd[st]);
                arrive_warp(&s.dec_free[st]);
                wait(&s.i_full[st], c >> 1);
                wait(&s.o_full, c);
                tc_fence_after();
                uint8_t *stage = sm + kOffV + c % kRing * kTile;  // V is through, but for odd_row
                if (odd.x | odd.y | odd.z | odd.w) {
                    const unsigned rows[4] = {odd.x, odd.y, odd.z, odd.w};
                    odd_row(tbase + kColP + 128 * st, tbase + kColO, quad, i, first, rows, stage);
                    tc_fence_before();  // Q K^T takes the place of the P that was read
                }
                arrive_warp(&s.odd_read);
                if (odd.x | odd.y | odd.z | odd.w) wait(&s.odd_read, c);  // a bounded wait, where warps that gave up differ
                if (t == 0) mbar_arrive(&s.p_free[st]);
                // Whole chunks go through the place of V and a tensor copy: rows stored from here would take a
                // transaction per row and store, half of what the memory pipe can do.
                const bool whole = n == kC;
                const int cols = i < n ? nv : 0;
                __nv_bfloat16 *row = o + i * a.ld_o;
#pragma unroll 1
                for (int q = 0; q < kDVT; q += 16) {
                    float x[16], y[16];
                    __syncwarp();
                    ld_cols(lane_addr(tbase, quad, kColI + 64 * st + q), lane_addr(tbase, quad, kColO + q), x, y);
                    if (again != 1.f)
#pragma unroll
                        for (int e = 0; e < 16; ++e) mul_here(x[e], again);
                    if (cut)  // nothing of the state before, infinite or not
#pragma unroll
                        for (int e = 0; e < 16; ++e) x[e] = 0.f;
                    uint32_t f[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        float lo, hi;
                        unpack2(fma2(pack2(x[2 * e], x[2 * e + 1]), start, pack2(y[2 * e], y[2 * e + 1])), lo, hi);
                        f[e] = narrow_pair(lo, hi);
                    }
                    const uint4 f0 = make_uint4(f[0], f[1], f[2], f[3]), f1 = make_uint4(f[4], f[5], f[6], f[7]);
                    if (whole) {
                        *reinterpret_cast<uint4 *>(stage + sw128(i, q / 8)) = f0;
                        *reinterpret_cast<uint4 *>(stage + sw128(i, q / 8 + 1)) = f1;
                    } else {
                        if (q < cols) *reinterpret_cast<uint4 *>(row + q) = f0;
                        if (q + 8 < cols) *reinterpret_cast<uint4 *>(row + q + 8) = f1;
                    }
                }
                tc_fence_before();
                arrive_warp(&s.o_free[st]);
                fence_async_smem();
                arrive_warp(&s.o_staged[c % kRing]);
            }
        }
    } else if (warp == kWarpIssue) {
        // ---- P V
        if (!kStates && elect_one()) {
            const uint32_t base = smem_u32(sm);
#pragma unroll 1
            for (int c = 0; c < chunks; ++c) {
                const int st = c & 1;
                const uint32_t p = tbase + kColP + 128 * st;
                wait(&s.w_ready[st], c >> 1);  // V is finite, and zero past the end
                mbar_arrive(&s.dec_free[st]);  // seen: two chunks on the barrier's phase would look like this one's
                wait(&s.p_ready[st], c >> 1);
                wait(&s.v_full[c % kRing], c / kRing);
                if (c > 0) wait(&s.o_free[st ^ 1], (c - 1) >> 1);
                tc_fence_after();
                const uint64_t v = sdesc_sw128(base + kOffV + c % kRing * kTile, kTile, 1024);
#pragma unroll 1
                for (int part = 0; part < kHalves; ++part)
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        mma_f16kind_ts(tbase + kColO, p + 16 * i + 8 * part, v + mn_step(i),
                                       idesc_bf16_f32(128, 64, 0, 1), part + i > 0);
                mma_commit(&s.o_full);
            }
            drain(&s.drained[0], abort_flag, a.status);
        }
    } else if (warp == kWarpIssue + 1) {
        // ---- K^T V, decayed
        if (elect_one()) {
            const uint32_t base = smem_u32(sm);
#pragma unroll 1
            for (int c = 0; c < chunks; ++c) {
                const int st = c & 1;
                wait(&s.k_full[st], c >> 1);
                if (c > 0) wait(&s.u_free, c - 1);
                const uint64_t k = sdesc_sw128(base + kOffK + st * 2 * kTile, kTile, 1024);
                const uint64_t w = sdesc_sw128(base + kOffW, kTile, 1024);
                // 64 tokens at a time: the next chunk's take their place while the others are still read
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    wait(&s.w_half[half], c);
                    tc_fence_after();
#pragma unroll 1
                    for (int part = 0; part < kParts; ++part)
#pragma unroll
                        for (int i = 4 * half; i < 4 * half + 4; ++i)
                            mma_f16kind(tbase + kColU, k + mn_step(i), w + part * (kTile >> 4) + mn_step(i),
                                        idesc_bf16_f32(128, 64, 1, 1), half + part + i > 0);
                    mma_commit(&s.w_gone[half]);
                }
                mma_commit(&s.u_full);
                mma_commit(&s.k_free[st]);
                if (kStates) mma_commit(&s.v_free[c % kRing]);
            }
            drain(&s.drained[1], abort_flag, a.status);
        }
    } else if (warp == kWarpIssue + 2) {
        // ---- Q S^T of a chunk, then Q K^T of the next in the place of P of the one before: Q has one stage
        if (!kStates && elect_one()) {
            const uint32_t base = smem_u32(sm);
            const uint64_t q = sdesc_sw128(base + kOffQ, 16, 1024);
#pragma unroll 1
            for (int c = -1; c < chunks; ++c) {
                const int st = c & 1, to = st ^ 1;
                if (c >= 0) {
                    wait(&s.s_ready, c);
                    if (c > 1) wait(&s.o_free[st], (c - 2) >> 1);
                    tc_fence_after();
                    const uint64_t S = sdesc_sw128(base + kOffS, kTile, 1024);
#pragma unroll 1
                    for (int part = 0; part < kHalves; ++part)
#pragma unroll
                        for (int i = 0; i < KS; ++i)
                            mma_f16kind(tbase + kColI + 64 * st, q + k_step(i), S + part * (kTile >> 4) + mn_step(i),
                                        idesc_bf16_f32(128, 64, 0, 1), part + i > 0);
                    mma_commit(&s.q_free);
                    mma_commit(&s.i_full[st]);
                }
                if (c + 1 < chunks) {
                    wait(&s.k_full[to], (c + 1) >> 1);
                    wait(&s.q_full, c + 1);
                    if (c > 0) wait(&s.p_free[to], (c - 1) >> 1);
                    tc_fence_after();
                    const uint64_t k = sdesc_sw128(base + kOffK + to * 2 * kTile, 16, 1024);
#pragma unroll
                    for (int i = 0; i < KS; ++i)
                        mma_f16kind(tbase + kColP + 128 * to, q + k_step(i), k + k_step(i), idesc_bf16_f32(128, 128, 0, 0), i > 0);
                    mma_commit(&s.qk_full[to]);
                    mma_commit(&s.k_free[to]);
                }
            }
            drain(&s.drained[2], abort_flag, a.status);
        }
    } else if (elect_one()) {
        // ---- tensor copies: K, Q, V, and the outputs that take the place of V, whichever can go on.  Chunks
        // ahead of the rings are fetched to L2.
        int k = min(2, chunks), q = kStates ? chunks : min(1, chunks);  // chunks loaded
        int v = min(kRing, chunks), put = 0;  // and chunks whose V is through and whose outputs are stored
        uint64_t idle = 0;    // since when there is nothing to do
        while ((k < chunks || q < chunks || put < chunks) && !*abort_flag) {
            bool moved = false;
            if (q < chunks && mbar_test_wait(&s.q_free, (q - 1) & 1)) {
                load_q(q, false);
                if (q + kAhead < chunks) load_q(q + kAhead, true);
                ++q;
                moved = true;
            }
            if (k < chunks && mbar_test_wait(&s.k_free[k & 1], (k - 2) >> 1 & 1)) {
                load_k(k, false);
                if (k + kAhead < chunks) load_k(k + kAhead, true);
                ++k;
                moved = true;
            }
            if (put < chunks && mbar_test_wait(kStates ? &s.v_free[put % kRing] : &s.o_staged[put % kRing], put / kRing & 1)) {
                if (!kStates && u.len - put * kC >= kC) {
                    tma_store_3d(&tm_o, sm + kOffV + put % kRing * kTile, v0, h, row(put));
                    bulk_commit();
                    bulk_wait_read();
                }
                if (v < chunks) load_v(v++);
                ++put;
                moved = true;
            }
            if (moved) {
                idle = 0;
            } else {
                const uint64_t now = globaltimer_ns();
                if (!idle) idle = now;
                if (now - idle > kWaitLimitNs) {
                    *abort_flag = 1;
                    atomicOr(a.status, GDN_DEV_WAIT_TIMEOUT);
                }
            }
        }
        // no copy is on its way when the block ends, also where the waits for it gave up
#pragma unroll 1
        for (int c = max(0, k - 2); c < k; ++c) wait(&s.k_full[c & 1], c >> 1);
        if (!kStates && q > 0) wait(&s.q_full, q - 1);
#pragma unroll 1
        for (int c = max(0, v - kRing); c < v; ++c) wait(&s.v_full[c % kRing], c / kRing);
        bulk_wait_all();
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

// [rows][heads][width] bf16 with a row stride, in boxes of `high` rows x 1 head x 64.
bool make_map(CUtensorMap *m, const void *base, int64_t rows, int heads, int width, int64_t ld, int high)
{
    const cuuint64_t dim[3] = {(cuuint64_t)width, (cuuint64_t)heads, (cuuint64_t)rows};
    const cuuint64_t stride[2] = {(cuuint64_t)width * 2, (cuuint64_t)ld * 2};
    const cuuint32_t box[3] = {64, 1, (cuuint32_t)high}, es[3] = {1, 1, 1};
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
           a.ld_q < ((int64_t)1 << 38) && a.ld_k < ((int64_t)1 << 38) && a.ld_v < ((int64_t)1 << 38) && a.ld_o < ((int64_t)1 << 38) && rows > 0 &&
           rows < ((int64_t)1 << 31) - 2 * kC && aligned16(a.q) && aligned16(a.k) && aligned16(a.v) && aligned16(a.o) &&
           encoder();
}

cudaError_t gdn_linattn_tc(const GdnLinattnArgs &a, bool states_only, cudaStream_t s)
{
    const int64_t rows = a.cu_seqlens ? a.T : (int64_t)a.N * a.T;
    const int tiles = (a.dv + kDVT - 1) / kDVT;
    const int64_t blocks = (a.segment ? a.pieces : a.N) * a.heads * tiles;
    if (blocks > 0x7fffffff) return cudaErrorInvalidConfiguration;
    CUtensorMap q, k, v, o;
    if (!make_map(&q, a.q, rows, a.groups, a.dk, a.ld_q, kC / 4) || !make_map(&k, a.k, rows, a.groups, a.dk, a.ld_k, kC) ||
        !make_map(&v, a.v, rows, a.heads, a.dv, a.ld_v, kC) || !make_map(&o, a.o, rows, a.heads, a.dv, a.ld_o, kC))
        return cudaErrorInvalidValue;
    auto *kernel = states_only  ? gdn_linattn_tc_kernel<true, 8>
                   : a.dk <= 64 ? gdn_linattn_tc_kernel<false, 4>
                   : a.dk <= 96 ? gdn_linattn_tc_kernel<false, 6>
                                : gdn_linattn_tc_kernel<false, 8>;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
    if (e != cudaSuccess) return e;
    kernel<<<(unsigned)blocks, kThreads, kSmemBytes, s>>>(a, tiles, q, k, v, o);
    return cudaGetLastError();
}

// Device helpers shared by the operators around the recurrence: element types,
// vector accesses, activations, and which sequence a block works on.
#pragma once

#include <cuda_bf16.h>
#include <float.h>
#include <stdint.h>

#include "gdn.h"

namespace gdn_layer {

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
template <typename E> __device__ __forceinline__ E from_f(float x);
template <> __device__ __forceinline__ float from_f<float>(float x) { return x; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float x)
{
    return __float2bfloat16_rn(x);
}

// N consecutive elements as one word, and its fp32 values.  N sizeof(E) is 2 to
// 16 bytes, aligned to its size.
template <int BYTES> struct Word;
template <> struct Word<2> { typedef unsigned short type; };
template <> struct Word<4> { typedef uint32_t type; };
template <> struct Word<8> { typedef uint2 type; };
template <> struct Word<16> { typedef uint4 type; };

__device__ __forceinline__ void widen(unsigned short u, float (&x)[1])
{
    x[0] = __uint_as_float((uint32_t)u << 16);
}
__device__ __forceinline__ void widen_pair(uint32_t u, float &lo, float &hi)
{
    lo = __uint_as_float(u << 16);
    hi = __uint_as_float(u & 0xffff0000u);
}
__device__ __forceinline__ void widen(uint32_t u, float (&x)[2]) { widen_pair(u, x[0], x[1]); }
__device__ __forceinline__ void widen(uint2 u, float (&x)[4])
{
    widen_pair(u.x, x[0], x[1]);
    widen_pair(u.y, x[2], x[3]);
}
__device__ __forceinline__ void widen(uint4 u, float (&x)[8])
{
    widen_pair(u.x, x[0], x[1]);
    widen_pair(u.y, x[2], x[3]);
    widen_pair(u.z, x[4], x[5]);
    widen_pair(u.w, x[6], x[7]);
}
__device__ __forceinline__ void widen(uint32_t u, float (&x)[1]) { x[0] = __uint_as_float(u); }
__device__ __forceinline__ void widen(uint2 u, float (&x)[2])
{
    x[0] = __uint_as_float(u.x);
    x[1] = __uint_as_float(u.y);
}
__device__ __forceinline__ void widen(uint4 u, float (&x)[4])
{
    x[0] = __uint_as_float(u.x);
    x[1] = __uint_as_float(u.y);
    x[2] = __uint_as_float(u.z);
    x[3] = __uint_as_float(u.w);
}

__device__ __forceinline__ uint32_t narrow_pair(float lo, float hi)
{
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
}
__device__ __forceinline__ void narrow(unsigned short &u, const float (&x)[1])
{
    u = (unsigned short)narrow_pair(x[0], 0.f);
}
__device__ __forceinline__ void narrow(uint32_t &u, const float (&x)[2]) { u = narrow_pair(x[0], x[1]); }
__device__ __forceinline__ void narrow(uint2 &u, const float (&x)[4])
{
    u = make_uint2(narrow_pair(x[0], x[1]), narrow_pair(x[2], x[3]));
}
__device__ __forceinline__ void narrow(uint4 &u, const float (&x)[8])
{
    u = make_uint4(narrow_pair(x[0], x[1]), narrow_pair(x[2], x[3]), narrow_pair(x[4], x[5]),
                   narrow_pair(x[6], x[7]));
}
__device__ __forceinline__ void narrow(uint32_t &u, const float (&x)[1]) { u = __float_as_uint(x[0]); }
__device__ __forceinline__ void narrow(uint2 &u, const float (&x)[2])
{
    u = make_uint2(__float_as_uint(x[0]), __float_as_uint(x[1]));
}
__device__ __forceinline__ void narrow(uint4 &u, const float (&x)[4])
{
    u = make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]),
                   __float_as_uint(x[3]));
}

// N elements from memory as fp32 and back, in words of at most 16 bytes.
template <typename E, int N> __device__ __forceinline__ void ld_vec(const E *p, float (&x)[N])
{
    if constexpr (N * sizeof(E) > 16) {
        constexpr int H = N / 2;
        float a[H], b[H];
        ld_vec<E, H>(p, a);
        ld_vec<E, H>(p + H, b);
#pragma unroll
        for (int i = 0; i < H; ++i) {
            x[i] = a[i];
            x[H + i] = b[i];
        }
    } else {
        widen(*reinterpret_cast<const typename Word<N * sizeof(E)>::type *>(p), x);
    }
}

template <typename E, int N> __device__ __forceinline__ void st_vec(E *p, const float (&x)[N])
{
    if constexpr (N * sizeof(E) > 16) {
        constexpr int H = N / 2;
        float a[H], b[H];
#pragma unroll
        for (int i = 0; i < H; ++i) {
            a[i] = x[i];
            b[i] = x[H + i];
        }
        st_vec<E, H>(p, a);
        st_vec<E, H>(p + H, b);
    } else {
        typename Word<N * sizeof(E)>::type u;
        narrow(u, x);
        *reinterpret_cast<typename Word<N * sizeof(E)>::type *>(p) = u;
    }
}

// 2^v and 1 / v to 2 and 1 ulp, flushing subnormals like the rest of the
// library's fp32 arithmetic.
__device__ __forceinline__ float ex2(float v)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(v));
    return y;
}

__device__ __forceinline__ float rcp(float v)
{
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(v));
    return y;
}

// Two fp32 operations in one instruction.
typedef unsigned long long f32x2;

__device__ __forceinline__ f32x2 pack2(float lo, float hi)
{
    f32x2 v;
    asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(lo), "f"(hi));
    return v;
}

__device__ __forceinline__ void unpack2(f32x2 v, float &lo, float &hi)
{
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}

__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c)
{
    f32x2 d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}

__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b)
{
    f32x2 d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b)
{
    f32x2 d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

__device__ __forceinline__ f32x2 dup2(float v) { return pack2(v, v); }

__device__ __forceinline__ f32x2 ex2x2(f32x2 v)
{
    float a, b;
    unpack2(v, a, b);
    return pack2(ex2(a), ex2(b));
}

__device__ __forceinline__ f32x2 rcp2(f32x2 v)
{
    float a, b;
    unpack2(v, a, b);
    return pack2(rcp(a), rcp(b));
}

constexpr float kLog2e = 1.4426950408889634f;

// Added to the exponent of a state's decay 2^v, v <= 0.  ex2.approx comes out
// low on average, by 5e-9 to 9e-9 of its value for v above -2^-8 and by 1.8e-8 to
// 2.7e-8 down to -1/4 (measured, 2^20 values per binade), and a chain of tokens
// adds that up: states that keep 1000 tokens would end 1e-5 low.  With this the
// mean is within 3e-9 above -2^-8 and never further off than without; 2^0 is
// still 1.
constexpr float kDecayShift = 1.15e-8f;

// A log2 e, the factor of d in a decay's exponent.  Infinities become the largest
// number, so that d = 0 (in the scan also the rows past a sequence's end) decays
// nothing and does not make NaN; any d above 5e-37 still decays everything.
__device__ __forceinline__ float decay_rate(float A)
{
    float v;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(v) : "f"(A * kLog2e), "f"(-FLT_MAX));  // NaN stays
    asm("min.NaN.f32 %0, %0, %1;" : "+f"(v) : "f"(FLT_MAX));
    return v;
}

// v / (1 + e^-v).
__device__ __forceinline__ float silu(float v) { return v * rcp(1.f + ex2(-kLog2e * v)); }

__device__ __forceinline__ f32x2 silu2(f32x2 v)
{
    return mul2(v, rcp2(add2(dup2(1.f), ex2x2(mul2(v, dup2(-kLog2e))))));
}

// log(1 + e^v) = max(v, 0) + log1p(w) with w = e^-|v| in (0, 1], and
// log1p(w) = 2 artanh(r), r = w / (2 + w) <= 1/3.  2 artanh(r) / r as a
// polynomial in r^2, interpolated at the Chebyshev nodes of [0, 1/9] (relative
// error below 2^-26).  Small w keeps its relative precision, which
// log(1 + w) would round away (a step size of 1e-3 would be off by 6e-5).
__device__ __forceinline__ f32x2 softplus2(f32x2 v)
{
    float a, b;
    unpack2(v, a, b);
    const f32x2 w = pack2(ex2(-kLog2e * fabsf(a)), ex2(-kLog2e * fabsf(b)));
    const f32x2 r = mul2(w, rcp2(add2(dup2(2.f), w))), q = mul2(r, r);
    f32x2 p = fma2(dup2(0.281746566f), q, dup2(0.27961418f));
    p = fma2(p, q, dup2(0.400248528f));
    p = fma2(p, q, dup2(0.66666317f));
    p = fma2(p, q, dup2(2.f));
    return fma2(r, p, pack2(fmaxf(a, 0.f), fmaxf(b, 0.f)));
}

__device__ __forceinline__ float softplus(float v)
{
    float a, b;
    unpack2(softplus2(dup2(v)), a, b);
    return a;
}

// A sequence's tile of tokens, found from the block's tile slot.
struct Span {
    int n;        // sequence
    int tile;     // tile of `tl` tokens within it
    int len;      // its tokens
    int64_t row;  // its first row
};

// Tile slots.  Without cu_seqlens sequence n has slots [n tiles, (n + 1)
// tiles).  Packed, the lengths are on the device and the host can only bound
// the slots: sequence n spanning [lo, hi) starts at slot lo / tl + n and has
// max(1, ceil((hi - lo) / tl)) of them.  floor(hi / tl) + n + 1 is at least
// that start plus that count, so no two sequences share a slot and
// T / tl + N slots are enough.  The warp looks at 32 sequences at a time, so a
// malformed span hides none of the others.  Called by whole warps; false when
// the slot has no tile.
__device__ __forceinline__ bool find_span(const int32_t *cu, int N, int T, int tl, int64_t slot,
                                          int tiles, unsigned int *status, Span &s)
{
    if (!cu) {
        s.n = (int)(slot / tiles);
        s.tile = (int)(slot % tiles);
        s.len = T;
        s.row = (int64_t)s.n * T;
        return true;
    }
    bool found = false;
    for (int base = 0; base < N && (!found || slot == 0); base += 32) {
        const int n = base + (threadIdx.x & 31);
        int lo = 0, hi = 0, first = 0;
        bool hit = false;
        if (n < N) {
            lo = cu[n];
            hi = cu[n + 1];
            if (lo < 0 || hi < lo || hi > T) {
                if (slot == 0) atomicOr(status, GDN_DEV_BAD_SEQLENS);
            } else {
                first = lo / tl + n;
                const int count = hi > lo ? (hi - lo - 1) / tl + 1 : 1;
                hit = slot >= first && slot < (int64_t)first + count;
            }
        }
        const unsigned m = __ballot_sync(0xffffffffu, hit);
        if (m && !found) {
            const int src = __ffs(m) - 1;
            s.n = base + src;
            s.tile = (int)slot - __shfl_sync(0xffffffffu, first, src);
            s.row = __shfl_sync(0xffffffffu, lo, src);
            s.len = __shfl_sync(0xffffffffu, hi, src) - (int)s.row;
            found = true;
        }
    }
    return found;
}

// The packed sequence of a given rank by length, longest first, of at most 64
// (of more, the sequence of that number): blocks start about in the order of
// their numbers, and a sequence that takes as long as the rest together must
// not be the last to start.  Called by whole warps; false for a malformed span.
__device__ __forceinline__ bool find_ranked(const int32_t *cu, int N, int T, int rank,
                                            unsigned int *status, Span &s)
{
    const int lane = threadIdx.x & 31;
    int n = rank;
    if (N <= 64) {
        int len[2], ahead[2] = {0, 0};
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int m = lane + 32 * i;
            len[i] = m < N ? cu[m + 1] - cu[m] : INT32_MIN;
        }
        for (int m = 0; m < N; ++m) {
            const int other = __shfl_sync(0xffffffffu, m < 32 ? len[0] : len[1], m & 31);
#pragma unroll
            for (int i = 0; i < 2; ++i) ahead[i] += other > len[i] || (other == len[i] && m < lane + 32 * i);
        }
        const unsigned lo = __ballot_sync(0xffffffffu, lane < N && ahead[0] == rank);
        const unsigned hi = __ballot_sync(0xffffffffu, lane + 32 < N && ahead[1] == rank);
        n = lo ? __ffs(lo) - 1 : 31 + __ffs(hi);
    }
    const int first = cu[n], end = cu[n + 1];
    if (first < 0 || end < first || end > T) {
        atomicOr(status, GDN_DEV_BAD_SEQLENS);
        return false;
    }
    s.n = n;
    s.tile = 0;
    s.len = end - first;
    s.row = first;
    return true;
}

// The pool entry of sequence n's state, or -1 when it keeps none.
__device__ __forceinline__ int state_entry(const int32_t *slots, int n, int pool,
                                           unsigned int *status)
{
    if (!slots) return n;
    const int e = slots[n];
    if (e >= pool) {
        atomicOr(status, GDN_DEV_BAD_SLOT);
        return -1;
    }
    return e < 0 ? -1 : e;
}

// Asynchronous copies to shared memory.
__device__ __forceinline__ uint32_t smem_addr(const void *p)
{
    return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}

template <int BYTES> __device__ __forceinline__ void copy_async(void *dst, const void *src)
{
    if (BYTES == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_addr(dst)), "l"(src) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(smem_addr(dst)), "l"(src), "n"(BYTES)
                     : "memory");
}

__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }

// Wait until at most PENDING of this thread's copy groups are in flight.
template <int PENDING> __device__ __forceinline__ void copy_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(PENDING) : "memory");
}

__device__ __forceinline__ void prefetch(const void *p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

// One arrival at `bar` once this thread's copies so far have landed.
__device__ __forceinline__ void copy_arrive(uint64_t *bar)
{
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_addr(bar)) : "memory");
}

// A tensor copy of the box at column x (on a 16-byte boundary), row y of a
// matrix, completing on `bar`.
__device__ __forceinline__ void copy_box(void *dst, const void *map, int x, int y, uint64_t *bar)
{
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4}], [%2];" ::"r"(smem_addr(dst)),
        "l"(map), "r"(smem_addr(bar)), "r"(x), "r"(y)
        : "memory");
}

// Barrier `id` between parts of a block: arrivals that do not wait, and waits.
__device__ __forceinline__ void part_arrive(int id, int threads)
{
    asm volatile("bar.arrive %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

__device__ __forceinline__ void part_sync(int id, int threads)
{
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// Grids of x by any number of blocks: the second dimension holds 65 535 and goes on in the third.
inline dim3 grid_of(unsigned x, int64_t blocks)
{
    const unsigned z = (unsigned)((blocks + 65534) / 65535);
    return dim3(x, (unsigned)((blocks + z - 1) / z), z);
}
__device__ __forceinline__ unsigned block_of() { return blockIdx.z * gridDim.y + blockIdx.y; }

inline bool aligned_to(const void *p, size_t al) { return reinterpret_cast<uintptr_t>(p) % al == 0; }
inline bool aligned16(const void *p) { return aligned_to(p, 16); }

}  // namespace gdn_layer

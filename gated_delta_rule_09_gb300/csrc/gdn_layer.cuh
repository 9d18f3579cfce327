// Device helpers shared by the operators around the recurrence: element types,
// vector accesses, activations, and which sequence a block works on.
#pragma once

#include <cuda_bf16.h>
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

// VEC consecutive elements as floats: one 16-byte access for the widths the
// vectorised kernels use (8 bf16 or 4 fp32), element by element otherwise.
template <typename E, int VEC> struct alignas(VEC * sizeof(E)) Pack {
    E v[VEC];
};

template <typename E, int VEC>
__device__ __forceinline__ void ld_vec(const E *p, float (&x)[VEC])
{
    const Pack<E, VEC> u = *reinterpret_cast<const Pack<E, VEC> *>(p);
#pragma unroll
    for (int i = 0; i < VEC; ++i) x[i] = to_f(u.v[i]);
}

template <typename E, int VEC>
__device__ __forceinline__ void st_vec(E *p, const float (&x)[VEC])
{
    Pack<E, VEC> u;
#pragma unroll
    for (int i = 0; i < VEC; ++i) u.v[i] = from_f<E>(x[i]);
    *reinterpret_cast<Pack<E, VEC> *>(p) = u;
}

__device__ __forceinline__ float silu(float v) { return __fdividef(v, 1.f + __expf(-v)); }

// log(1 + e^v) = max(v, 0) + log1p(w) with w = e^-|v| in (0, 1].  log1p by the
// series of 2 artanh(r), r = w / (2 + w) <= 1/3: nine odd terms leave less than
// 2^-31 of the value, and small w keeps its relative precision, which
// log(1 + w) would round away (a step size of 1e-3 would be off by 6e-5).
__device__ __forceinline__ float softplus(float v)
{
    const float w = __expf(-fabsf(v));
    const float r = __fdividef(w, 2.f + w), q = r * r;
    float p = 1.f / 17.f;
    p = fmaf(p, q, 1.f / 15.f);
    p = fmaf(p, q, 1.f / 13.f);
    p = fmaf(p, q, 1.f / 11.f);
    p = fmaf(p, q, 1.f / 9.f);
    p = fmaf(p, q, 1.f / 7.f);
    p = fmaf(p, q, 1.f / 5.f);
    p = fmaf(p, q, 1.f / 3.f);
    p = fmaf(p, q, 1.f);
    return fmaxf(v, 0.f) + 2.f * r * p;
}

// 2^v, flushing to zero like the rest of the library's fp32 arithmetic.
__device__ __forceinline__ float ex2(float v)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(v));
    return y;
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
                const int count = hi > lo ? (hi - lo + tl - 1) / tl : 1;
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

inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

}  // namespace gdn_layer

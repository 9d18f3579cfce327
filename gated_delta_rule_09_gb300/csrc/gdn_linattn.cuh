// Device helpers shared by the linear attention kernels: decays of a block of 32
// tokens, and which unit of work a block takes.
#pragma once

#include "gdn_layer.cuh"
#include "gdn_layer.h"

namespace gdn_linattn {

using namespace gdn_layer;

// A decay below 2^-126 is zero in fp32: such a token forgets what was before it.
constexpr float kForget = -126.f;

// Decays of 32 consecutive tokens, one per lane, as base-2 logarithms.  Factors
// between two tokens are products over the tokens between; every one used here is
// a sum of terms that are added up, never a difference of two long sums, but for
// pairs within the block (`in` of one minus `in` of the other), which have `rest` beside
// them.  Tokens that forget count as zero in the sums and stand in `mask`, so that an
// infinite decay makes no NaN.
struct Decays {
    float in;       // sum over the block's tokens up to and with the lane's
    float after;    // sum over the block's tokens behind the lane's
    float total;    // of the block
    unsigned mask;  // lanes that forget

    __device__ __forceinline__ void scan(float log_decay)
    {
        const int lane = threadIdx.x & 31;
        const float g = log_decay * kLog2e;
        const bool forget = g <= kForget;
        mask = __ballot_sync(0xffffffffu, forget);
        in = forget ? 0.f : g;
        float back = in;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const float x = __shfl_up_sync(0xffffffffu, in, o), y = __shfl_down_sync(0xffffffffu, back, o);
            if (lane >= o) in += x;
            if (lane + o < 32) back += y;
        }
        total = __shfl_sync(0xffffffffu, in, 31);
        after = __shfl_down_sync(0xffffffffu, back, 1);
        if (lane == 31) after = 0.f;
    }

    // `in` anew with what its rounding leaves out, for differences between tokens behind a
    // steep one: they depend on what lies between, not on how far the block has come (eight
    // tokens of e^-60, then flat: 7e-5 off without).  Sums in fixed point, steps of 2^-40, are
    // exact, where fp64 has a sixtieth of the rate.  Lanes behind a decay that does not fit, 2^17
    // and more or NaN, keep what they have.
    __device__ __forceinline__ float exact(float log_decay)
    {
        const int lane = threadIdx.x & 31;
        const float g = log_decay * kLog2e;
        const bool fits = fabsf(g) < 131072.f;
        long long x = fits && g > kForget ? __float2ll_rn(g * 1099511627776.f) : 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x += y;
        }
        const unsigned out = __ballot_sync(0xffffffffu, !fits && !(g <= kForget));
        if (out & (0xffffffffu >> (31 - lane))) return 0.f;
        const float high = __ll2float_rn(x);
        in = high * 9.094947017729282e-13f;
        return __ll2float_rn(x - __float2ll_rn(high)) * 9.094947017729282e-13f;
    }

    // Whether some token up to and with lane i, or behind it, forgets.
    __device__ __forceinline__ bool cut_upto(int i) const { return mask & (0xffffffffu >> (31 - i)); }
    __device__ __forceinline__ bool cut_behind(int i) const { return mask & (0xfffffffeu << i); }
};

// The first token of the block that token i still sees.
__device__ __forceinline__ int first_seen(unsigned mask, int i)
{
    const unsigned m = mask & (0xffffffffu >> (31 - i));
    return m ? 31 - __clz(m) : 0;
}

// 2^x of a sum of decays; kDecayShift as in the scan's decays.
__device__ __forceinline__ float decay_of(float x) { return ex2(x + kDecayShift); }

// The same to half a step of fp32 and a little more, for the factors that follow one
// another in a state: what ex2.approx is off, 2 steps at most, adds up over the chunks
// (131 072 tokens in chunks of 32, heads that keep 8192: 2.0e-6 off with it).  2^f of the
// fraction f, |f| <= 1/2, by the series of e^(f ln 2), whose ninth term is below 2^-32.
__device__ __forceinline__ float chained_decay_of(float x)
{
    const float n = rintf(fmaxf(x, -127.f)), f = fmaxf(x, -127.f) - n;
    float p = 1.321548679e-06f;
    p = fmaf(p, f, 1.525273380e-05f);
    p = fmaf(p, f, 1.540353039e-04f);
    p = fmaf(p, f, 1.333355815e-03f);
    p = fmaf(p, f, 9.618129108e-03f);
    p = fmaf(p, f, 5.550410866e-02f);
    p = fmaf(p, f, 2.402265070e-01f);
    p = fmaf(p, f, 6.931471806e-01f);
    p = fmaf(p, f, 1.f);
    return x < -126.f ? 0.f : x != x ? x : x > 127.f ? ex2(x) : p * __int_as_float(((int)n + 127) << 23);
}

// 2^(x / 2), twice of which takes a state over a sum of decays x whose own 2^x is zero or
// infinite, though what it multiplies to need not be.  Kept from zero and, for a finite x,
// from infinity: an infinite state stays infinite and a zero one zero, as token by token.
__device__ __forceinline__ float half_decay_of(float x)
{
    const float h = 0.5f * x;
    return chained_decay_of(h < -126.f ? -126.f : h > 127.f && h < 3e38f ? 127.f : h);
}

// Sums of decays below -126, whose 2^x is zero in fp32 and would drop an infinite state that
// no token forgets, are applied as two factors 2^once(x); where a scale goes with them, sums
// below -60, so that either factor has room for it.
__device__ __forceinline__ bool is_far(float x, float from = -126.f) { return x < from; }
__device__ __forceinline__ float once(float x, float from = -126.f) { return is_far(x, from) ? fmaxf(0.5f * x, -100.f) : x; }

// The root of the decay over a piece, from its chunks' sums as they come; zero where a token forgets.
struct PieceDecay {
    double sum = 0.;
    bool cut = false;
    __device__ __forceinline__ void add(float total, unsigned mask)
    {
        sum += total;
        cut |= mask != 0;
    }
    __device__ __forceinline__ float all() const { return cut ? 0.f : half_decay_of((float)sum); }
};

// What a block works on: a whole sequence or a piece of one, and the states it
// reads and writes.
struct Unit {
    int64_t row;       // first row
    int len;           // tokens
    const float *in;   // state before them, or null (zeros): [dv, dk] of the head
    float *out;        // state after them, or null
};

// The unit of a span number (a sequence's rank, or a piece slot).  Called by whole
// warps with the same arguments; false: nothing to do.
__device__ __forceinline__ bool find_unit(const GdnLinattnArgs &a, int64_t span, int h, bool states_only, Unit &u)
{
    Span s;
    const int64_t per = (int64_t)a.dv * a.dk;
    if (a.segment) {
        const int tiles = (int)(((int64_t)a.T + a.segment - 1) / a.segment);
        if (!find_span(a.cu_seqlens, a.N, a.T, a.segment, span, tiles, a.status, s)) return false;
        const int64_t from = (int64_t)s.tile * a.segment;
        const bool last = s.len - from <= a.segment;
        if (states_only && last) return false;  // nobody starts from what it adds
        u.row = s.row + from;
        u.len = (int)min((int64_t)a.segment, s.len - from);
        float *mine = a.piece_state + (span * a.heads + h) * per;
        u.in = states_only ? nullptr : mine;
        u.out = states_only ? mine : nullptr;
        if (!states_only && last && a.state_out) {
            const int e = state_entry(a.slots, s.n, a.pool, a.status);
            if (e >= 0) u.out = a.state_out + ((int64_t)e * a.heads + h) * per;
        }
        return true;
    }
    if (a.cu_seqlens) {
        if (!find_ranked(a.cu_seqlens, a.N, a.T, (int)span, a.status, s)) return false;
    } else {
        s.n = (int)span;
        s.len = a.T;
        s.row = span * a.T;
    }
    u.row = s.row;
    u.len = s.len;
    const int e = a.state_in || a.state_out ? state_entry(a.slots, s.n, a.pool, a.status) : -1;
    const int64_t at = ((int64_t)e * a.heads + h) * per;
    u.in = a.state_in && e >= 0 ? a.state_in + at : nullptr;
    u.out = a.state_out && e >= 0 ? a.state_out + at : nullptr;
    return true;
}

}  // namespace gdn_linattn

// Selective state space scan: how prompts are cut, and the step for single
// tokens.  Per channel c with d_state fp32 states
//
//     h[s] = exp(d A[c, s]) h[s] + d B[s] x        y = (sum_s C[s] h[s] + D x) silu(z)
//
// A step reads and writes every state once, 8 bytes of fp32 for five operations:
// bound by HBM for large batches, by latency for small ones.  A lane holds four
// consecutive states of a channel (one 16-byte access each way), the LPC = 1..32
// lanes of a channel (d_state padded to 4 LPC) are neighbours, and their parts
// of y meet in a butterfly.  A has the size of a sequence's states, so a thread
// keeps its four of A for kRows sequences; their loads are in flight together.
// 256 sequences x 4096 channels x 16 states, bf16: 31 us, 4.6 TB/s (1024
// sequences 5.2); with one sequence per thread, and softplus, gate and store in
// every lane of a channel, 46.
#include "gdn_layer.h"
#include "gdn_layer.cuh"

namespace {

using namespace gdn_layer;

constexpr int kThreads = 128;

template <bool VEC> __device__ __forceinline__ void ld_state(const float *p, int s0, int ds, float (&h)[4])
{
    if (VEC) {
        if (s0 < ds) {
            ld_vec<float, 4>(p + s0, h);
            return;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) h[j] = 0.f;
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) h[j] = s0 + j < ds ? p[s0 + j] : 0.f;
    }
}

// Four of B or C, as loaded until they are used; zeros past the end.
template <bool VEC, typename E> struct Four {
    typename Word<4 * sizeof(E)>::type v;
    __device__ __forceinline__ void load(const E *p, int s0, int ds)
    {
        v = typename Word<4 * sizeof(E)>::type();
        if (s0 < ds) v = *reinterpret_cast<const typename Word<4 * sizeof(E)>::type *>(p + s0);
    }
    __device__ __forceinline__ void get(float (&f)[4]) const { widen(v, f); }
};
template <typename E> struct Four<false, E> {
    float v[4];
    __device__ __forceinline__ void load(const E *p, int s0, int ds)
    {
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = s0 + j < ds ? to_f(p[s0 + j]) : 0.f;
    }
    __device__ __forceinline__ void get(float (&f)[4]) const
    {
#pragma unroll
        for (int j = 0; j < 4; ++j) f[j] = v[j];
    }
};

// kRows <= LPC sequences per thread.  What is needed once per channel (softplus,
// gate, store) is done for sequence r by the channel's lanes q with q % kRows = r
// and passed round; the butterfly leaves that lane with that sequence's y.
template <typename E, int LPC, int kRows, bool VEC>
__global__ void __launch_bounds__(kThreads, kRows > 1 ? 8 : 1) gdn_ssm_step_kernel(const GdnSsmArgs a)
{
    const int c = block_of() * (kThreads / LPC) + threadIdx.x / LPC;
    const bool live = c < a.channels;
    const int cc = live ? c : a.channels - 1;
    const int q = threadIdx.x % LPC, s0 = 4 * q, ds = a.d_state;
    const int g = cc / (a.channels / a.groups);
    const int n0 = blockIdx.x * kRows, own = n0 + q % kRows;
    // the lane's own sequence; rows past the end repeat the last and store nothing
    const int64_t row = min(own, a.N - 1);
    const int mine = own < a.N ? state_entry(a.slots, own, a.pool, a.status) : -1;
    int entry[kRows];
    float h[kRows][4];
    Four<VEC, E> B[kRows], C[kRows];
    const E *b = static_cast<const E *>(a.Bm) + (int64_t)n0 * a.ld_b + (int64_t)g * ds;
    const E *cm = static_cast<const E *>(a.Cm) + (int64_t)n0 * a.ld_c + (int64_t)g * ds;
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
        entry[r] = kRows == 1 ? mine : __shfl_sync(0xffffffffu, mine, (threadIdx.x & 31) / LPC * LPC + r);
#pragma unroll
        for (int j = 0; j < 4; ++j) h[r][j] = 0.f;
        if (a.state_in && entry[r] >= 0)
            ld_state<VEC>(a.state_in + ((size_t)entry[r] * a.channels + cc) * ds, s0, ds, h[r]);
    }
    float d = to_f(static_cast<const E *>(a.delta)[row * a.ld_delta + cc]);
    const float x = to_f(static_cast<const E *>(a.x)[row * a.ld_x + cc]);
    const float z = a.z ? to_f(static_cast<const E *>(a.z)[row * a.ld_z + cc]) : 0.f;
    float A[4];
    ld_state<VEC>(a.A + (size_t)cc * ds, s0, ds, A);
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
        B[r].load(b, s0, ds);
        C[r].load(cm, s0, ds);
        if (n0 + r + 1 < a.N) {
            b += a.ld_b;
            cm += a.ld_c;
        }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) A[j] = decay_rate(A[j]);
    d += a.delta_bias ? a.delta_bias[cc] : 0.f;
    if (a.softplus) d = softplus(d);
    const float dx = d * x;
    float y[kRows];
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
        const int from = (threadIdx.x & 31) / LPC * LPC + r;
        const float dr = kRows == 1 ? d : __shfl_sync(0xffffffffu, d, from);
        float dxr = kRows == 1 ? dx : __shfl_sync(0xffffffffu, dx, from);
        // places past the last state stay zero, or out of y: an infinite d x times zero is NaN
        if (VEC && s0 >= ds) dxr = 0.f;
        float bv[4], cv[4];
        B[r].get(bv);
        C[r].get(cv);
        y[r] = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            h[r][j] = fmaf(ex2(fmaf(dr, A[j], kDecayShift)), h[r][j], dxr * bv[j]);
            if (VEC || s0 + j < ds) y[r] = fmaf(cv[j], h[r][j], y[r]);
        }
        if (!live || entry[r] < 0) continue;
        float *out = a.state_out + ((size_t)entry[r] * a.channels + cc) * ds;
        if (VEC) {
            if (s0 < ds) st_vec<float, 4>(out + s0, h[r]);
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (s0 + j < ds) out[s0 + j] = h[r][j];
        }
    }
    // each halving step sends the sums that the partner's sequences need; then the rest of the lanes
#pragma unroll
    for (int o = kRows / 2; o >= 1; o /= 2)
#pragma unroll
        for (int r = 0; r < o; ++r) {
            const float send = q & o ? y[r] : y[r + o], keep = q & o ? y[r + o] : y[r];
            y[r] = keep + __shfl_xor_sync(0xffffffffu, send, o);
        }
#pragma unroll
    for (int o = kRows; o < LPC; o <<= 1) y[0] += __shfl_xor_sync(0xffffffffu, y[0], o);
    if (!live || q >= kRows || own >= a.N) return;
    float v = a.D ? fmaf(a.D[cc], x, y[0]) : y[0];
    if (a.z) v *= silu(z);
    static_cast<E *>(a.y)[row * a.ld_y + cc] = from_f<E>(v);
}

template <typename E, int LPC, int kRows> cudaError_t launch_step(const GdnSsmArgs &a, cudaStream_t s)
{
    const int per = kThreads / LPC;
    const dim3 grid = grid_of((a.N + kRows - 1) / kRows, (a.channels + per - 1) / per);
    const bool vec = a.d_state % 4 == 0 && aligned16(a.state_in) && aligned16(a.state_out) && aligned16(a.A) &&
                     a.ld_b % 4 == 0 && a.ld_c % 4 == 0 && aligned_to(a.Bm, 4 * sizeof(E)) &&
                     aligned_to(a.Cm, 4 * sizeof(E));
    if (vec)
        gdn_ssm_step_kernel<E, LPC, kRows, true><<<grid, kThreads, 0, s>>>(a);
    else
        gdn_ssm_step_kernel<E, LPC, kRows, false><<<grid, kThreads, 0, s>>>(a);
    return cudaGetLastError();
}

// Up to four sequences per thread once that still leaves a few blocks per SM; a
// small batch is spread as widely as it goes.  bf16, 4096 channels x 16 states,
// us with one against four: 8 sequences (256 blocks of four) 3.6 : 4.2, 16
// 5.3 : 4.9, 32 7.7 : 6.0, 256 43.3 : 31.0.
template <typename E, int LPC> cudaError_t by_rows(const GdnSsmArgs &a, cudaStream_t s)
{
    constexpr int kRows = LPC < 4 ? LPC : 4;
    const int per = kThreads / LPC;
    const int64_t blocks = (int64_t)((a.N + kRows - 1) / kRows) * ((a.channels + per - 1) / per);
    return blocks >= 512 ? launch_step<E, LPC, kRows>(a, s) : launch_step<E, LPC, 1>(a, s);
}

template <typename E> cudaError_t step(const GdnSsmArgs &a, cudaStream_t s)
{
    if (a.d_state <= 4) return by_rows<E, 1>(a, s);
    if (a.d_state <= 8) return by_rows<E, 2>(a, s);
    if (a.d_state <= 16) return by_rows<E, 4>(a, s);
    if (a.d_state <= 32) return by_rows<E, 8>(a, s);
    if (a.d_state <= 64) return by_rows<E, 16>(a, s);
    return by_rows<E, 32>(a, s);
}

}  // namespace

int gdn_ssm_sms()
{
    static int sms = 0;  // the same for every caller
    int dev = 0;
    if (!sms && (cudaGetDevice(&dev) != cudaSuccess ||
                 cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess))
        sms = 152;
    return sms;
}

// Whether sequences are cut, by the time either way.  A block (64 channels of a
// sequence) takes kAlone ns per token when it has its SM to itself, an SM gets
// through a token of a block every kShared ns when blocks share it, and cut
// sequences take kCut ns instead, the piece pass included, but not less than a
// piece alone in each of the two launches and kLaunch.  A grid of a few blocks
// per SM is long enough to even out.  One sequence of 131 072 tokens x 1024
// channels: 1.08 ms cut, 6.42 ms whole (16 blocks); four of 4096 tokens x 2048
// channels: 210 us whole, 264 to 313 cut into 512 to 2048 tokens; a pack of eight,
// 27 610 tokens with a longest of 7671, x 4096 channels: 498 us whole, 854 cut.
// More states take longer either way: one sequence of 16 384 tokens x 1024
// channels 0.33 cut : 1.18 ms whole with 32, 0.55 : 2.06 with 64, 1.03 : 3.59 with
// 128; fp32, 16 states 0.23 : 0.86.
// The constants are those of bf16, 16 states and tensor copies.
//
// Blocks end with their group, so groups make more of them; the workspace is
// sized for one group.  More blocks only make pieces longer or a call whole:
// each way's time grows with them, a cut call's at least as fast.
void gdn_ssm_plan(int N, int T, int channels, int groups, bool packed, int asked, int *segment,
                  int64_t *piece_slots)
{
    int64_t seg = ((int64_t)asked + 63) / 64 * 64;
    if (asked <= 0) {
        const int sms = gdn_ssm_sms();
        constexpr double kAlone = 51, kShared = 41, kCut = 79, kLaunch = 10000;
        const int64_t chunks = (int64_t)groups * ((channels / groups + kScanChannels - 1) / kScanChannels);
        const double tokens = (double)(packed ? T : (int64_t)N * T);
        // a packed sequence may be the longest by far; twice the mean is taken for it
        const double longest = packed && N > 1 ? 2. * T / N : T, work = tokens * chunks / sms;
        const double whole = longest * kAlone > work * kShared ? longest * kAlone : work * kShared;
        seg = ((int64_t)(work / 6.7) + 63) / 64 * 64;
        if (seg < 256) seg = 256;
        const double cut = work * kCut > 2 * seg * kAlone ? work * kCut : 2 * seg * kAlone;
        if (cut + kLaunch >= whole) seg = T;
    }
    *segment = 0;
    *piece_slots = 0;
    if (seg >= T) return;
    *segment = (int)seg;
    *piece_slots = packed ? T / seg + N : N * ((T + seg - 1) / seg);
}

cudaError_t gdn_launch_ssm_fwd(const GdnSsmArgs &a, cudaStream_t s, int *launches)
{
    *launches = a.segment ? 2 : 1;
    return a.dtype == 1 ? gdn_ssm_scan_bf16(a, s) : gdn_ssm_scan_f32(a, s);
}

cudaError_t gdn_launch_ssm_step(const GdnSsmArgs &a, cudaStream_t s)
{
    return a.dtype == 1 ? step<__nv_bfloat16>(a, s) : step<float>(a, s);
}

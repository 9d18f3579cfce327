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

template <typename E, int LPC, int kRows, bool VEC>
__global__ void __launch_bounds__(kThreads, kRows > 1 ? 8 : 1) gdn_ssm_step_kernel(const GdnSsmArgs a)
{
    const int per_block = kThreads / LPC;
    const int c = blockIdx.y * per_block + threadIdx.x / LPC;
    const bool live = c < a.channels;
    const int cc = live ? c : a.channels - 1;
    const int s0 = 4 * (threadIdx.x % LPC), ds = a.d_state;
    const int g = cc / (a.channels / a.groups);
    const int n0 = blockIdx.x * kRows;
    float h[kRows][4], d[kRows], x[kRows], z[kRows];
    Four<VEC, E> B[kRows], C[kRows];
    int entry[kRows];
#pragma unroll
    for (int r = 0; r < kRows; ++r) entry[r] = n0 + r < a.N ? state_entry(a.slots, n0 + r, a.pool, a.status) : -1;
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
        const int64_t n = min(n0 + r, a.N - 1);
#pragma unroll
        for (int j = 0; j < 4; ++j) h[r][j] = 0.f;
        if (a.state_in && entry[r] >= 0)
            ld_state<VEC>(a.state_in + ((size_t)entry[r] * a.channels + cc) * ds, s0, ds, h[r]);
        d[r] = to_f(static_cast<const E *>(a.delta)[n * a.ld_delta + cc]);
        x[r] = to_f(static_cast<const E *>(a.x)[n * a.ld_x + cc]);
        z[r] = a.z ? to_f(static_cast<const E *>(a.z)[n * a.ld_z + cc]) : 0.f;
        B[r].load(static_cast<const E *>(a.Bm) + n * a.ld_b + (size_t)g * ds, s0, ds);
        C[r].load(static_cast<const E *>(a.Cm) + n * a.ld_c + (size_t)g * ds, s0, ds);
    }
    float A[4];
    ld_state<VEC>(a.A + (size_t)cc * ds, s0, ds, A);
    const float bias = a.delta_bias ? a.delta_bias[cc] : 0.f, D = a.D ? a.D[cc] : 0.f;
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
        d[r] += bias;
        if (a.softplus) d[r] = softplus(d[r]);
        const float dx = d[r] * x[r];
        float y = 0.f, b[4], cm[4];
        B[r].get(b);
        C[r].get(cm);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            h[r][j] = fmaf(ex2(d[r] * (A[j] * kLog2e)), h[r][j], dx * b[j]);
            y = fmaf(cm[j], h[r][j], y);
        }
#pragma unroll
        for (int o = 1; o < LPC; o <<= 1) y += __shfl_xor_sync(0xffffffffu, y, o);
        if (!live || n0 + r >= a.N) continue;
        if (threadIdx.x % LPC == 0) {
            y = fmaf(D, x[r], y);
            if (a.z) y *= silu(z[r]);
            static_cast<E *>(a.y)[(int64_t)(n0 + r) * a.ld_y + cc] = from_f<E>(y);
        }
        if (entry[r] < 0) continue;
        float *out = a.state_out + ((size_t)entry[r] * a.channels + cc) * ds;
        if (VEC) {
            if (s0 < ds) st_vec<float, 4>(out + s0, h[r]);
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (s0 + j < ds) out[s0 + j] = h[r][j];
        }
    }
}

template <typename E, int LPC, int kRows> cudaError_t launch_step(const GdnSsmArgs &a, cudaStream_t s)
{
    const int per = kThreads / LPC;
    const dim3 grid((a.N + kRows - 1) / kRows, (a.channels + per - 1) / per);
    const bool vec = a.d_state % 4 == 0 && aligned16(a.state_in) && aligned16(a.state_out) && aligned16(a.A) &&
                     a.ld_b % 4 == 0 && a.ld_c % 4 == 0 && aligned_to(a.Bm, 4 * sizeof(E)) &&
                     aligned_to(a.Cm, 4 * sizeof(E));
    if (vec)
        gdn_ssm_step_kernel<E, LPC, kRows, true><<<grid, kThreads, 0, s>>>(a);
    else
        gdn_ssm_step_kernel<E, LPC, kRows, false><<<grid, kThreads, 0, s>>>(a);
    return cudaGetLastError();
}

// Four sequences per thread once that still leaves a few blocks per SM; a small
// batch is spread as widely as it goes.
template <typename E, int LPC> cudaError_t by_rows(const GdnSsmArgs &a, cudaStream_t s)
{
    const int per = kThreads / LPC;
    const int64_t blocks = (int64_t)((a.N + 3) / 4) * ((a.channels + per - 1) / per);
    return blocks >= 1024 ? launch_step<E, LPC, 4>(a, s) : launch_step<E, LPC, 1>(a, s);
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

// Whether sequences are cut, by the time either way.  A block (64 channels of a
// sequence) takes kAlone ns per token when it has its SM to itself, an SM gets
// through a token of a block every kShared ns when blocks share it, and cut
// sequences take kCut ns instead, the piece pass included, but not less than a
// piece alone in each of the two launches and kLaunch.  A grid of a few blocks
// per SM is long enough to even out.
void gdn_ssm_plan(int N, int T, int channels, int d_state, bool packed, int asked, int *segment,
                  int64_t *piece_slots)
{
    int64_t seg = ((int64_t)asked + 63) / 64 * 64;
    if (asked <= 0) {
        static int sms = 0;
        int dev = 0;
        if (!sms && (cudaGetDevice(&dev) != cudaSuccess ||
                     cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess))
            sms = 152;
        constexpr double kAlone = 58, kShared = 53, kCut = 85, kLaunch = 10000;
        const int64_t chunks = (channels + kScanChannels - 1) / (kScanChannels);
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

// Linear attention with a decay for each head: S <- e^g S + v k^T, o = scale S q,
// S in R^{d_v x d_k} per (sequence, head), g per head or per token and head, q and
// k shared by the heads of a group.
//
// Prompts go chunk by chunk.  With b_i the sum of g up to and with token i of a
// chunk of n tokens,
//
//     o_i = scale (e^{b_i} S q_i + sum_{j <= i} e^{b_i - b_j} (q_i k_j) v_j)
//     S  <- e^{b_n} S + sum_j e^{b_n - b_j} v_j k_j^T
//
// bf16 calls whose rows tensor copies can take run on the tensor cores
// (gdn_linattn_tc.cu); this file has the kernel for every other call, in fp32 on
// CUDA cores, the step for single tokens, and what joins the pieces of a long
// sequence: a first pass forms what each piece adds to the state, and its decay, a
// chain over a sequence's pieces turns these into the states they start from, and
// the second pass is the ordinary one over all pieces at once.
#include "gdn_linattn.cuh"

namespace {

using namespace gdn_linattn;

constexpr int kC = 32;        // tokens per chunk: one warp's worth of decays
constexpr int kThreads = 256;

// Tiles of a block: DK columns of q and k (d_k filled up with zeros), DV of v.  The
// state's rows follow those of k, and v lies along the tokens: every product reads both
// of its factors as words of four along the sum.  Rows are 4 words longer than a
// multiple of 32: eight rows' words of 16 bytes lie in different banks.
template <int DK, int DV> struct Smem {
    float q[kC][DK + 4], k[kC + DV][DK + 4];
    float v[DV][kC + 4], P[kC][kC + 4];
    float add[kC], in[kC], rest[kC], start[kC], early[kC];  // early: a second factor of start
    int first[kC];
    int kept;    // tokens before this one are forgotten by the end of the chunk
    float all, before;  // the decay over the chunk, in two factors; 0 when it forgets
};

__device__ __forceinline__ bool not_finite(float f) { return !(fabsf(f) <= 3.402823466e38f); }

__device__ __forceinline__ float at_least(float x, float least)  // NaN stays
{
    float y;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(x), "f"(least));
    return y;
}

// What a decay below 2^-126 leaves of x beside infinities: those stay, and what is finite
// still has its sign in their products.
__device__ __forceinline__ float least_of(float x)
{
    return not_finite(x) || x == 0.f ? x : copysignf(1.175494351e-38f, x);
}

// kC rows of W columns, on their way from memory: all of a thread's loads are in
// flight together.  A warp takes every eighth row.  Zeros past n rows and `cols` columns.
template <typename E, int W> struct Rows {
    static constexpr int kRowsOf = kC * 32 / kThreads, kStep = kThreads / 32, kCols = W / 32;
    E x[kRowsOf][kCols];
    __device__ __forceinline__ void load(const E *from, int64_t ld, int n, int cols)
    {
        const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
        const E *row = from + warp * ld + lane;
#pragma unroll
        for (int i = 0; i < kRowsOf; ++i, row += kStep * ld)
#pragma unroll
            for (int c = 0; c < kCols; ++c)
                x[i][c] = warp + kStep * i < n && lane + 32 * c < cols ? row[32 * c] : from_f<E>(0.f);
    }
    // To shared memory; whether something of it is infinite or NaN.
    template <int L> __device__ __forceinline__ bool store(float (*to)[L]) const
    {
        const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
        bool odd = false;
#pragma unroll
        for (int i = 0; i < kRowsOf; ++i)
#pragma unroll
            for (int c = 0; c < kCols; ++c) {
                const float f = to_f(x[i][c]);
                to[warp + kStep * i][lane + 32 * c] = f;
                odd |= not_finite(f);
            }
        return odd;
    }
    // The same transposed.
    template <int L> __device__ __forceinline__ bool turn(float (*to)[L]) const
    {
        const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
        bool odd = false;
#pragma unroll
        for (int i = 0; i < kRowsOf; ++i)
#pragma unroll
            for (int c = 0; c < kCols; ++c) {
                const float f = to_f(x[i][c]);
                to[lane + 32 * c][warp + kStep * i] = f;
                odd |= not_finite(f);
            }
        return odd;
    }
};

__device__ __forceinline__ void dot4(const float4 &x, const float4 &y, f32x2 &sum)
{
    sum = fma2(pack2(x.x, x.y), pack2(y.x, y.y), sum);
    sum = fma2(pack2(x.z, x.w), pack2(y.z, y.w), sum);
}

// A warp's lanes are 4 rows by 8 columns of a product: its loads of either factor are
// free of bank conflicts, 4 x 3 sums a thread of Q [K; S]^T for 7 words of 16 bytes, 4 x
// 8 of V^T K for 12 floats a token.  Bound by what shared memory gives to registers, 128
// bytes a cycle (4 x 4096 tokens x 16 heads fp32: 995 us, about 12 000 of a chunk's
// 16 000 cycles; fused multiply-adds 6000).  512 threads with half the sums each, and so
// more words for them, took 1352; one sum a thread along rows of o 1395.  The next
// chunk's rows are loaded while this one's are worked on.
template <typename E, int DK, int DV>
__global__ void __launch_bounds__(kThreads, 2) gdn_linattn_kernel(const GdnLinattnArgs a, int tiles, int states_only)
{
    extern __shared__ __align__(16) uint8_t raw[];
    Smem<DK, DV> &m = *reinterpret_cast<Smem<DK, DV> *>(raw);
    const int t = threadIdx.x, lane = t & 31, warp = t / 32;
    const int64_t unit = blockIdx.x;
    const int v0 = (int)(unit % tiles) * DV, h = (int)(unit / tiles % a.heads);
    Unit u;
    if (!find_unit(a, unit / tiles / a.heads, h, states_only, u)) return;
    const int dk = a.dk, nv = min(DV, a.dv - v0), g = h / (a.heads / a.groups);
    const E *q = static_cast<const E *>(a.q) + u.row * a.ld_q + (int64_t)g * dk;
    const E *k = static_cast<const E *>(a.k) + u.row * a.ld_k + (int64_t)g * dk;
    const E *v = static_cast<const E *>(a.v) + u.row * a.ld_v + (int64_t)h * a.dv + v0;
    const float *decay = a.log_decay + u.row * a.ld_decay + h;
    E *o = static_cast<E *>(a.o) + u.row * a.ld_o + (int64_t)h * a.dv + v0;

    Rows<E, DK> qr, kr;
    Rows<E, DV> vr;
    float decay_next = 0.f;
    auto load = [&](int c) {
        const int n = u.len - c;
        kr.load(k + c * a.ld_k, a.ld_k, n, dk);
        vr.load(v + c * a.ld_v, a.ld_v, n, nv);
        if (!states_only) qr.load(q + c * a.ld_q, a.ld_q, n, dk);
        if (t < 32) decay_next = lane < n ? decay[(int64_t)(c + lane) * a.ld_decay] : 0.f;
    };
    load(0);
    for (int i = t; i < DK * DV; i += kThreads) {
        const int kk = i % DK, d = i / DK;
        m.k[kC + d][kk] = u.in && kk < dk && d < nv ? u.in[(int64_t)(v0 + d) * dk + kk] : 0.f;
    }
    constexpr int OV = DV / 32;                                              // columns of o of a thread
    const int i0 = lane / 8 + warp % 2 * 4, j0 = lane % 8 + warp / 2 * 8;    // rows 8 apart; columns 32 apart
    constexpr int SV = DV / 16, SK = DK / 32;                                // rows and pairs of columns of S
    const int d0 = lane / 8 + warp / 2 * 4, k0 = 2 * (lane % 8 + warp % 2 * 8);  // 16 and 32 apart
    PieceDecay piece;
    for (int c = 0; c < u.len; c += kC) {
        const int n = min(kC, u.len - c);
        __syncthreads();
        const bool inf_k = kr.store(m.k), inf_v = vr.turn(m.v);
        if (!states_only) qr.store(m.q);
        if (t < 32) {
            Decays d;
            const float decay_now = decay_next;
            d.scan(decay_now);
            // Sums up to 2^8 are off by 5e-7 at most.  Which lanes have the exact ones depends on no
            // token behind them.
            const unsigned steep = __ballot_sync(0xffffffffu, !(fabsf(d.in) <= 8.f));
            float rest = 0.f;
            if (steep) {
                const float plain = d.in;
                rest = d.exact(decay_now);
                if (!(steep & (0xffffffffu >> (31 - lane)))) {
                    d.in = plain;
                    rest = 0.f;
                }
            }
            m.rest[lane] = rest;
            m.in[lane] = d.in;
            m.first[lane] = first_seen(d.mask, lane);
            const float start = decay_of(once(d.in));
            m.start[lane] = d.cut_upto(lane) ? 0.f : start;
            m.early[lane] = is_far(d.in) ? start : 1.f;
            m.add[lane] = d.cut_behind(lane) ? 0.f : decay_of(d.after);
            if (lane == 0) {
                m.kept = first_seen(d.mask, 31);
                const float all = chained_decay_of(once(d.total));
                m.all = d.mask ? 0.f : all;
                m.before = is_far(d.total) ? all : 1.f;
                if (states_only) piece.add(d.total, d.mask);
            }
        }
        const bool odd = __syncthreads_or(inf_k || inf_v);
        load(c + kC);
        float acc[4][OV];
        const float least = odd ? 1.175494351e-38f : 0.f;  // a decay that no token forgets leaves infinities as they are
        if (!states_only) {
            f32x2 sum[4][1 + OV] = {};
#pragma unroll 2
            for (int kk = 0; kk < DK; kk += 4) {
                float4 x[4], y[1 + OV];
#pragma unroll
                for (int e = 0; e < 4; ++e) x[e] = *reinterpret_cast<const float4 *>(&m.q[i0 + 8 * e][kk]);
#pragma unroll
                for (int f = 0; f <= OV; ++f) y[f] = *reinterpret_cast<const float4 *>(&m.k[j0 + 32 * f][kk]);
#pragma unroll
                for (int e = 0; e < 4; ++e)
#pragma unroll
                    for (int f = 0; f <= OV; ++f) dot4(x[e], y[f], sum[e][f]);
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int i = i0 + 8 * e;
                const float w = m.start[i], early = m.early[i];
                float lo, hi;
                unpack2(sum[e][0], lo, hi);
                const float f = at_least(decay_of(m.in[i] - m.in[j0] + (m.rest[i] - m.rest[j0])), least);
                m.P[i][j0] = j0 <= i && j0 >= m.first[i] ? (lo + hi) * f : 0.f;
#pragma unroll
                for (int f = 0; f < OV; ++f) {
                    unpack2(sum[e][1 + f], lo, hi);
                    acc[e][f] = w == 0.f ? 0.f : w * (early * (lo + hi));
                }
            }
        }
        __syncthreads();
        if (!states_only) {
            if (!odd) {
                f32x2 sum[4][OV] = {};
#pragma unroll 2
                for (int j = 0; j < kC; j += 4) {
                    float4 x[4], y[OV];
#pragma unroll
                    for (int e = 0; e < 4; ++e) x[e] = *reinterpret_cast<const float4 *>(&m.P[i0 + 8 * e][j]);
#pragma unroll
                    for (int f = 0; f < OV; ++f) y[f] = *reinterpret_cast<const float4 *>(&m.v[j0 + 32 * f][j]);
#pragma unroll
                    for (int e = 0; e < 4; ++e)
#pragma unroll
                        for (int f = 0; f < OV; ++f) dot4(x[e], y[f], sum[e][f]);
                }
#pragma unroll
                for (int e = 0; e < 4; ++e)
#pragma unroll
                    for (int f = 0; f < OV; ++f) {
                        float lo, hi;
                        unpack2(sum[e][f], lo, hi);
                        acc[e][f] += lo + hi;
                    }
            } else {  // a token sees nothing of those behind it, infinite or not; same order of sums
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int i = i0 + 8 * e;
#pragma unroll
                    for (int f = 0; f < OV; ++f) {
                        float sum[2] = {};
#pragma unroll
                        for (int r = 0; r < 2; ++r)
#pragma unroll 1
                            for (int j = r; j <= i; j += 2)
                                if (j >= m.first[i]) sum[r] = fmaf(m.P[i][j], m.v[j0 + 32 * f][j], sum[r]);
                        acc[e][f] += sum[0] + sum[1];
                    }
                }
            }
#pragma unroll
            for (int e = 0; e < 4; ++e)
#pragma unroll
                for (int f = 0; f < OV; ++f) {
                    const int i = i0 + 8 * e, d = j0 + 32 * f;
                    if (i < n && d < nv) o[(c + i) * a.ld_o + d] = from_f<E>(a.scale * acc[e][f]);
                }
        }
        if (odd) {  // what is forgotten adds nothing, where its factor of zero would make NaN
            __syncthreads();
            for (int i = t; i < m.kept * DK; i += kThreads) m.k[i / DK][i % DK] = 0.f;
            for (int i = t; i < m.kept * DV; i += kThreads) m.v[i % DV][i / DV] = 0.f;
            for (int i = m.kept * DV + t; i < kC * DV; i += kThreads)
                if (m.add[i / DV] == 0.f) m.v[i % DV][i / DV] = least_of(m.v[i % DV][i / DV]);
            __syncthreads();
            if (t < kC && t >= m.kept && m.add[t] == 0.f) m.add[t] = 1.f;
            __syncthreads();
        }
        f32x2 s[SV][SK] = {};
#pragma unroll 1
        for (int j = 0; j < n; j += 4) {
            float w[SV][4], f[4];
            ld_vec<float, 4>(&m.add[j], f);
#pragma unroll
            for (int x = 0; x < SV; ++x) {
                ld_vec<float, 4>(&m.v[d0 + 16 * x][j], w[x]);
#pragma unroll
                for (int e = 0; e < 4; ++e) w[x][e] *= f[e];
            }
#pragma unroll
            for (int e = 0; e < 4; ++e)
#pragma unroll
                for (int y = 0; y < SK; ++y) {
                    const float2 kk = *reinterpret_cast<const float2 *>(&m.k[j + e][k0 + 32 * y]);
#pragma unroll
                    for (int x = 0; x < SV; ++x)
                        s[x][y] = fma2(pack2(w[x][e], w[x][e]), pack2(kk.x, kk.y), s[x][y]);
                }
        }
        const float all = m.all, again = m.before;
#pragma unroll
        for (int x = 0; x < SV; ++x)
#pragma unroll
            for (int y = 0; y < SK; ++y) {
                float2 *S = reinterpret_cast<float2 *>(&m.k[kC + d0 + 16 * x][k0 + 32 * y]);
                const float2 before = *S;
                float lo, hi;
                unpack2(s[x][y], lo, hi);
                // columns past d_k stay zero: an infinite v makes NaN of their zeros
                lo = all == 0.f ? lo : fmaf(all, again * before.x, lo);
                hi = all == 0.f ? hi : fmaf(all, again * before.y, hi);
                *S = make_float2(k0 + 32 * y < dk ? lo : 0.f, k0 + 32 * y + 1 < dk ? hi : 0.f);
            }
    }
    __syncthreads();
    if (states_only && v0 == 0 && t == 0) a.piece_decay[unit / tiles] = piece.all();
    if (u.out)
        for (int i = t; i < DK * DV; i += kThreads) {
            const int kk = i % DK, d = i / DK;
            if (kk < dk && d < nv) u.out[(int64_t)(v0 + d) * dk + kk] = m.k[kC + d][kk];
        }
}

// The states that the pieces of each sequence start from, in place of what the
// pieces add; a piece's decay by its root, twice.  A block walks 4 x kThreads elements of one head's state through
// the pieces; the next piece's are in flight while this one's are added.
__global__ void __launch_bounds__(kThreads) gdn_linattn_chain_kernel(const GdnLinattnArgs a, int blocks)
{
    const int64_t per = (int64_t)a.dv * a.dk;
    const int64_t head = blockIdx.x / blocks;
    const int h = (int)(head % a.heads), n = (int)(head / a.heads);
    int64_t first;
    int count;
    if (a.cu_seqlens) {
        const int lo = a.cu_seqlens[n], hi = a.cu_seqlens[n + 1];
        if (lo < 0 || hi < lo || hi > a.T) return;
        first = lo / a.segment + n;
        count = hi > lo ? (hi - lo - 1) / a.segment + 1 : 1;
    } else {
        count = (int)(((int64_t)a.T + a.segment - 1) / a.segment);
        first = (int64_t)n * count;
    }
    const int e = a.state_in ? state_entry(a.slots, n, a.pool, a.status) : -1;
    const float *in = e >= 0 ? a.state_in + ((int64_t)e * a.heads + h) * per : nullptr;
    const int64_t i0 = (int64_t)(blockIdx.x % blocks) * (4 * kThreads) + threadIdx.x;
    float S[4], next[4];
    float *at = a.piece_state + (first * a.heads + h) * per;
#pragma unroll
    for (int x = 0; x < 4; ++x) {
        const int64_t i = i0 + x * kThreads;
        S[x] = in && i < per ? in[i] : 0.f;
        next[x] = count > 1 && i < per ? at[i] : 0.f;
    }
    for (int p = 0; p < count; ++p, at += a.heads * per) {
        float add[4];
        const bool more = p + 2 < count;
        const float f = p + 1 < count ? a.piece_decay[(first + p) * a.heads + h] : 0.f;
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            const int64_t i = i0 + x * kThreads;
            add[x] = next[x];
            if (more && i < per) next[x] = at[a.heads * per + i];
            if (i < per) at[i] = S[x];
            S[x] = f == 0.f ? add[x] : fmaf(f * S[x], f, add[x]);
        }
    }
}

// One new token per sequence.  Row i of S needs only itself, k, q and v_i: a warp
// takes kRows rows of one head at a time, a row over its lanes.  Bound by HBM:
// the state is read and written once (256 sequences x 16 heads of 128, 541 MB: 81 us, 6.7 TB/s).
constexpr int kRows = 8;

template <typename T, int V> __device__ __forceinline__ void ld_part(const T *p, int dk, int lane, bool vec, float (&x)[V])
{
    if (vec) {
        if (V * lane < dk) {
            ld_vec<T, V>(p + V * lane, x);
        } else {
#pragma unroll
            for (int j = 0; j < V; ++j) x[j] = 0.f;
        }
    } else {
#pragma unroll
        for (int j = 0; j < V; ++j) x[j] = lane + 32 * j < dk ? to_f(p[lane + 32 * j]) : 0.f;
    }
}

// Sums over the warp of 8 values at a time; lane l holds that of value l / 4.
__device__ __forceinline__ float sum_rows(const float (&x)[kRows], int lane)
{
    float y[4], z[2];
    const bool b16 = lane & 16, b8 = lane & 8, b4 = lane & 4;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        y[i] = (b16 ? x[i + 4] : x[i]) + __shfl_xor_sync(0xffffffffu, b16 ? x[i] : x[i + 4], 16);
#pragma unroll
    for (int i = 0; i < 2; ++i)
        z[i] = (b8 ? y[i + 2] : y[i]) + __shfl_xor_sync(0xffffffffu, b8 ? y[i] : y[i + 2], 8);
    float w = (b4 ? z[1] : z[0]) + __shfl_xor_sync(0xffffffffu, b4 ? z[0] : z[1], 4);
    w += __shfl_xor_sync(0xffffffffu, w, 2);
    return w + __shfl_xor_sync(0xffffffffu, w, 1);
}

// VEC: rows in words of V elements (d_k a multiple of V, V lane of each lane);
// else elements lane + 32 j.
template <typename E, int V, bool VEC>
__global__ void __launch_bounds__(kThreads) gdn_linattn_step_kernel(const GdnLinattnArgs a, int64_t items, int groups_of_rows)
{
    const int lane = threadIdx.x & 31;
    const int64_t warps = (int64_t)gridDim.x * (kThreads / 32);
    const int dk = a.dk, dv = a.dv, share = a.heads / a.groups;
    const int64_t per = (int64_t)dv * dk;
    for (int64_t it = (int64_t)blockIdx.x * (kThreads / 32) + threadIdx.x / 32; it < items; it += warps) {
        const int r0 = (int)(it % groups_of_rows) * kRows;
        const int64_t nh = it / groups_of_rows;
        const int n = (int)(nh / a.heads), h = (int)(nh % a.heads);
        const int e = state_entry(a.slots, n, a.pool, a.status);
        const int64_t at = ((int64_t)e * a.heads + h) * per + (int64_t)r0 * dk;
        float s[kRows][V];
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            if (a.state_in && e >= 0 && r0 + r < dv) {
                ld_part<float, V>(a.state_in + at + r * dk, dk, lane, VEC, s[r]);
            } else {
#pragma unroll
                for (int j = 0; j < V; ++j) s[r][j] = 0.f;
            }
        }
        const int row = lane / 4;
        const float d = chained_decay_of(a.log_decay[n * a.ld_decay + h] * kLog2e);
        float kk[V], qq[V];
        ld_part<E, V>(static_cast<const E *>(a.k) + n * a.ld_k + (int64_t)(h / share) * dk, dk, lane, VEC, kk);
        ld_part<E, V>(static_cast<const E *>(a.q) + n * a.ld_q + (int64_t)(h / share) * dk, dk, lane, VEC, qq);
        const float vr = r0 + row < dv ? to_f(static_cast<const E *>(a.v)[n * a.ld_v + (int64_t)h * dv + r0 + row]) : 0.f;
        float dot[kRows];
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            const float w = __shfl_sync(0xffffffffu, vr, 4 * r);
            dot[r] = 0.f;
#pragma unroll
            for (int j = 0; j < V; ++j) {
                // a lane without this column keeps zero: an infinite v would make NaN of it
                const float add = (VEC ? V * lane : lane + 32 * j) < dk ? w * kk[j] : 0.f;
                s[r][j] = d == 0.f ? add : fmaf(d, s[r][j], add);
                dot[r] = fmaf(s[r][j], qq[j], dot[r]);
            }
        }
        const float sum = sum_rows(dot, lane);
        if (lane % 4 == 0 && r0 + row < dv)
            static_cast<E *>(a.o)[n * a.ld_o + (int64_t)h * dv + r0 + row] = from_f<E>(a.scale * sum);
        if (e < 0) continue;
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            if (r0 + r >= dv) break;
            float *p = a.state_out + at + r * dk;
            if (VEC) {
                if (V * lane < dk) st_vec<float, V>(p + V * lane, s[r]);
            } else {
#pragma unroll
                for (int j = 0; j < V; ++j)
                    if (lane + 32 * j < dk) p[lane + 32 * j] = s[r][j];
            }
        }
    }
}

template <typename E, int V, bool VEC> cudaError_t step(const GdnLinattnArgs &a, cudaStream_t s)
{
    static int fit = 0;  // blocks resident at once; the same for every caller
    if (!fit) {
        int blocks = 0;
        const cudaError_t e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(
            &blocks, gdn_linattn_step_kernel<E, V, VEC>, kThreads, 0);
        if (e != cudaSuccess) return e;
        fit = gdn_ssm_sms() * (blocks > 0 ? blocks : 1);
    }
    const int rows = (a.dv + kRows - 1) / kRows;
    const int64_t items = (int64_t)a.N * a.heads * rows, need = (items + kThreads / 32 - 1) / (kThreads / 32);
    gdn_linattn_step_kernel<E, V, VEC><<<(unsigned)(need < fit ? need : fit), kThreads, 0, s>>>(a, items, rows);
    return cudaGetLastError();
}

template <typename E> cudaError_t step_by_width(const GdnLinattnArgs &a, cudaStream_t s)
{
    const int V = a.dk > 64 ? 4 : 2;
    const size_t al = V * sizeof(E);
    const bool vec = a.dk % V == 0 && a.ld_q % V == 0 && a.ld_k % V == 0 && aligned_to(a.q, al) && aligned_to(a.k, al) &&
                     aligned_to(a.state_in, V * 4) && aligned_to(a.state_out, V * 4);
    if (V == 4) return vec ? step<E, 4, true>(a, s) : step<E, 4, false>(a, s);
    return vec ? step<E, 2, true>(a, s) : step<E, 2, false>(a, s);
}

int64_t spans(const GdnLinattnArgs &a) { return a.segment ? a.pieces : a.N; }

template <typename E, int DK, int DV> cudaError_t simt_of(const GdnLinattnArgs &a, bool states_only, cudaStream_t s)
{
    const int tiles = (a.dv + DV - 1) / DV;
    const int64_t blocks = spans(a) * a.heads * tiles;
    if (blocks > 0x7fffffff) return cudaErrorInvalidConfiguration;
    const cudaError_t e = cudaFuncSetAttribute(gdn_linattn_kernel<E, DK, DV>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               (int)sizeof(Smem<DK, DV>));
    if (e != cudaSuccess) return e;
    gdn_linattn_kernel<E, DK, DV><<<(unsigned)blocks, kThreads, sizeof(Smem<DK, DV>), s>>>(a, tiles, states_only);
    return cudaGetLastError();
}

// 32 columns of v per block where 64 would leave multiprocessors empty.  us, fp32, d_k
// 128, of 32 and of 64: 4096 tokens x 16 heads (32 blocks of 64) 763, 998; 4 x 4096 x 16
// with d_v 64 (64 blocks) 763, 1010; with d_v 128 (128) 1252, 999.
template <typename E, int DK> cudaError_t simt(const GdnLinattnArgs &a, bool states_only, cudaStream_t s)
{
    const int64_t blocks = spans(a) * a.heads * ((a.dv + 63) / 64);
    return a.dv <= 32 || 5 * blocks < 4 * gdn_ssm_sms() ? simt_of<E, DK, 32>(a, states_only, s) : simt_of<E, DK, 64>(a, states_only, s);
}

template <typename E> cudaError_t simt_by_width(const GdnLinattnArgs &a, bool states_only, cudaStream_t s)
{
    if (a.dk <= 32) return simt<E, 32>(a, states_only, s);
    if (a.dk <= 64) return simt<E, 64>(a, states_only, s);
    if (a.dk <= 96) return simt<E, 96>(a, states_only, s);
    return simt<E, 128>(a, states_only, s);
}

cudaError_t pass(const GdnLinattnArgs &a, bool states_only, cudaStream_t s)
{
    if (gdn_linattn_tc_supported(a)) return gdn_linattn_tc(a, states_only, s);
    return a.dtype == 1 ? simt_by_width<__nv_bfloat16>(a, states_only, s) : simt_by_width<float>(a, states_only, s);
}

}  // namespace

// Whole sequences or pieces: the quicker by what was measured, us per chunk of 128
// tokens for the first block of a multiprocessor and for each more, and beside all
// chunks.
// Tensor cores: one document of 131 072 tokens x 8 heads whole 2592, in pieces 530; 4096
// tokens x 16 heads whole 92, 4 pieces 59; 2048 tokens whole 51, 4 pieces 39.5; 1024 tokens
// x 8 heads whole 29, 2 pieces 36; 4096 tokens x 32 heads whole 94.5, 2 pieces 98.
// CUDA cores, fp32 (blocks of 32 columns; one of 64 takes the time of two): 4096 tokens x
// 4 heads whole 752, pieces of 512 156, of 128 101; 16 heads whole 756, pieces of 2048 550,
// 512 320; 4 x 4096 x 16 whole 995; 517 x 2 heads whole 106, 5 pieces 53.
// Sequences of a pack are not seen from here: one that has nearly all of its rows (131 072
// rows x 8 heads, 8 sequences) is not cut, 2693, where pieces of 6912 take 554.
// Pieces are chosen to fill the multiprocessors once or up to as often as there is room.
void gdn_linattn_plan(bool tensor_cores, int N, int T, int heads, int dk, int dv, bool packed, int asked, int *segment,
                      int64_t *piece_slots)
{
    const double wide = 0.4 + 0.6 * ((dk + 31) / 32) / 4;  // tiles of d_k on CUDA cores
    const double kWhole = tensor_cores ? 2.55 : 21.5 * wide, kWholeMore = tensor_cores ? kWhole : 10 * wide, kWholeStart = 10;
    const double kCut = tensor_cores ? 4.5 : 31.5 * wide, kCutMore = tensor_cores ? kCut : 14 * wide, kCutStart = 20;
    const int kFills = tensor_cores ? 3 : 4;
    constexpr double kBytesPerUs = 6e6;
    constexpr int64_t kChunk = 128;
    const int64_t least = tensor_cores ? 4 : 1;  // chunks of a piece
    *segment = 0;
    *piece_slots = 0;
    if (N < 1 || T < 1) return;
    int64_t seg = ((int64_t)asked + kChunk - 1) / kChunk;
    if (asked <= 0) {
        const int sms = gdn_ssm_sms();
        const bool uneven = packed && N > 1;
        const int64_t per = (int64_t)heads * (tensor_cores ? (dv + 63) / 64 : (dv + 31) / 32), seqs = uneven ? 1 : N;
        // a packed sequence may be the longest by far; twice the mean is taken for it
        const int64_t all = (T + kChunk - 1) / kChunk, longest = uneven ? (2 * all + N - 1) / N : all;
        const double share = (double)all * seqs * per / sms;  // chunks per multiprocessor
        auto more = [&](int64_t blocks) { return (double)((blocks + sms - 1) / sms - 1); };
        const double chain = (double)heads * dk * dv * 16 / kBytesPerUs;  // per piece: its state written, read, written, read
        double best = kWholeStart + (!uneven ? (kWhole + kWholeMore * more(N * per)) * all
                                     : kWholeMore * share > kWhole * longest ? kWholeMore * share : kWhole * longest);
        seg = all;
        for (int k = 1; k <= kFills; ++k) {
            int64_t s = uneven ? (int64_t)(share / k) + 1 : (all * N * per + (int64_t)k * sms - 1) / ((int64_t)k * sms);
            if (!uneven) {  // as many pieces of a sequence as fit
                const int64_t p = (int64_t)k * sms / (N * per);
                if (p < 2) continue;
                s = (all + p - 1) / p;
            }
            if (s < least) s = least;
            if (s >= longest) continue;
            const int64_t pieces = uneven ? all / s + N : N * ((all + s - 1) / s);
            const double t = kCutStart + chain * pieces +
                             (uneven ? kCut * s + kCutMore * share : (kCut + kCutMore * more(pieces * per)) * s);
            if (t < best) {
                best = t;
                seg = s;
            }
        }
    }
    if (seg * kChunk >= T) return;
    *segment = (int)(seg * kChunk);
    *piece_slots = packed ? (int64_t)T / *segment + N : (int64_t)N * (((int64_t)T + *segment - 1) / *segment);
}

cudaError_t gdn_launch_linattn_fwd(const GdnLinattnArgs &a, cudaStream_t s, int *launches)
{
    *launches = 0;
    if (a.segment) {
        cudaError_t e = pass(a, true, s);
        if (e != cudaSuccess) return e;
        const int per_head = (int)(((int64_t)a.dv * a.dk + 4 * kThreads - 1) / (4 * kThreads));
        const int64_t chains = (int64_t)a.N * a.heads * per_head;
        if (chains > 0x7fffffff) return cudaErrorInvalidConfiguration;
        gdn_linattn_chain_kernel<<<(unsigned)chains, kThreads, 0, s>>>(a, per_head);
        e = cudaGetLastError();
        if (e != cudaSuccess) return e;
        *launches = 2;
    }
    *launches += 1;
    return pass(a, false, s);
}

cudaError_t gdn_launch_linattn_step(const GdnLinattnArgs &a, cudaStream_t s)
{
    return a.dtype == 1 ? step_by_width<__nv_bfloat16>(a, s) : step_by_width<float>(a, s);
}

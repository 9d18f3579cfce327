// Selective state space scan over prompts: the kernel and its launch, for one
// element type (gdn_ssm_bf16.cu, gdn_ssm_f32.cu).
//
// Per channel c with d_state fp32 states, token by token:
//
//     h[s] = exp(d A[c, s]) h[s] + d B[t, s] x        y = sum_s C[t, s] h[s] + D x
//
// with d = softplus(delta + bias); exp is 2^(d A log2 e).
//
// What bounds it is arithmetic: per token, channel and state an exponential (32
// per clock and SM) and four fp32 operations (128 lanes per clock), so 32 states
// per clock at best; a loop of this mix alone reaches 24.  HBM would allow 58
// for bf16 and 16 states.  Shared memory (128 bytes per clock into registers)
// comes next, at 16 to 80 bytes per lane and token by how operands are shared.
// The work is split so that no pipe does what another can:
//
//  - Recurrence warps (4 per block, 16 channels each; 8 with half the states
//    each when d_state > 16) do nothing but the recurrence and y = C h.  A lane
//    holds NS states of a pair of neighbouring channels, the operations on the
//    pair in packed instructions, and stores its part of the pair's y.
//  - What is done once per token and channel is done by other warps.  Four
//    prepare: the softplus, (d, d x) of a channel pair as one 16-byte word in a
//    hand-over buffer, and B and C widened.  Four finish: the sum of the parts of
//    y, D x, the gate and the store.  The recurrence warps need most registers and
//    take over what the others leave of the block's.
//  - Tiles of kTile tokens come into a ring by tensor copies where the rows allow
//    it, five per tile from one finishing thread (from a preparing one they
//    lengthened the whole block's turn: 236 against 210 us on the first shape
//    below).  Other rows come by copies of 16 or 4 bytes or through registers,
//    per thread (240 us with 2044 channels instead of 2048).  A bulk copy per row,
//    80 per tile, took 38 clocks each and twice the time.
//
// Measured, 16 states: 4 x 4096 tokens x 2048 channels 209 us in bf16 (a block per
// SM, 128 of 152 busy: 51 ns per token), 221 in fp32; x 9728 channels 662 us (two
// blocks per SM: 13 states per clock and SM).  More states, 2048 channels, bf16
// (fp32): 32 301 us (326), 64 522 (538), 128 908 (917).
//
// Everything is fp32 until y is stored, as in the step for single tokens.  The
// sum over states on the tensor cores (m16n8k8, tf32: the states as operand as
// they stand, of each product the one column of its token) takes 202 us when h is
// cut to that operand's 11 bits, which leaves y 3.5e-4 of sum |C h| short on
// average; with h in two such parts 270, with the lanes' fp32 parts of y added
// there in two parts 228.  The four lanes' parts added by shuffles, over four
// tokens at a time, took 219.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>
#include <string.h>

#include <type_traits>

#include "gdn_layer.h"
#include "gdn_layer.cuh"
#include "sm100_ptx.cuh"

namespace {

using namespace gdn_layer;

constexpr uint64_t kWaitLimit = 2000000000;     // ns a wait for a copy may take,
constexpr uint64_t kWaitAfterTimeout = 50000;   // and every later one once that ran out
constexpr int kTile = 16;            // tokens handed over at a time
constexpr int kHands = 2;            // hand-over buffers; a third: 213 against 208 us
constexpr int kPairs = 32;           // channel pairs per block: 4 warps of 8 pairs
constexpr int kCols = kPairs / 4;    // 8-channel columns of a token row
constexpr int kPrep = 128;           // preparing threads, and finishing ones: a column of a row each
static_assert(kCols * kTile == kPrep && 2 * kPairs == kScanChannels, "a column of a row per thread");

// The state in place s.  Places past the last state begin again with the first: a
// state of zeros there would become d x times zero, NaN for an infinite d x, and
// C's zero does not take that out of y.  The places of one state share its C.
__device__ __forceinline__ int wrapped(int s, int ds) { return s < ds ? s : s % ds; }

// The share of its state's C that place s of `places` has: 1/2, 1/4 and so on,
// the last one as much as the one before, so that products are exact and add up.
__device__ __forceinline__ float share_of(int s, int ds, int places)
{
    const int copies = (places - 1 - wrapped(s, ds)) / ds;  // beside the first
    return __uint_as_float((uint32_t)(127 - min(s / ds + 1, copies)) << 23);
}

template <int W> __device__ __forceinline__ void ld_state(const float *p, const int (&at)[W], float (&h)[W])
{
#pragma unroll
    for (int j = 0; j < W; ++j) h[j] = p[at[j]];
}

template <int W> __device__ __forceinline__ void st_state(float *p, int s0, int ds, const float (&h)[W])
{
#pragma unroll
    for (int j = 0; j < W; ++j)
        if (s0 + j < ds) p[s0 + j] = h[j];
}

// What a launch over tiles of tokens does.  A call whose sequences are one
// tile each is kWhole.  Cut into pieces, kPieces finds every piece's end state
// (the first from the sequence's own state, the others from zero) and the sum
// of its d, and kOutputs starts each piece from the states chained up to it:
// a run of tokens takes h to exp(A sum d) h + (its end state from zero).  The
// last piece's end state is not needed, and its place keeps the sequence's
// start state instead: kOutputs writes the final state while the first piece
// may still be starting, so in place that piece cannot read it from the pool.
enum Mode { kWhole, kPieces, kOutputs };

// How wide the copies into the ring can be.
enum Width { kWide, kWord, kSingle };  // 16 bytes (pairs whole); 4 bytes; through registers

// Threads and shared memory of one block of 64 channels.  The states are in H
// parts, a lane has NS of a part: d_state is padded to 4 NS H.  PIECES: the pass
// that has no C and no y.
template <typename E, int NS, int H, bool PIECES = false> struct Layout {
    static constexpr int kRecur = 4 * kPairs * H;         // recurrence threads
    static constexpr int kStates = 4 * NS * H;
    static constexpr int kBC = kTile * kStates / 2;       // pairs of B (and of C) per tile
    static constexpr int kRowElems = kTile * 2 * kPairs;
    // Tiles of inputs held or on their way.  A tile is fetched once the tile kRing before it is
    // finished, and waited for before the tile kHands before it is through the recurrence.
    static constexpr int kRing = sizeof(E) * kStates > 256 ? 4 : sizeof(E) * H > 4 ? 5 : 6;
    static constexpr size_t kSlot = sizeof(E) * (3 * kRowElems + 4 * kBC);  // x, delta, z, B, C
    static constexpr size_t kHandD = 16 * (size_t)kTile * kPairs;           // (d, d, d x, d x) per pair
    static constexpr size_t kHandB = 8 * (size_t)kBC;                       // B, and C, widened
    static constexpr size_t kHandC = kHandB;
    static constexpr size_t kPartY = 32 * (size_t)kTile * kPairs;           // y per pair, four lanes' parts of it
    static constexpr size_t kHand = kHandD + kHandB + (PIECES ? 0 : kHandC + H * kPartY);
    static constexpr size_t kBytes = kRing * kSlot + kHands * kHand + 8 * kRing;
    static_assert(kBC % kPrep == 0 && kBytes <= 227 * 1024 && kRing >= kHands + 2, "");
};

// The inputs as matrices of rows, for tensor copies of a tile's 64 channels (or
// padded states) by kTile rows.
struct Maps {
    CUtensorMap x, delta, z, b, c;
};

// Place of a channel pair's word in a token row of a hand-over buffer: a
// preparing thread writes four neighbouring words, which this spreads over the
// banks.
__device__ __forceinline__ int place(int pair) { return pair ^ ((pair >> 3) & 3); }

// Place, in 16-byte words, of word w (0 to 7) of y of an 8-channel column: words 2
// i and 2 i + 1 are the parts of its pair i from lanes 0, 1 and 2, 3.  A half warp
// writes all words of a column, a finishing thread reads word w of its own.
__device__ __forceinline__ int y_place(int col, int w) { return 8 * col + (w ^ col); }

// State i of lane quarter q in part `part`: runs of four, 16 apart.
template <int NS> __device__ __forceinline__ int state_of(int part, int q, int i)
{
    return part * 4 * NS + 16 * (i / 4) + 4 * q + i % 4;
}

// Eight elements of a row, the first `valid` of them from memory, zeros after.
template <typename E>
__device__ __forceinline__ void ring_copy(E *dst, const E *src, int valid, int width)
{
    constexpr int step = 16 / sizeof(E), word = 4 / sizeof(E);
    if (width == kWide && valid == 8) {
#pragma unroll
        for (int i = 0; i < 8; i += step) copy_async<16>(dst + i, src + i);
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; i += word) {  // `valid` is a multiple of a word here
        if (i < valid)
            copy_async<4>(dst + i, src + i);
        else
            *reinterpret_cast<uint32_t *>(dst + i) = 0;
    }
}

// Elements from[0] and from[1] of a row of B or C, neighbours where they are
// copied as one; zeros for a row past the end.
template <typename E>
__device__ __forceinline__ void ring_copy_pair(E *dst, const E *row, const int (&from)[2], bool live, int width)
{
    if (!live) {
        dst[0] = dst[1] = from_f<E>(0.f);
    } else if (width == kWide) {
        copy_async<2 * sizeof(E)>(dst, row + from[0]);
    } else if (sizeof(E) == 4) {
        copy_async<4>(dst, row + from[0]);
        copy_async<4>(dst + 1, row + from[1]);
    }
}

// The same for rows that no copy fits (bf16 off 4 bytes): through registers,
// loaded well before they are stored.
template <typename E, int N> struct Held {
    E v[N];
    __device__ __forceinline__ void load(const E *src, int valid)
    {
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = i < valid ? src[i] : from_f<E>(0.f);
    }
    __device__ __forceinline__ void load_pair(const E *row, const int (&from)[2], bool live)
    {
        v[0] = live ? row[from[0]] : from_f<E>(0.f);
        v[N - 1] = live ? row[from[1]] : from_f<E>(0.f);
    }
    __device__ __forceinline__ void store(E *dst) const  // aligned to the N elements
    {
        if constexpr (sizeof(E) == 2 && N % 2 == 0) {
            uint32_t w[N / 2];
#pragma unroll
            for (int i = 0; i < N / 2; ++i)
                w[i] = __bfloat16_as_ushort(v[2 * i]) | (uint32_t)__bfloat16_as_ushort(v[2 * i + 1]) << 16;
            if constexpr (N == 8)
                *reinterpret_cast<uint4 *>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
            else
                *reinterpret_cast<uint32_t *>(dst) = w[0];
        }
    }
};

// 2^(v / 2), twice of which takes a state over a piece, where 2^v may pass the
// largest number although what it multiplies to does not.  Kept from zero and
// from infinity: a zero state stays zero and an infinite one infinite, as token
// by token.
__device__ __forceinline__ float half_decay(float v)
{
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(ex2(0.5f * v)), "f"(FLT_MIN));
    asm("min.NaN.f32 %0, %0, %1;" : "+f"(r) : "f"(FLT_MAX));
    return r;
}

// Whether rows that need copies per thread have four warps of their own for them.
// bf16, 4 x 4096 tokens, 16 states, us with the copies made by preparing, by
// finishing and by fetching threads: 2044 channels (4-byte copies) 302, 359, 247;
// 2043 channels (2-byte loads) 308, 393, 281; 2048 channels x 13 states (B and C
// through registers) 243, 310, 209 (the fetching ones with today's sum of y: 240,
// 298, 218).  fp32 loses by them (203 channels 100 against
// 110: its recurrence wants the registers), and with more states per lane there
// are no registers for more warps.
template <typename E, int NS, int MODE, bool BULK> struct Fetchers {
    static constexpr bool on = !BULK && MODE != kPieces && NS == 4 && sizeof(E) == 2;
};

// Threads of a block: recurrence, then preparing, finishing, fetching ones.
template <typename E, int NS, int H, int MODE, bool BULK> struct Threads {
    static constexpr int n = Layout<E, NS, H>::kRecur +
                             (MODE == kPieces ? 1 : Fetchers<E, NS, MODE, BULK>::on ? 3 : 2) * kPrep;
};

template <typename E, int NS, int H, int MODE, bool BULK>
__global__ void __launch_bounds__(Layout<E, NS, H>::kRecur + (Fetchers<E, NS, MODE, BULK>::on ? 3 : 2) * kPrep,
                                  NS == 4 && H == 1 && BULK ? 2 : 1)
    gdn_ssm_fwd_kernel(const GdnSsmArgs a, const __grid_constant__ Maps maps, int tl, int tiles,
                       unsigned slots, int row_width, int bc_width)
{
    using L = Layout<E, NS, H, MODE == kPieces>;
    constexpr int kRing = L::kRing, kRecur = L::kRecur;
    extern __shared__ __align__(128) unsigned char smem[];
    Span s;
    // Pieces of one chunk of channels side by side; whole packed sequences by length, each with
    // its chunks side by side.
    const bool ranked = MODE == kWhole && a.cu_seqlens;
    const unsigned chunks = gridDim.x / slots;
    const int64_t slot = ranked ? blockIdx.x / chunks : blockIdx.x % slots;
    const int chunk = ranked ? blockIdx.x % chunks : blockIdx.x / slots;
    if (ranked ? !find_ranked(a.cu_seqlens, a.N, a.T, (int)slot, a.status, s)
               : !find_span(a.cu_seqlens, a.N, a.T, tl, slot, tiles, a.status, s))
        return;
    const int pieces = s.len > tl ? (s.len - 1) / tl + 1 : 1;
    if (MODE == kPieces && s.tile == pieces - 1) return;
    const int t0 = s.tile * tl, t1 = t0 + min(s.len - t0, tl);
    const int ntiles = (t1 - t0 + kTile - 1) / kTile;
    // the block's channels: [cbase, cend), all of one group
    const int per_group = a.channels / a.groups;
    const int blocks = (per_group + 2 * kPairs - 1) / (2 * kPairs);
    const int g = chunk / blocks;
    const int cbase = g * per_group + (chunk % blocks) * 2 * kPairs;
    const int cend = min(cbase + 2 * kPairs, (g + 1) * per_group);

    auto hand = [&](int k) { return smem + kRing * L::kSlot + k % kHands * L::kHand; };
    auto hand_b = [&](int k) { return hand(k) + L::kHandD; };
    auto hand_c = [&](int k) { return hand(k) + L::kHandD + L::kHandB; };
    auto part_y = [&](int k, int part) { return hand(k) + L::kHandD + L::kHandB + L::kHandC + part * L::kPartY; };
    auto next = [](int at) { return at + 1 == kRing ? 0 : at + 1; };
    uint64_t *landed = reinterpret_cast<uint64_t *>(smem + kRing * L::kSlot + kHands * L::kHand);  // per ring slot
    uint64_t limit = kWaitLimit;
    // Tiles that other threads than the preparing ones copy are waited for at these; else each
    // preparing thread waits for its own copies, and the finishing ones learn of them at kDone.
    constexpr bool kFetch = Fetchers<E, NS, MODE, BULK>::on, kLanded = BULK || kFetch;
    auto wait_for = [&](int at, int round) {  // the copies of ring slot `at`, its `round`th use
        if (!sm100::mbar_wait(&landed[at], round & 1, limit)) {
            atomicOr(a.status, GDN_DEV_WAIT_TIMEOUT);
            limit = kWaitAfterTimeout;
        }
    };
    if (kLanded) {
        if (threadIdx.x == 0) {
            for (int i = 0; i < kRing; ++i) sm100::mbar_init(&landed[i], BULK ? 1 : 2 * kPrep);
            sm100::fence_mbar_init();
        }
        __syncthreads();
    }
    // Barriers.  Of hand-over buffer i: kFull + i, prepared (prepare -> recurrence); kDone + i,
    // read, and y written (recurrence -> prepare, finish, fetch).  kFree: y read and the ring slot
    // with it (finish -> prepare).  kPieces has no finishing warps.
    enum { kFull = 1, kDone = kFull + kHands, kFree = kDone + kHands };
    constexpr int kFullN = kRecur + kPrep, kDoneN = Threads<E, NS, H, MODE, BULK>::n;

    // Two blocks of 384 threads leave 80 registers each: 112 for the recurrence warps, 64 for
    // the other eight (112 + 2 x 64 = 3 x 80).
    constexpr bool kSplit = NS == 4 && H == 1 && BULK && MODE != kPieces;

    if (threadIdx.x < kRecur) {  // ---- recurrence
        if (kSplit) asm volatile("setmaxnreg.inc.sync.aligned.u32 112;");
        const int part = H == 1 ? 0 : threadIdx.x / (4 * kPairs);
        const int q = threadIdx.x & 3, pair = (threadIdx.x >> 2) & (kPairs - 1);
        const int c = cbase + 2 * pair, ds = a.d_state;
        const int entry = state_entry(a.slots, s.n, a.pool, a.status);
        const int64_t slot0 = slot - s.tile;  // the sequence's first piece
        f32x2 h[NS], A[NS], dsum = 0;
#pragma unroll
        for (int i = 0; i < NS; i += 4) {
            const int s0 = state_of<NS>(part, q, i);
            const int at[4] = {wrapped(s0, ds), wrapped(s0 + 1, ds), wrapped(s0 + 2, ds), wrapped(s0 + 3, ds)};
            float hv[2][4], Av[2][4];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
#pragma unroll
                for (int u = 0; u < 4; ++u) hv[j][u] = Av[j][u] = 0.f;
                if (c + j >= cend) continue;
                auto piece = [&](int64_t k) { return a.piece_state + ((size_t)k * a.channels + c + j) * ds; };
                ld_state(a.A + (size_t)(c + j) * ds, at, Av[j]);
#pragma unroll
                for (int u = 0; u < 4; ++u) Av[j][u] = decay_rate(Av[j][u]);
                if (MODE == kOutputs && pieces > 1) {
                    ld_state(piece(s.tile == 0 ? slot0 + pieces - 1 : slot0), at, hv[j]);
                    for (int k = 1; k < s.tile; ++k) {
                        const float sum = a.piece_delta[(size_t)(slot0 + k) * a.channels + c + j];
                        float e[4];
                        ld_state(piece(slot0 + k), at, e);
#pragma unroll
                        for (int u = 0; u < 4; ++u) {
                            const float half = half_decay(sum * Av[j][u]);
                            hv[j][u] = fmaf(half * hv[j][u], half, e[u]);
                        }
                    }
                } else if (s.tile == 0 && a.state_in && entry >= 0) {
                    ld_state(a.state_in + ((size_t)entry * a.channels + c + j) * ds, at, hv[j]);
                }
                if (MODE == kPieces && s.tile == 0) st_state(piece(slot0 + pieces - 1), s0, ds, hv[j]);
            }
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                h[i + u] = pack2(hv[0][u], hv[1][u]);
                A[i + u] = pack2(Av[0][u], Av[1][u]);
            }
        }
        // A warp has its scheduler nearly to itself, so it covers its own latencies: a token's
        // words are loaded and its decays computed (kAhead) while the token before goes through
        // the states, and its y is picked up one token later.  With more states per lane there is
        // as much to overlap within a token, and no registers for this.
        constexpr int kAhead = NS == 4 ? 1 : 0;
        for (int k = 0; k < ntiles; ++k) {
            const ulonglong2 *dx = reinterpret_cast<const ulonglong2 *>(hand(k)) + place(pair);
            const float4 *B = reinterpret_cast<const float4 *>(hand_b(k)) + state_of<NS>(part, q, 0) / 4;
            const float4 *C = reinterpret_cast<const float4 *>(hand_c(k)) + state_of<NS>(part, q, 0) / 4;
            unsigned char *yout = part_y(k, part) + 16 * y_place(pair / 4, 2 * (pair & 3) + q / 2) + 8 * (q & 1);
            ulonglong2 dv[2 + kAhead];
            float4 bv[2 + kAhead], cv[2 + kAhead];
            f32x2 e[1 + kAhead][NS], w[1 + kAhead][NS], tile_sum = 0;
            auto word = [&](const float4 *p, int t, int i) { return p[(t * L::kStates + 4 * i) / 4]; };
            auto load = [&](int t) {
                dv[t % (2 + kAhead)] = dx[t * kPairs];  // d, d x
                if (NS > 4) return;
                bv[t % (2 + kAhead)] = word(B, t, 0);
                if (MODE != kPieces) cv[t % (2 + kAhead)] = word(C, t, 0);
            };
            auto decay = [&](int t) {
                const ulonglong2 v = dv[t % (2 + kAhead)];
                const int p = t % (1 + kAhead);
                if (MODE == kPieces) tile_sum = add2(tile_sum, v.x);
                float x0, x1;
                unpack2(v.y, x0, x1);
#pragma unroll
                for (int i = 0; i < NS; i += 4) {
                    const float4 b4 = NS == 4 ? bv[t % (2 + kAhead)] : word(B, t, i);
                    const float bb[4] = {b4.x, b4.y, b4.z, b4.w};
#pragma unroll
                    for (int u = 0; u < 4; ++u) {
                        e[p][i + u] = ex2x2(fma2(v.x, A[i + u], dup2(kDecayShift)));
                        w[p][i + u] = pack2(x0 * bb[u], x1 * bb[u]);
                    }
                }
            };
            part_sync(kFull + k % kHands, kFullN);
            load(0);
            if (kAhead) {
                load(1);
                decay(0);
            }
#pragma unroll
            for (int t = 0; t < kTile; ++t) {
                if (t + 1 + kAhead < kTile) load(t + 1 + kAhead);
                if (t + kAhead < kTile) decay(t + kAhead);
#pragma unroll
                for (int i = 0; i < NS; ++i) h[i] = fma2(e[t % (1 + kAhead)][i], h[i], w[t % (1 + kAhead)][i]);
                if constexpr (MODE != kPieces) {
                    float y0 = 0.f, y1 = 0.f;
#pragma unroll
                    for (int i = 0; i < NS; i += 4) {
                        const float4 c4 = NS == 4 ? cv[t % (2 + kAhead)] : word(C, t, i);
                        const float cc[4] = {c4.x, c4.y, c4.z, c4.w};
#pragma unroll
                        for (int u = 0; u < 4; ++u) {
                            float h0, h1;
                            unpack2(h[i + u], h0, h1);
                            y0 = fmaf(cc[u], h0, y0);
                            y1 = fmaf(cc[u], h1, y1);
                        }
                    }
                    *reinterpret_cast<f32x2 *>(yout + 32 * kPairs * t) = pack2(y0, y1);
                }
            }
            if (MODE == kPieces) dsum = add2(dsum, tile_sum);
            part_arrive(kDone + k % kHands, kDoneN);
        }
        float d1[2];
        unpack2(dsum, d1[0], d1[1]);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            if (c + j >= cend) continue;
            float *out = nullptr;
            if (MODE == kPieces) {
                out = a.piece_state + ((size_t)slot * a.channels + c + j) * ds;
                if (q == 0 && part == 0) a.piece_delta[(size_t)slot * a.channels + c + j] = d1[j];
            } else if (s.tile == pieces - 1 && a.state_out && entry >= 0) {
                out = a.state_out + ((size_t)entry * a.channels + c + j) * ds;
            }
            if (!out) continue;
#pragma unroll
            for (int i = 0; i < NS; i += 4) {
                float v[4];
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    float lo, hi;
                    unpack2(h[i + u], lo, hi);
                    v[u] = j ? hi : lo;
                }
                st_state(out, state_of<NS>(part, q, i), ds, v);
            }
        }
        return;
    }

    if (kSplit) asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
    // ---- prepare and finish: a thread has one 8-channel column of one row of every tile
    const int id = threadIdx.x & (kPrep - 1), col = id % kCols, row = id / kCols;
    const int c = cbase + 8 * col, nc = max(0, min(8, cend - c)), off = id * 8;
    const int rows = nc > 0 ? t1 - t0 - row : 0;  // this thread's rows are those of tiles k with 16 k < rows
    const int64_t first = s.row + t0, mine = first + (rows > 0 ? row : 0);
    const int cc = nc > 0 ? c : cbase;
    auto column = [&](const float *p, f32x2 (&v)[4]) {  // of a vector over channels
#pragma unroll
        for (int i = 0; i < 4; ++i)
            v[i] = pack2(p && 2 * i < nc ? p[c + 2 * i] : 0.f, p && 2 * i + 1 < nc ? p[c + 2 * i + 1] : 0.f);
    };

    // One thread fetches a tile: whole boxes, where rows past the piece's end are another's or
    // zeros, and masked later.  Five copies take a warp longer than its share of a tile's other
    // work, so it is a finishing warp's, the ones with time to spare.
    auto fetch = [&](int k, int at) {
        if (k >= ntiles) return;
        constexpr int kX = L::kRowElems * sizeof(E), kB = 2 * L::kBC * sizeof(E);
        unsigned char *r = smem + at * L::kSlot;
        const int y = (int)(first + k * kTile), sc = g * a.d_state;
        sm100::mbar_arrive_expect_tx(&landed[at], MODE == kPieces ? 2 * kX + kB : (a.z ? 3 : 2) * kX + 2 * kB);
        copy_box(r, &maps.x, cbase, y, &landed[at]);
        copy_box(r + kX, &maps.delta, cbase, y, &landed[at]);
        copy_box(r + 3 * kX, &maps.b, sc, y, &landed[at]);
        if (MODE == kPieces) return;
        copy_box(r + 3 * kX + kB, &maps.c, sc, y, &landed[at]);
        if (a.z) copy_box(r + 2 * kX, &maps.z, cbase, y, &landed[at]);
    };

    // pair p = id + i kPrep of B and C of a tile: a token's states 2 (p % kHalf) and the next
    constexpr int kHalf = L::kStates / 2, kPer = L::kBC / kPrep, kTokStep = kPrep / kHalf;
    const int st = 2 * (id % kHalf), tok0 = id / kHalf;
    const int from[2] = {wrapped(st, a.d_state), wrapped(st + 1, a.d_state)};
    const float share[2] = {share_of(st, a.d_state, L::kStates), share_of(st + 1, a.d_state, L::kStates)};
    const int64_t channel = (int64_t)g * a.d_state;

    // Copies per thread: what it copies next; rows past the end are never read
    // (their address stays on the piece's first row).
    const E *x_in = nullptr, *d_in = nullptr, *z_in = nullptr, *b_in = nullptr, *c_in = nullptr;
    if (!BULK) {
        x_in = static_cast<const E *>(a.x) + mine * a.ld_x + cc;
        d_in = static_cast<const E *>(a.delta) + mine * a.ld_delta + cc;
        z_in = a.z ? static_cast<const E *>(a.z) + mine * a.ld_z + cc : nullptr;
        b_in = static_cast<const E *>(a.Bm) + first * a.ld_b + channel;
        c_in = static_cast<const E *>(a.Cm) + first * a.ld_c + channel;
    }

    constexpr bool kHold = !BULK && sizeof(E) == 2;
    Held<E, kHold ? 8 : 1> held_x, held_d, held_z;
    Held<E, kHold ? 2 : 1> held_b[kHold ? kPer : 1], held_c[kHold ? kPer : 1];
    auto hold = [&](int k) {  // the next issue's rows that have to go through registers
        if (!kHold || k >= ntiles) return;
        if (row_width == kSingle) {
            const int valid = k * kTile < rows ? nc : 0;
            held_x.load(x_in, valid);
            held_d.load(d_in, valid);
            held_z.load(z_in, MODE != kPieces && a.z ? valid : 0);
            if (kFetch && (k + 1) * kTile < rows) {  // the next turn's loads then wait for L2 alone
                prefetch(x_in + kTile * a.ld_x);
                prefetch(d_in + kTile * a.ld_delta);
                if (a.z) prefetch(z_in + kTile * a.ld_z);
            }
        }
        if (bc_width == kSingle)
#pragma unroll
            for (int i = 0; i < (kHold ? kPer : 1); ++i) {
                const int t = tok0 + i * kTokStep;
                const bool live = k * kTile + t < t1 - t0;
                held_b[i].load_pair(b_in + t * a.ld_b, from, live);
                held_c[i].load_pair(c_in + t * a.ld_c, from, MODE != kPieces && live);
            }
    };
    auto issue = [&](int k, int at) {  // tile k into ring slot `at`
        if (BULK) {
            if (MODE == kPieces && id == 0) fetch(k, at);
            return;
        }
        if (k < ntiles) {
            E *r = reinterpret_cast<E *>(smem + at * L::kSlot);
            const int valid = k * kTile < rows ? nc : 0;
            if (kHold && row_width == kSingle) {
                held_x.store(r + off);
                held_d.store(r + L::kRowElems + off);
                held_z.store(r + 2 * L::kRowElems + off);
            } else {
                ring_copy<E>(r + off, x_in, valid, row_width);
                ring_copy<E>(r + L::kRowElems + off, d_in, valid, row_width);
                if (MODE != kPieces && a.z) ring_copy<E>(r + 2 * L::kRowElems + off, z_in, valid, row_width);
            }
            E *rb = r + 3 * L::kRowElems + 2 * id, *rc = rb + 2 * L::kBC;
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                const int t = tok0 + i * kTokStep;
                const bool live = k * kTile + t < t1 - t0;
                if (kHold && bc_width == kSingle) {
                    held_b[i].store(rb + 2 * i * kPrep);
                    held_c[i].store(rc + 2 * i * kPrep);
                } else {
                    ring_copy_pair<E>(rb + 2 * i * kPrep, b_in + t * a.ld_b, from, live, bc_width);
                    if (MODE != kPieces) ring_copy_pair<E>(rc + 2 * i * kPrep, c_in + t * a.ld_c, from, live, bc_width);
                }
            }
            if ((k + 1) * kTile < rows) {
                x_in += kTile * a.ld_x;
                d_in += kTile * a.ld_delta;
                z_in += kTile * a.ld_z;
            }
            b_in += kTile * a.ld_b;
            c_in += kTile * a.ld_c;
            if (kLanded) {  // once for the copies, once for what was stored
                copy_arrive(&landed[at]);
                sm100::mbar_arrive(&landed[at]);
            }
        }
        if (!kLanded) copy_commit();  // one group per tile, so that a group's number is its tile's
    };

    if (kFetch && threadIdx.x >= kRecur + 2 * kPrep) {  // ---- fetch
#pragma unroll 1
        for (int k = 0; k < kRing - 1; ++k) {
            hold(k);
            issue(k, k);
        }
#pragma unroll 1
        for (int k = 0, at = kRing - 1; k < ntiles; ++k, at = next(at)) {
            hold(k - 1 + kRing);
            part_sync(kDone + k % kHands, kDoneN);  // as at the end of a finishing thread's turn
            issue(k - 1 + kRing, at);
        }
        return;
    }

    if (MODE != kPieces && threadIdx.x >= kRecur + kPrep) {  // ---- finish
        if (BULK && id == 0)
            for (int k = 0; k < kRing - 1; ++k) fetch(k, k);
        f32x2 D[4];
        column(a.D, D);
        E *out = static_cast<E *>(a.y) + mine * a.ld_y + cc;
        for (int k = 0, at = 0, round = 0; k < ntiles; ++k, at = next(at), round += at == 0) {
            const E *r = reinterpret_cast<const E *>(smem + at * L::kSlot);
            float x[8], z[8];
            f32x2 sum[4];
            if (kLanded) wait_for(at, round);
            part_sync(kDone + k % kHands, kDoneN);
            ld_vec<E, 8>(r + off, x);
            if (a.z) ld_vec<E, 8>(r + 2 * L::kRowElems + off, z);
#pragma unroll
            for (int part = 0; part < H; ++part) {
                const ulonglong2 *p = reinterpret_cast<const ulonglong2 *>(part_y(k, part)) + row * 2 * kPairs;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const ulonglong2 u = p[y_place(col, 2 * i)], v = p[y_place(col, 2 * i + 1)];
                    const f32x2 four = add2(add2(u.x, u.y), add2(v.x, v.y));
                    sum[i] = part ? add2(sum[i], four) : four;
                }
            }
            part_arrive(kFree, 2 * kPrep);
            if (k * kTile < rows) {
                float y[8];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    f32x2 v = sum[i];
                    if (a.D) v = fma2(D[i], pack2(x[2 * i], x[2 * i + 1]), v);  // not 0 x: x may be infinite
                    if (a.z) v = mul2(v, silu2(pack2(z[2 * i], z[2 * i + 1])));
                    unpack2(v, y[2 * i], y[2 * i + 1]);
                }
                if (BULK || row_width == kWide) {
                    st_vec<E, 8>(out, y);
                } else if (sizeof(E) == 2 && row_width == kWord) {
#pragma unroll
                    for (int i = 0; i < 8; i += 2)
                        if (i < nc) *reinterpret_cast<uint32_t *>(out + i) = narrow_pair(y[i], y[i + 1]);
                } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        if (i < nc) out[i] = from_f<E>(y[i]);
                }
                out += kTile * a.ld_y;
            }
            // every finishing thread came to this tile's barrier, so the slot before is free
            if (BULK && id == 0) fetch(k - 1 + kRing, at == 0 ? kRing - 1 : at - 1);
        }
        return;
    }

    // ---- prepare
    f32x2 bias[4];
    column(a.delta_bias, bias);
    // Tile k from ring slot `at` into its hand-over buffer.  `edge`: rows past the end, where
    // the ring may hold anything, are set to zero, and padding repeats states.
    auto prepare_as = [&](int k, int at, auto edge) {
        constexpr bool kEdge = decltype(edge)::value;
        const E *r = reinterpret_cast<const E *>(smem + at * L::kSlot);
        float x[8], d[8];
        ld_vec<E, 8>(r + L::kRowElems + off, d);
        ld_vec<E, 8>(r + off, x);
        ulonglong2 *dx = reinterpret_cast<ulonglong2 *>(hand(k)) + row * kPairs;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f32x2 v = add2(pack2(d[2 * i], d[2 * i + 1]), bias[i]);
            if (a.softplus) v = softplus2(v);
            ulonglong2 word = make_ulonglong2(v, mul2(v, pack2(x[2 * i], x[2 * i + 1])));
            if (kEdge && k * kTile >= rows) word = make_ulonglong2(0, 0);  // exp(0) h + 0
            dx[place(4 * col + i)] = word;
        }
        const E *rb = r + 3 * L::kRowElems + 2 * id, *rc = rb + 2 * L::kBC;
        float2 *B = reinterpret_cast<float2 *>(hand_b(k)) + id;
        float2 *C = reinterpret_cast<float2 *>(hand_c(k)) + id;
        auto pair = [&](const E *p, float (&v)[2]) {
            if (kEdge && BULK) {  // boxes hold other groups' states in padding; copied pairs are right
                v[0] = to_f(p[from[0] - st]);
                v[1] = to_f(p[from[1] - st]);
            } else {
                ld_vec<E, 2>(p, v);
            }
        };
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const bool live = !kEdge || k * kTile + tok0 + i * kTokStep < t1 - t0;
            float v[2];
            pair(rb + 2 * i * kPrep, v);
            B[i * kPrep] = live ? make_float2(v[0], v[1]) : make_float2(0.f, 0.f);
            if (MODE == kPieces) continue;
            pair(rc + 2 * i * kPrep, v);
            if (kEdge) {
                v[0] *= share[0];
                v[1] *= share[1];
            }
            C[i * kPrep] = live ? make_float2(v[0], v[1]) : make_float2(0.f, 0.f);
        }
    };
    auto prepare = [&](int k, int at) {
        if ((k + 1) * kTile <= t1 - t0 && a.d_state == L::kStates && cend - cbase == 2 * kPairs)
            prepare_as(k, at, std::false_type());
        else
            prepare_as(k, at, std::true_type());
    };

    if (!kFetch) {
#pragma unroll 1
        for (int k = 0; k < kRing; ++k) {
            hold(k);
            issue(k, k);
        }
    }
    auto wait_tile = [&](int k, int at, int round) {  // copies of tile k, of at least k + 1 and at most
        if (kLanded)                                   // k + kRing - kHands + 1 issued by this thread
            wait_for(at, round);
        else
            copy_wait<kRing - kHands - 1>();
    };
    if (!kLanded) copy_wait<kRing - kHands>();
    for (int k = 0; k < kHands && k < ntiles; ++k) {
        if (kLanded) wait_for(k, 0);
        prepare(k, k);
        part_arrive(kFull + k, kFullN);
    }
#pragma unroll 1
    for (int k = 0, done = 0, ahead = kHands % kRing, round = 0; k < ntiles;
         ++k, done = next(done), ahead = next(ahead)) {
        round += ahead == 0;
        if (!kFetch) hold(k + kRing);
        if (k + kHands < ntiles) wait_tile(k + kHands, ahead, round);
        part_sync(kDone + k % kHands, kDoneN);
        if (k + kHands < ntiles) prepare(k + kHands, ahead);
        if (MODE != kPieces) part_sync(kFree, 2 * kPrep);
        if (k + kHands < ntiles) part_arrive(kFull + k % kHands, kFullN);
        if (!kFetch) issue(k + kRing, done);
    }
}

// Copy widths into the ring: 16 bytes when whole 8-channel columns start on
// 16-byte boundaries in every matrix, 4 bytes when bf16 pairs are aligned (fp32
// elements always are).
template <typename E> int row_width(const GdnSsmArgs &a)
{
    const int per_group = a.channels / a.groups;
    const void *p[] = {a.x, a.delta, a.y, a.z};
    const int64_t ld[] = {a.ld_x, a.ld_delta, a.ld_y, a.z ? a.ld_z : 0};
    bool wide = per_group % 8 == 0, word = per_group % (4 / sizeof(E)) == 0;
    for (int i = 0; i < 4; ++i) {
        wide = wide && aligned16(p[i]) && ld[i] * sizeof(E) % 16 == 0;
        word = word && aligned_to(p[i], 4) && ld[i] * sizeof(E) % 4 == 0;
    }
    return wide ? kWide : word ? kWord : kSingle;
}

template <typename E> int bc_width(const GdnSsmArgs &a)
{
    const bool pairs = a.d_state % 2 == 0 && a.ld_b % 2 == 0 && a.ld_c % 2 == 0 &&
                       aligned_to(a.Bm, 2 * sizeof(E)) && aligned_to(a.Cm, 2 * sizeof(E));
    return pairs ? kWide : sizeof(E) == 4 ? kWord : kSingle;
}

// Tensor copies want a matrix and its rows on 16-byte boundaries, boxes that
// start on them, and row numbers of 31 bits.
template <typename E> bool box_rows(const GdnSsmArgs &a)
{
    const int64_t rows = a.cu_seqlens ? a.T : (int64_t)a.N * a.T;
    return row_width<E>(a) == kWide && a.d_state * sizeof(E) % 16 == 0 && a.ld_b * sizeof(E) % 16 == 0 &&
           a.ld_c * sizeof(E) % 16 == 0 && aligned16(a.Bm) && aligned16(a.Cm) && rows > 0 &&
           rows <= 0x7fffffff - kTile;
}

PFN_cuTensorMapEncodeTiled_v12000 map_encoder()
{
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;  // the same for every thread
    if (!fn) {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    }
    return fn;
}

template <typename E> bool make_maps(const GdnSsmArgs &a, int states, Maps *m)
{
    const PFN_cuTensorMapEncodeTiled_v12000 encode = map_encoder();
    if (!encode) return false;
    const cuuint64_t rows = a.cu_seqlens ? a.T : (cuuint64_t)a.N * a.T;
    auto map = [&](CUtensorMap *to, const void *p, int64_t ld, int columns, int box_columns) {
        const cuuint64_t dims[2] = {(cuuint64_t)columns, rows}, strides[1] = {(cuuint64_t)ld * sizeof(E)};
        const cuuint32_t box[2] = {(cuuint32_t)box_columns, kTile}, steps[2] = {1, 1};
        return encode(to, sizeof(E) == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32,
                      2, const_cast<void *>(p), dims, strides, box, steps, CU_TENSOR_MAP_INTERLEAVE_NONE,
                      CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                      CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
    };
    return map(&m->x, a.x, a.ld_x, a.channels, 2 * kPairs) &&
           map(&m->delta, a.delta, a.ld_delta, a.channels, 2 * kPairs) &&
           (!a.z || map(&m->z, a.z, a.ld_z, a.channels, 2 * kPairs)) &&
           map(&m->b, a.Bm, a.ld_b, a.groups * a.d_state, states) &&
           map(&m->c, a.Cm, a.ld_c, a.groups * a.d_state, states);
}

template <typename E, int NS, int H, int MODE, bool BULK>
cudaError_t launch_mode(const GdnSsmArgs &a, const Maps &maps, int tl, int tiles, int64_t slots, cudaStream_t s)
{
    using L = Layout<E, NS, H, MODE == kPieces>;
    const int per_group = a.channels / a.groups;
    const int64_t grid = slots * a.groups * ((per_group + 2 * kPairs - 1) / (2 * kPairs));
    if (grid > 0x7fffffff) return cudaErrorInvalidConfiguration;
    cudaError_t e = cudaFuncSetAttribute(gdn_ssm_fwd_kernel<E, NS, H, MODE, BULK>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, (int)L::kBytes);
    if (e != cudaSuccess) return e;
    gdn_ssm_fwd_kernel<E, NS, H, MODE, BULK><<<(unsigned)grid, Threads<E, NS, H, MODE, BULK>::n, L::kBytes, s>>>(
        a, maps, tl, tiles, (unsigned)slots, row_width<E>(a), bc_width<E>(a));
    return cudaGetLastError();
}

template <typename E, int NS, int H, bool BULK> cudaError_t launch_modes(const GdnSsmArgs &a, cudaStream_t s)
{
    Maps maps;
    memset(&maps, 0, sizeof(maps));
    if (BULK && !make_maps<E>(a, Layout<E, NS, H>::kStates, &maps)) return cudaErrorInvalidValue;
    if (a.segment) {
        const int tiles = (a.T - 1) / a.segment + 1;
        const cudaError_t e = launch_mode<E, NS, H, kPieces, BULK>(a, maps, a.segment, tiles, a.pieces, s);
        return e != cudaSuccess ? e : launch_mode<E, NS, H, kOutputs, BULK>(a, maps, a.segment, tiles, a.pieces, s);
    }
    const int tl = a.T > 0 ? a.T : 1;
    return launch_mode<E, NS, H, kWhole, BULK>(a, maps, tl, 1, a.N, s);
}

template <typename E, int NS, int H> cudaError_t launch_fwd(const GdnSsmArgs &a, cudaStream_t s)
{
    return box_rows<E>(a) ? launch_modes<E, NS, H, true>(a, s) : launch_modes<E, NS, H, false>(a, s);
}

// Two warps per scheduler cover one another's latencies where a lane would have
// more than four states.  4 x 4096 tokens x 2048 channels, bf16, us with the
// states in one part against two: 32 states 344 : 317, 64 states 935 : 530 (301
// and 522 with today's sum of y).
template <typename E> cudaError_t scan(const GdnSsmArgs &a, cudaStream_t s)
{
    if (a.d_state <= 16) return launch_fwd<E, 4, 1>(a, s);
    if (a.d_state <= 32) return launch_fwd<E, 4, 2>(a, s);
    if (a.d_state <= 64) return launch_fwd<E, 8, 2>(a, s);
    return launch_fwd<E, 16, 2>(a, s);
}

}  // namespace

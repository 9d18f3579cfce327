// Sums over a team of a norm, for the kernels that normalise rows.
#pragma once

#include <stdint.h>

namespace gdn_layer {

constexpr int kTeamWarps = 16;  // of the largest block

// Sums over the team, T lanes of a warp or the block, of R values at a time.  A
// block's warps meet in one of two buffers: by the time one is filled again, the
// barrier of the sum between has seen everybody through reading it.
template <int BLOCK, int R> struct TeamSum {
    float (*sh)[R][kTeamWarps];
    int turn;

    __device__ __forceinline__ void operator()(float (&v)[R], int T)
    {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            if (!BLOCK && o >= T) continue;
#pragma unroll
            for (int r = 0; r < R; ++r) v[r] += __shfl_xor_sync(0xffffffffu, v[r], o);
        }
        if constexpr (BLOCK != 0) {
            if ((threadIdx.x & 31) == 0)
#pragma unroll
                for (int r = 0; r < R; ++r) sh[turn][r][threadIdx.x >> 5] = v[r];
            __syncthreads();
#pragma unroll
            for (int r = 0; r < R; ++r) {
                v[r] = 0.f;
#pragma unroll
                for (int i = 0; i < BLOCK / 32; ++i) v[r] += sh[turn][r][i];
            }
            turn ^= 1;
        }
    }
};

}  // namespace gdn_layer

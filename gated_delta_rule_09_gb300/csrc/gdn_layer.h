// Internal interface of the operators around the recurrence: between their
// C-ABI front end (gdn_layer_api.cu) and the kernels, and what that front end
// uses of gdn_api.cu.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "gdn.h"

// The front end's bookkeeping (gdn_api.cu), for entry points in other files.
gdn_status_t gdn_fail(gdn_status_t st, const char *fmt, ...);  // sets the thread's message
gdn_status_t gdn_device_status_word(unsigned int **out);       // the GDN_DEV_* word's address
void gdn_begin_call();                                         // clears the message
void gdn_record_launch(int launches, int path);

struct GdnConvArgs {
    const void *x;               // rows of `channels`, stride ld_x, dtype
    const float *weight;         // [channels, width]
    const float *bias;           // [channels] or null
    const void *state_in;        // [pool, width - 1, channels] dtype, or null (zeros)
    const int32_t *slots;        // [N] pool entry per sequence, or null (n)
    void *y;                     // rows of `channels`, stride ld_y, dtype
    void *state_out;             // [pool, width - 1, channels] or null; may equal state_in
    int N, T, channels, width;   // T: tokens per sequence, or packed rows with cu_seqlens
    int64_t ld_x, ld_y;
    int pool;
    const int32_t *cu_seqlens;   // device [N + 1] or null
    int act;                     // GDN_ACT_*
    int dtype;                   // 0 = fp32, 1 = bf16
    unsigned int *status;
};

cudaError_t gdn_launch_conv_fwd(const GdnConvArgs &a, cudaStream_t s);
cudaError_t gdn_launch_conv_step(const GdnConvArgs &a, cudaStream_t s);

struct GdnSsmArgs {
    const void *x, *delta, *Bm, *Cm, *z;  // rows, dtype; z may be null
    const float *A;              // [channels, d_state]
    const float *D, *delta_bias; // [channels] or null
    const float *state_in;       // [pool, channels, d_state] or null (zeros)
    const int32_t *slots;        // [N] or null
    void *y;
    float *state_out;            // [pool, channels, d_state] or null; may equal state_in
    int N, T, channels, d_state, groups;
    int64_t ld_x, ld_delta, ld_b, ld_c, ld_z, ld_y;
    int pool;
    const int32_t *cu_seqlens;
    int softplus;
    int dtype;
    unsigned int *status;
    int segment;                 // tokens per piece; 0: one piece per sequence
    int64_t pieces;              // piece slots of the whole call, segment > 0
    float *piece_state;          // [piece slot, channels, d_state] workspace
    float *piece_delta;          // [piece slot, channels] sum of d over the piece
};

// Pieces a call is cut into: *segment tokens each (0: not cut), and the number
// of piece slots the workspace holds.  Never more slots than with one group.
void gdn_ssm_plan(int N, int T, int channels, int groups, bool packed, int asked, int *segment,
                  int64_t *piece_slots);
constexpr int kScanChannels = 64;  // of one group, per block of the scan
int gdn_ssm_sms();                 // multiprocessors of the current device
cudaError_t gdn_ssm_scan_bf16(const GdnSsmArgs &a, cudaStream_t s);
cudaError_t gdn_ssm_scan_f32(const GdnSsmArgs &a, cudaStream_t s);
cudaError_t gdn_launch_ssm_fwd(const GdnSsmArgs &a, cudaStream_t s, int *launches);
cudaError_t gdn_launch_ssm_step(const GdnSsmArgs &a, cudaStream_t s);

struct GdnNormArgs {
    const void *x, *gate;        // rows, dtype; gate may be null
    const float *weight, *bias;  // [channels] or null
    void *y;                     // may equal x or gate
    int64_t rows;
    int channels, groups;
    int64_t ld_x, ld_gate, ld_y;
    float eps;
    int rms, act, dtype;
};

cudaError_t gdn_launch_group_norm(const GdnNormArgs &a, cudaStream_t s);

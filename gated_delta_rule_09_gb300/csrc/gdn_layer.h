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

struct GdnLinattnArgs {
    const void *q, *k, *v;       // rows of groups x dk, groups x dk, heads x dv, dtype
    const float *log_decay;      // rows of `heads`, stride ld_decay (0: one row for every token)
    const float *state_in;       // [pool, heads, dv, dk] or null (zeros)
    const int32_t *slots;        // [N] or null
    void *o;                     // rows of heads x dv, dtype
    float *state_out;            // [pool, heads, dv, dk] or null; may equal state_in
    int N, T, heads, groups, dk, dv;
    int64_t ld_q, ld_k, ld_v, ld_decay, ld_o;
    int pool;
    const int32_t *cu_seqlens;
    float scale;
    int dtype;
    unsigned int *status;
    int segment;                 // tokens per piece; 0: one piece per sequence
    int64_t pieces;              // piece slots of the whole call, segment > 0
    float *piece_state;          // [piece slot, heads, dv, dk]: what a piece adds, then the state it starts from
    float *piece_decay;          // [piece slot, heads] root of the decay over the piece; 0: forgotten
};

// Pieces a call is cut into, as gdn_ssm_plan, by the kernel it runs on.
void gdn_linattn_plan(bool tensor_cores, int N, int T, int heads, int dk, int dv, bool packed, int asked, int *segment,
                      int64_t *piece_slots);
cudaError_t gdn_launch_linattn_fwd(const GdnLinattnArgs &a, cudaStream_t s, int *launches);
cudaError_t gdn_launch_linattn_step(const GdnLinattnArgs &a, cudaStream_t s);

// The tensor-core kernel over whole sequences or pieces (gdn_linattn_tc.cu), for calls it accepts.
bool gdn_linattn_tc_supported(const GdnLinattnArgs &a);
cudaError_t gdn_linattn_tc(const GdnLinattnArgs &a, bool states_only, cudaStream_t s);

struct GdnBlockNormArgs {
    const void *y, *gate;        // rows, dtype; gate may be null
    const void *residual;        // rows, dtype or fp32; may be null (zeros)
    const float *post_weight, *post_bias, *pre_weight, *pre_bias, *scale;  // [channels] or null
    void *residual_out, *h;      // rows; may equal residual (residual_out), y, gate (h); h null without a norm before
    int64_t rows;
    int channels;
    int64_t ld_y, ld_gate, ld_residual, ld_residual_out, ld_h;
    float residual_scale, eps;
    int rms, post, gate_act, dtype, residual_dtype;
};

// By the types of the rows and of the residual stream.
cudaError_t gdn_block_norm_bf16(const GdnBlockNormArgs &a, cudaStream_t s);
cudaError_t gdn_block_norm_bf16_f32(const GdnBlockNormArgs &a, cudaStream_t s);
cudaError_t gdn_block_norm_f32(const GdnBlockNormArgs &a, cudaStream_t s);

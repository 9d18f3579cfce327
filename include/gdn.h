/*
 * gdn.h — C ABI of libgdn: the chunkwise-parallel forward pass of the gated
 * delta rule on one NVIDIA GB300 (sm_103a).
 *
 * The operation (north-star recurrence; "从零开始的 GDN 推导", §"Gated Delta
 * Rule Chunk-wise Parallel 前向推导", recurrent form, written here with column
 * vectors so that the state S is d_v x d_k):
 *
 *     S_t = alpha_t * S_{t-1} (I - beta_t k_t k_t^T) + beta_t v_t k_t^T
 *     o_t = S_t q_t
 *
 * evaluated chunk by chunk with the WY / UT-transform form of the same page
 * (§"UT transform", §"S 的推导", §"O 的推导", §"总结"): inside a chunk of C
 * tokens everything is dense matrix algebra; only the d_v x d_k state is
 * carried from one chunk to the next ("RNN的复兴03：现代RNN的并行计算", §四:
 * parallel inside a chunk, dependent between chunks).  The result equals the
 * sequential recurrence up to floating-point rounding.
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 *  - Tensor pointers are DEVICE pointers (cudaMalloc / torch CUDA memory) on
 *    the current device, row-major and contiguous.  The caller allocates and
 *    owns all of them; the library keeps no reference after the call returns.
 *  - The library allocates no device memory in these calls.
 *  - Calls are asynchronous on `stream` (a cudaStream_t; NULL = the legacy
 *    default stream): they validate on the host, enqueue kernels and return.
 *  - On any status other than GDN_OK nothing was enqueued, and
 *    gdn_get_last_error() returns a message for the calling thread.
 *  - There is no CPU fallback: a call either runs its CUDA kernels or fails.
 */
#ifndef GDN_H_
#define GDN_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    GDN_OK = 0,
    GDN_ERR_INVALID_ARG = 1, /* null/misaligned pointer, bad size, overlap   */
    GDN_ERR_UNSUPPORTED = 2, /* shape or dtype outside the compiled set      */
    GDN_ERR_CUDA = 3,        /* a CUDA runtime call or a launch failed        */
    GDN_ERR_TIMEOUT = 4,     /* gdn_get_device_status: a bounded device wait
                                ran out (GDN_DEV_WAIT_TIMEOUT is among the
                                flags; the results of that call are invalid) */
    GDN_ERR_RANGE = 5        /* gdn_get_device_status: a tensor-core operand
                                left the fp16 range (GDN_DEV_F16_RANGE is
                                among the flags; results are invalid) */
} gdn_status_t;

typedef enum { GDN_F32 = 0, GDN_BF16 = 1 } gdn_dtype_t;

/* Activation of the layer operators (gdn_conv_*, gdn_group_norm). */
typedef enum { GDN_ACT_NONE = 0, GDN_ACT_SILU = 1 /* v / (1 + e^-v) */ } gdn_act_t;

/* Device-side status bits returned by gdn_get_device_status(). */
#define GDN_DEV_BAD_SEQLENS 0x1u /* a cu_seqlens span was negative or past T */
#define GDN_DEV_WAIT_TIMEOUT 0x2u /* a bounded pipeline wait gave up          */
#define GDN_DEV_F16_RANGE 0x4u    /* a tensor-core operand left the fp16 range  */
#define GDN_DEV_F16_PRECISION 0x8u /* a unit's state-chain operands all stayed
                                      below 2^-10: fp16 kept few bits of them   */
#define GDN_DEV_BAD_SLOT 0x10u   /* a state slot was past the end of its pool  */

/*
 * gdn_chunk_fwd — forward pass of the gated delta rule, chunkwise.
 *
 * Arguments (N = B, the number of sequences):
 *   q          [B, T, H, d_k]  dtype   queries
 *   k          [B, T, H, d_k]  dtype   keys (the method assumes nothing about
 *                                      their norm; unit norm is the usual input)
 *   v          [B, T, H, d_v]  dtype   values
 *   log_alpha  [B, T, H]       fp32    log of the decay gate alpha_t (<= 0 is
 *                                      the usual range; not required)
 *   beta       [B, T, H]       fp32    write strength beta_t (any real value;
 *                                      (0, 2) is the extended DeltaNet range)
 *   S0         [N, H, d_v, d_k] fp32   initial state per (sequence, head), or
 *                                      NULL for zeros
 *   o          [B, T, H, d_v]  dtype   output, o_t = S_t q_t (state after
 *                                      token t); must not overlap any input
 *   S_final    [N, H, d_v, d_k] fp32   state after each sequence's last token,
 *                                      or NULL if not wanted; may be exactly
 *                                      S0 (in-place carry), must not overlap
 *                                      anything else
 *   B, H, T    batch, heads, tokens per sequence
 *   d_k, d_v   key and value head dimensions
 *   C          chunk length: 16, 32 or 64
 *   cu_seqlens device int32 [N + 1] or NULL.  When given, the sequences are
 *              packed along the token axis: q/k/v/o are [1, T, H, *],
 *              log_alpha/beta are [1, T, H], B is the number of sequences N,
 *              sequence n spans tokens [cu_seqlens[n], cu_seqlens[n+1]), and
 *              T is the packed length.  Chunks never cross a sequence; each
 *              sequence starts from its own S0[n].  Spans that are negative or
 *              run past T are skipped on the device and raise
 *              GDN_DEV_BAD_SEQLENS (see gdn_get_device_status).  On the
 *              tensor-core path, up to 256 packed sequences are started
 *              longest first, whatever their order in the pack.
 *   dtype      GDN_F32 or GDN_BF16 (q, k, v and o share it).  fp32 runs in
 *              fp32 on CUDA cores.  bf16 runs on the tensor cores with fp16
 *              operands (11-bit significand) and fp32 accumulation and
 *              state.  A bf16 input converts to fp16 exactly when its
 *              magnitude lies in [2^-14, 65504]; below 2^-14 fp16 keeps fewer
 *              bits (subnormals), above 65504 it overflows.  An operand that
 *              leaves the fp16 range raises GDN_DEV_F16_RANGE; a (sequence,
 *              head) whose state chain ran entirely below 2^-10 in magnitude
 *              (e.g. v and S0 of order 1e-6) raises GDN_DEV_F16_PRECISION:
 *              the method is linear in v and S0, so scaling both up (and the
 *              results back down) avoids it
 *   stream     cudaStream_t to enqueue on
 *
 * Alignment: q, k, v, o must be aligned to 16 bytes; log_alpha, beta, S0 and
 * S_final to 4 bytes (16 bytes lets the fastest path run).
 * Supported shapes: d_k in [1, 128], d_v >= 1, C in {16, 32, 64}.  The
 * tcgen05 tensor-core kernel serves bf16 with C = 64 and d_k, d_v multiples
 * of 8 (tiles zero-padded to 128); every other supported shape runs on the
 * fp32 CUDA-core kernel (gdn_last_launch_count reports which ran).  Both are CUDA kernels
 * of this library.
 *
 * Returns GDN_OK once the work is enqueued, or an error status (nothing
 * enqueued).  Errors detected by the kernels are reported through
 * gdn_get_device_status().
 */
gdn_status_t gdn_chunk_fwd(const void *q, const void *k, const void *v,
                           const float *log_alpha, const float *beta,
                           const float *S0, void *o, float *S_final,
                           int B, int H, int T, int d_k, int d_v, int C,
                           const int32_t *cu_seqlens, gdn_dtype_t dtype,
                           void *stream);

/*
 * gdn_chunk_fwd_eta — gdn_chunk_fwd with a write strength eta_t separate
 * from the erase strength beta_t ("RNN的复兴03：现代RNN的并行计算", §一, the
 * general delta-rule recurrence):
 *
 *     S_t = alpha_t S_{t-1} (I - beta_t k_t k_t^T) + eta_t v_t k_t^T
 *
 * In the chunk form only U changes, U = T diag(eta) V; A and W keep beta.
 * With eta = beta this is gdn_chunk_fwd.  eta is fp32 [B, T, H] (the layout
 * of beta), non-NULL when there is work, 4-byte aligned and not overlapping
 * o or S_final.  Every other argument, and every rule, is gdn_chunk_fwd's.
 */
gdn_status_t gdn_chunk_fwd_eta(const void *q, const void *k, const void *v,
                               const float *log_alpha, const float *beta, const float *eta,
                               const float *S0, void *o, float *S_final,
                               int B, int H, int T, int d_k, int d_v, int C,
                               const int32_t *cu_seqlens, gdn_dtype_t dtype,
                               void *stream);

/*
 * gdn_chunk_fwd_scan — gdn_chunk_fwd for few, long sequences: each sequence
 * is cut into `segments` pieces at chunk boundaries that run in parallel.
 * A segment's final state is an affine function of its initial state,
 * S_end = S_start M + B ("从零开始的 GDN 推导", §"S 的推导": every chunk step is
 * affine in S), and affine maps compose associatively ("Параллельность
 * RNN?", §"Уровень 2: рекуррентность линейна, и потому ассоциативна"): a
 * first pass computes every segment's M (d_k x d_k) and B (d_v x d_k) on the
 * tensor cores, a scan chains them into each segment's initial state, and a
 * second pass runs every segment's forward pass from it.  The result equals
 * gdn_chunk_fwd up to rounding; the work is about 2 + d_k / d_v times the
 * forward pass, spread over B * H * segments units instead of B * H.
 *
 * Arguments as gdn_chunk_fwd, packed sequences (cu_seqlens) included, plus
 *   segments   pieces per sequence; <= 0 lets the library choose from the
 *              device's SM count and the (average) sequence length (1 means
 *              the plain pass).  Without cu_seqlens it is capped at
 *              ceil(T / C) and no piece is empty.  With cu_seqlens every
 *              sequence is cut into the same number of pieces of
 *              ceil(chunks_n / segments) chunks, capped at the chunks of
 *              the whole pack; a sequence shorter than that many chunks
 *              leaves its last pieces empty.  A span that is negative or
 *              runs past T raises GDN_DEV_BAD_SEQLENS; that sequence's
 *              outputs are not written and its S_final is its S0.
 *   workspace  device scratch of at least
 *              gdn_chunk_fwd_scan_workspace_size(B, H, T, d_k, d_v, C,
 *              cu_seqlens, segments) bytes (only whether cu_seqlens is NULL
 *              matters there), 256-byte aligned, caller-owned, not
 *              overlapping any argument; NULL is allowed when that size is 0
 *              or one segment is chosen.  Calls that share a workspace must
 *              not overlap in time.
 * Supported: bf16, C = 64, d_k <= 128 and d_k, d_v multiples of 8 (the
 * tensor-core kernel); anything else returns GDN_ERR_UNSUPPORTED.  Four
 * kernels are enqueued (gdn_last_launch_count reports path 3) plus one
 * device-to-device copy per sequence for S_final.
 */
size_t gdn_chunk_fwd_scan_workspace_size(int B, int H, int T, int d_k, int d_v, int C,
                                         const int32_t *cu_seqlens, int segments);

gdn_status_t gdn_chunk_fwd_scan(const void *q, const void *k, const void *v,
                                const float *log_alpha, const float *beta,
                                const float *S0, void *o, float *S_final,
                                int B, int H, int T, int d_k, int d_v, int C,
                                const int32_t *cu_seqlens, gdn_dtype_t dtype, int segments,
                                void *workspace, size_t workspace_bytes, void *stream);

/*
 * gdn_chunk_fwd_scan_noalloc — gdn_chunk_fwd_scan for callers that cannot
 * allocate device memory: the scratch is a fixed 32 MiB array that is part of
 * the library's device image (reserved when the library's module is loaded
 * on a device), so the call allocates nothing.  The pages have no
 * counterpart: this is a deployment convenience around the same scan.
 *
 * Arguments and results as gdn_chunk_fwd_scan without the workspace.  A
 * problem whose scratch (gdn_chunk_fwd_scan_workspace_size with the same
 * arguments) exceeds 32 MiB is rejected with GDN_ERR_UNSUPPORTED and a
 * message; fewer segments need less.  Nothing in the scratch has to start
 * at zero (each call writes every byte it reads).  The scratch is shared by
 * every call on a device: calls that overlap in time (other streams, other
 * threads) race and must be serialised by the caller.
 */
gdn_status_t gdn_chunk_fwd_scan_noalloc(const void *q, const void *k, const void *v,
                                        const float *log_alpha, const float *beta,
                                        const float *S0, void *o, float *S_final,
                                        int B, int H, int T, int d_k, int d_v, int C,
                                        const int32_t *cu_seqlens, gdn_dtype_t dtype,
                                        int segments, void *stream);

/*
 * gdn_decode_step — the same recurrence evaluated token by token, for decoding
 * ("从零开始的 GDN 推导", recurrent form of the gated delta rule;
 * "RNN的复兴03：现代RNN的并行计算", §一, delta-rule update), batched over
 * (sequence, head).  Per token, with r = S k:
 *
 *     S <- alpha S + beta (v - alpha r) k^T      o = S q
 *
 * which is the spec update alpha S (I - beta k k^T) + beta v k^T
 * rearranged.  T is the number of tokens each sequence advances in this call
 * (1 for one decoding step); the state stays on chip between them.  The
 * state written by gdn_chunk_fwd (S_final) is the state this call reads, so a
 * prefill with gdn_chunk_fwd followed by decode steps reproduces the
 * recurrence over the whole sequence.
 *
 * Arguments:
 *   q, k       [N, T, H, d_k]  dtype   queries, keys
 *   v          [N, T, H, d_v]  dtype   values
 *   log_alpha  [N, T, H]       fp32    log of the decay gate
 *   beta       [N, T, H]       fp32    write strength (any real value)
 *   S_in       [N, H, d_v, d_k] fp32   state before the first token, or NULL
 *                                      for zeros
 *   o          [N, T, H, d_v]  dtype   outputs; must not overlap anything
 *   S_out      [N, H, d_v, d_k] fp32   state after the last token (required);
 *                                      may be exactly S_in (in-place update),
 *                                      must not overlap anything else.  With
 *                                      T = 0 it receives S_in (or zeros).
 *   N, H, T, d_k, d_v  sizes; d_k in [1, 128], d_v >= 1
 *   dtype      GDN_F32 or GDN_BF16 (q, k, v and o share it); arithmetic is
 *              fp32 on CUDA cores either way
 *   stream     cudaStream_t to enqueue on
 *
 * Alignment: q, k, v, o 16 bytes; log_alpha, beta, S_in, S_out 4 bytes
 * (16 bytes and d_k a multiple of 4 select the vectorised kernel).
 * Returns GDN_OK once the work is enqueued (one kernel; gdn_last_launch_count
 * reports path 2), or an error status with nothing enqueued.
 */
gdn_status_t gdn_decode_step(const void *q, const void *k, const void *v,
                             const float *log_alpha, const float *beta,
                             const float *S_in, void *o, float *S_out,
                             int N, int H, int T, int d_k, int d_v,
                             gdn_dtype_t dtype, void *stream);

/*
 * gdn_ut_inverse — batched UT transform inverse T = (I + A)^{-1} of the
 * chunk form ("从零开始的 GDN 推导", §"UT transform") for strictly lower C x C
 * matrices A, by one of two methods, for comparing them:
 *   method 0  blocked forward substitution on CUDA cores in fp32 (the
 *             routine the tensor-core chunk kernel runs per chunk;
 *             "RNN的复兴03：现代RNN的并行计算", §2.3.1);
 *   method 1  the nilpotent doubling product on the tensor cores:
 *             (I + A)^{-1} = (I - A)(I + A^2)(I + A^4)...(I + A^32) (the
 *             finite Neumann series of the same page, §2.3.2), powers in
 *             fp16 operands, products accumulated in fp32.
 * A  [count, C, C] fp32 row-major; entries on and above the diagonal are
 *    ignored.  T [count, C, C] fp32: unit diagonal, zeros above; must not
 *    overlap A.  C in {16, 32, 64}.  One kernel; gdn_last_launch_count
 *    reports path 4 + method.  A timed-out wait of method 1 raises
 *    GDN_DEV_WAIT_TIMEOUT.
 */
gdn_status_t gdn_ut_inverse(const float *A, float *T, int count, int C, int method, void *stream);

/*
 * ---------------------------------------------------------------------------
 * The layer around the recurrence: short causal convolution, selective state
 * space scan, group norm.  Rules these entry points share, beside the
 * conventions at the top of this file:
 *
 *  - Rows.  x, y, z and the like are matrices of token rows with unit stride
 *    along the channels and a row stride ld_* (in elements, at least the row's
 *    own width), so that each may be a slice of a projection's wider output.
 *    Prompts [B, T, *] are B * T rows one ld apart.  Outputs must not overlap
 *    inputs; two slices of the same rows (equal ld, separate columns) do not
 *    overlap.
 *  - Types.  x, y and what is drawn from the same projection share `dtype`;
 *    parameters (weight, bias, A, D, delta_bias) are fp32, arithmetic is fp32,
 *    the output is rounded once.  Alignment: that of the element type; 16
 *    bytes with row strides that are a multiple of 16 bytes selects the
 *    vectorised kernels.
 *  - Packed prompts (cu_seqlens, device int32 [B + 1]) follow gdn_chunk_fwd:
 *    B sequences along one token axis of T rows.  A span that is negative or
 *    leaves [0, T] is skipped and raises GDN_DEV_BAD_SEQLENS.  Where offsets go
 *    back so far that two other spans share rows, y of those sequences and
 *    their states are undefined (the bit is raised).  B, N and T are at most
 *    2^31 - 2^16.
 *  - States live in a pool of `pool` entries: sequence n owns entry n, or
 *    entry slots[n] when `slots` (device int32, one per sequence) is given,
 *    so a serving loop keeps one pool for prompts and steps.  state_in may be
 *    NULL (zeros); state_out NULL (prompts only) drops the final state.
 *    state_out may be exactly state_in (in place).  A negative slot marks a
 *    sequence that keeps no state: it starts from zeros and writes none (the
 *    padding rows of a fixed-size batch).  A slot >= pool is treated the same
 *    way and raises GDN_DEV_BAD_SLOT.  Two sequences must not share a slot.
 *    A sequence without tokens hands its state on unchanged.  Without states
 *    (both pointers NULL) the slots are not looked at.
 */

/*
 * gdn_conv_fwd — short causal depthwise convolution over prompts:
 *
 *     y[t, c] = act(bias[c] + sum_j weight[c, j] x[t - (width - 1) + j, c])
 *
 * with the inputs before a sequence's first token taken from its state (the
 * last width - 1 inputs, oldest first) or zero.
 *   x, y        [B, T, channels] dtype, row strides ld_x, ld_y
 *   weight      [channels, width] fp32; bias [channels] fp32 or NULL
 *   state_in, state_out  [pool, width - 1, channels] dtype; NULL allowed
 *   width       1 to 8
 * One kernel; gdn_last_launch_count reports path 6.
 */
gdn_status_t gdn_conv_fwd(const void *x, const float *weight, const float *bias,
                          const void *state_in, const int32_t *slots, void *y, void *state_out,
                          int B, int T, int channels, int width, int64_t ld_x, int64_t ld_y,
                          int pool, const int32_t *cu_seqlens, gdn_act_t act, gdn_dtype_t dtype,
                          void *stream);

/*
 * gdn_conv_step — the same for one new token of each of N sequences:
 * x, y [N, channels]; the state (required in state_out, NULL state_in =
 * zeros) moves on by one input.  One kernel, path 6.
 */
gdn_status_t gdn_conv_step(const void *x, const float *weight, const float *bias,
                           const void *state_in, const int32_t *slots, void *y, void *state_out,
                           int N, int channels, int width, int64_t ld_x, int64_t ld_y, int pool,
                           gdn_act_t act, gdn_dtype_t dtype, void *stream);

/*
 * gdn_ssm_fwd — selective state space scan over prompts.  Channel c of group
 * g = c / (channels / groups) carries d_state fp32 states; per token t
 *
 *     d      = delta[t, c] + delta_bias[c]       (softplus of it if asked)
 *     h[s]   = exp(d A[c, s]) h[s] + d B[t, g, s] x[t, c]
 *     y[t,c] = (sum_s C[t, g, s] h[s] + D[c] x[t, c]) * silu(z[t, c])
 *
 * softplus(v) = log(1 + e^v); without z the last factor is one, without D
 * the skip term is zero.
 *   x, delta, z, y  [B, T, channels] dtype, row strides ld_x, ld_delta, ld_z,
 *                   ld_y; z NULL allowed
 *   A               [channels, d_state] fp32 (negative for a decaying state;
 *                   -inf for one that forgets at once, which d = 0 leaves as
 *                   it is)
 *   Bm, Cm          [B, T, groups, d_state] dtype, row strides ld_b, ld_c
 *   D, delta_bias   [channels] fp32 or NULL
 *   state_in, state_out  [pool, channels, d_state] fp32; NULL allowed
 *   d_state 1 to 128; channels a multiple of groups; groups x d_state below 2^31
 *   segment         tokens per piece: long sequences are cut into pieces that
 *                   run in parallel (each piece's decay is exp(A sum d), so
 *                   the pieces chain exactly up to rounding); <= 0 lets the
 *                   library choose (possibly one piece), else rounded up to a
 *                   multiple of 64.  Packed lengths are on the device, so the
 *                   library reckons with a longest of twice the mean: a pack
 *                   with one far longer sequence should ask for pieces (one of
 *                   130 000 tokens and 31 of 20, 1024 channels: 6.4 ms whole,
 *                   1.1 ms in pieces of 2048)
 *   workspace       gdn_ssm_fwd_workspace_size(...) bytes, 16-byte aligned,
 *                   not overlapping any argument, not shared by calls that
 *                   overlap in time; NULL allowed when that size is 0
 * One kernel, or two when sequences are cut; path 7.
 */
size_t gdn_ssm_fwd_workspace_size(int B, int T, int channels, int d_state,
                                  const int32_t *cu_seqlens, int segment);

gdn_status_t gdn_ssm_fwd(const void *x, const void *delta, const float *A, const void *Bm,
                         const void *Cm, const float *D, const void *z, const float *delta_bias,
                         const float *state_in, const int32_t *slots, void *y, float *state_out,
                         int B, int T, int channels, int d_state, int groups, int64_t ld_x,
                         int64_t ld_delta, int64_t ld_b, int64_t ld_c, int64_t ld_z, int64_t ld_y,
                         int pool, const int32_t *cu_seqlens, int delta_softplus,
                         gdn_dtype_t dtype, int segment, void *workspace, size_t workspace_bytes,
                         void *stream);

/*
 * gdn_ssm_step — the same recurrence for one new token of each of N
 * sequences: x, delta, z, y [N, channels], Bm, Cm [N, groups, d_state].
 * state_out is required; state_in NULL = zeros.  One kernel, path 7.
 */
gdn_status_t gdn_ssm_step(const void *x, const void *delta, const float *A, const void *Bm,
                          const void *Cm, const float *D, const void *z, const float *delta_bias,
                          const float *state_in, const int32_t *slots, void *y, float *state_out,
                          int N, int channels, int d_state, int groups, int64_t ld_x,
                          int64_t ld_delta, int64_t ld_b, int64_t ld_c, int64_t ld_z, int64_t ld_y,
                          int pool, int delta_softplus, gdn_dtype_t dtype, void *stream);

/*
 * gdn_group_norm — group norm of token rows, channels last, the norm of the
 * heads' outputs (a group is a head): the channels of a row are cut into
 * `groups` equal runs, each normalised by its own statistics,
 *
 *     u = (x - mean) / sqrt(var + eps)     (rms != 0: x / sqrt(mean x^2 + eps))
 *     y = act(u * weight[c] + bias[c]) * silu(gate)
 *
 *   x, gate, y  [rows, channels] dtype, row strides ld_x, ld_gate, ld_y; gate
 *               NULL allowed (factor one); y may be exactly x or gate with
 *               the same stride (in place)
 *   weight, bias  [channels] fp32 or NULL; eps >= 0
 * Statistics are per token: tokens do not see one another.  One kernel, path 8.
 */
gdn_status_t gdn_group_norm(const void *x, const void *gate, const float *weight,
                            const float *bias, void *y, int64_t rows, int channels, int groups,
                            int64_t ld_x, int64_t ld_gate, int64_t ld_y, float eps, int rms,
                            gdn_act_t act, gdn_dtype_t dtype, void *stream);

/*
 * gdn_get_device_status — synchronise `stream`, then read and clear the
 * device-side status bits (GDN_DEV_*) raised by kernels of this library on the
 * current device since the last read.  *flags receives the bits (0 = clean).
 * Returns GDN_ERR_TIMEOUT when GDN_DEV_WAIT_TIMEOUT is among them (*flags is
 * still written): a kernel gave up on a bounded wait, finished without
 * completing its work, drained what it had in flight and freed its tensor
 * memory, so the device stays usable but that work's outputs are invalid.
 * Else GDN_ERR_RANGE when GDN_DEV_F16_RANGE is among them: an operand
 * overflowed fp16, so the outputs it fed are wrong.  The other bits (a bad
 * packed span: that sequence was skipped; fp16 precision: results are valid
 * but carry fewer bits; a bad slot: that sequence ran without a state) come
 * back with GDN_OK.
 * Returns GDN_ERR_CUDA if synchronising or reading fails.
 */
gdn_status_t gdn_get_device_status(void *stream, unsigned int *flags);

/* Message for the last non-OK status returned on the calling thread. */
const char *gdn_get_last_error(void);

/* Library version as MAJOR * 10000 + MINOR * 100 + PATCH. */
int gdn_version(void);

/*
 * gdn_last_launch_count — number of kernels the last successful gdn_chunk_fwd
 * gdn_chunk_fwd_scan, gdn_decode_step or layer operator on the calling thread
 * enqueued, and
 * in *path which kernel family ran (0 = fp32 CUDA-core chunk kernel,
 * 1 = tcgen05 tensor-core chunk kernel, 2 = recurrent decode kernel,
 * 3 = chunk-level scan over segments, 4 / 5 = UT inverse by forward
 * substitution / on the tensor cores, 6 = short convolution, 7 = state space
 * scan or step, 8 = group norm).  For
 * accounting in benchmarks; no device work.
 */
int gdn_last_launch_count(int *path);

#ifdef __cplusplus
}
#endif

#endif /* GDN_H_ */

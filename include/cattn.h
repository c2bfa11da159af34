/*
 * cattn.h -- C ABI of the mixer operators that follow the short convolution of cconv.h on
 * GB300 (sm_103a): the per-head norm of queries and keys with the position rotation, and
 * linear attention with a decay for each token and head, for prompts, for training and for
 * single tokens.  Library: libcattn.so.
 *
 * What the calls compute (heads: Hk of queries and keys, Hv = r * Hk of values; value head h
 * reads query and key head h / r):
 *
 *   norm      m = mean(x^2) (CATTN_NORM_RMS) or sum(x^2) (CATTN_NORM_L2) over the K channels
 *             u = w * x / sqrt(m + eps)
 *             y = u with the pairs (a, b) of its first R channels turned by their angle:
 *                 (a cos - b sin, b cos + a sin)
 *   linear    S_t = exp(g_t) S_{t-1} + k_t v_t^T          S: [K, V] for each value head
 *             o_t = scale * q_t^T S_t
 *
 * Conventions shared by every call (those of cconv.h):
 *   - Queries, keys, values, outputs and their gradients are bf16; g, the states, their
 *     gradients and the rotation tables are fp32; norm weights and their gradients share one
 *     dtype, `wdt` (bf16 or fp32).
 *   - All pointers are DEVICE pointers owned by the caller.  The library allocates nothing and
 *     keeps nothing from one call for the next.
 *   - All work is enqueued on `stream` with no host synchronisation and may be captured in a
 *     CUDA graph.  Argument errors are found on the host before anything is enqueued: the call
 *     returns a negative cconv_status and launches nothing.
 *   - Strides are in elements.  Element (t, h, c) of a [total, H, C] activation lies at
 *     base + t * st + h * sh + c; st and sh are positive multiples of 8 (ignored where the
 *     dimension they step over has extent 1) and every base is 16-byte aligned, so the
 *     convolution's [total, D] outputs are read in place.  Inputs may overlap one another;
 *     outputs are contiguous and overlap nothing.
 *   - Sequences are packed along the rows as in cconv_fwd_varlen: cu_seqlens is int32[nseq+1]
 *     in device memory, cu[0] = 0, non-decreasing, cu[nseq] = total; empty sequences are
 *     allowed.  The host never reads it.  An ill-formed vector gives unspecified results,
 *     every access stays inside the buffers, and cattn_device_fault() reports bit 4.
 *   - A workspace is the call's until its work on `stream` is done.
 *   - Precision: sums, norms, gates and states are fp32.  Rounded to bf16 are the results, once,
 *     and inside the linear attention's matrix products the decayed scores (in calls of at most
 *     64 rows they keep 16 bits) and, in the forward, the states as the queries read them: errors
 *     of 2.3e-3 in the 2-norm, of which the store alone makes 1.7e-3.  States, their gradients and
 *     dg are as exact as sums in fp32.
 *   - Results are bit-identical from run to run for the same inputs and device.
 */
#ifndef CATTN_H
#define CATTN_H

#include "cconv.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  CATTN_NORM_RMS = 0,
  CATTN_NORM_L2 = 1
} cattn_norm;

/*
 * cattn_qknorm_fwd -- norm and rotation of queries and keys, one launch for both.
 *
 *   q, k      [total, Hq, K], [total, Hk, K] bf16, strided.  total may be 0.
 *   wq, wk    [K] weights in wdt, or NULL (no weight).
 *   cos, sin  [P, R/2] fp32 contiguous tables, 32-byte aligned; not read when R == 0.
 *   R         rotated channels: 0 <= R <= K, a multiple of 16.
 *   interleaved  0: channel c < R/2 pairs with c + R/2; 1: channel 2c pairs with 2c + 1.
 *             Pair c turns by table column c.
 *   positions int32[total] table row of each token, or NULL (token t uses row t; total <= P).
 *             A position outside [0, P) uses the nearest row and cattn_device_fault() reports
 *             bit 8.
 *   yq, yk    [total, Hq, K], [total, Hk, K] bf16 contiguous outputs, 16-byte aligned.
 *   eps >= 0.  K % 8 == 0, 8 <= K <= 256, 1 <= Hq, Hk <= 65535, total < 2^31 - 16.
 */
CCONV_API int cattn_qknorm_fwd(const void* q, int64_t sqt, int64_t sqh, const void* k,
                               int64_t skt, int64_t skh, int64_t total, int64_t Hq, int64_t Hk,
                               int64_t K, const void* wq, const void* wk, cconv_dtype wdt,
                               cattn_norm mode, float eps, const float* cos, const float* sin,
                               int64_t P, int64_t R, int interleaved, const int32_t* positions,
                               void* yq, void* yk, cconv_stream_t stream);

/* Workspace cattn_qknorm_bwd needs on the current device (16-byte aligned). */
CCONV_API int cattn_qknorm_bwd_workspace_bytes(int64_t total, int64_t Hq, int64_t Hk, int64_t K,
                                               size_t* bytes);

/*
 * cattn_qknorm_bwd -- its gradient; the norm is recomputed from q and k.
 *
 *   dyq, dyk  [total, Hq, K], [total, Hk, K] bf16, strided.
 *   dq, dk    contiguous bf16 outputs, 16-byte aligned.
 *   dwq, dwk  [K] outputs in wdt, or NULL to skip them (the sums run over tokens and heads in
 *             a fixed order, in fp32).
 */
CCONV_API int cattn_qknorm_bwd(const void* q, int64_t sqt, int64_t sqh, const void* k,
                               int64_t skt, int64_t skh, const void* dyq, int64_t syqt,
                               int64_t syqh, const void* dyk, int64_t sykt, int64_t sykh,
                               int64_t total, int64_t Hq, int64_t Hk, int64_t K, const void* wq,
                               const void* wk, cconv_dtype wdt, cattn_norm mode, float eps,
                               const float* cos, const float* sin, int64_t P, int64_t R,
                               int interleaved, const int32_t* positions, void* dq, void* dk,
                               void* dwq, void* dwk, void* workspace, size_t workspace_bytes,
                               cconv_stream_t stream);

/* Workspace cattn_linear_fwd / cattn_linear_bwd need on the current device (16-byte aligned). */
CCONV_API int cattn_linear_fwd_workspace_bytes(int64_t total, int64_t nseq, int64_t Hk,
                                               int64_t Hv, int64_t K, int64_t V, size_t* bytes);
CCONV_API int cattn_linear_bwd_workspace_bytes(int64_t total, int64_t nseq, int64_t Hk,
                                               int64_t Hv, int64_t K, int64_t V, size_t* bytes);

/*
 * cattn_linear_fwd -- linear attention with decay over packed sequences.
 *
 *   q, k      [total, Hk, K] bf16, strided;  v  [total, Hv, V] bf16, strided.
 *   g         [total, Hv] fp32 natural logarithms of the decays, at g + t * sgt + h * sgh with
 *             any strides >= 0 (sgt = 0: one decay per head).  Values below -128 count as -128
 *             (exp(-128) is zero in fp32), so -inf forgets everything before the token.  Decays
 *             are at most 1 (g <= 0); what has decayed below 2^-127 counts as forgotten, also
 *             if later values of g are positive.
 *   scale     factor of the outputs.
 *   initial_state  [S, Hv, K, V] fp32 contiguous, 32-byte aligned (as the other states), or NULL
 *             (zeros).
 *   final_state    [S, Hv, K, V] fp32 output, or NULL.  May be the same array as initial_state.
 *   state_indices  int32[nseq] in device memory, or NULL: sequence i's state lives in slot
 *             state_indices[i] (else slot i, and S >= nseq).  Indices are checked on the device
 *             as cconv_fwd_varlen checks them: on an invalid vector (negative, >= S, repeated)
 *             no state is written, status_dev gets [CCONV_ERR_INDEX, offence bits], and o is
 *             computed with zero initial states for the unusable slots; otherwise status_dev
 *             gets [CCONV_OK, 0].  1 <= S <= CCONV_UPDATE_MAX_SLOTS with indices.
 *   status_dev  int32[2] in device memory (only with state_indices; then required).
 *   o         [total, Hv, V] bf16 contiguous output, 16-byte aligned.
 *   K % 8 == 0, 8 <= K <= 128;  V % 8 == 0, 8 <= V <= 256;  Hk >= 1, Hv a multiple of Hk;
 *   nseq >= 1, 0 <= total < 2^31 - 16.  A final state of an empty sequence is its initial one.
 *   Non-finite values of one sequence never reach another sequence's results; inside a
 *   sequence they may reach the outputs of up to 127 tokens before theirs.
 */
CCONV_API int cattn_linear_fwd(const void* q, int64_t sqt, int64_t sqh, const void* k,
                               int64_t skt, int64_t skh, const void* v, int64_t svt, int64_t svh,
                               const float* g, int64_t sgt, int64_t sgh, int64_t total,
                               int64_t Hk, int64_t Hv, int64_t K, int64_t V,
                               const int32_t* cu_seqlens, int64_t nseq, float scale,
                               const float* initial_state, float* final_state,
                               const int32_t* state_indices, int64_t S, int32_t* status_dev,
                               void* o, void* workspace, size_t workspace_bytes,
                               cconv_stream_t stream);

/*
 * cattn_linear_bwd -- its gradient: dq, dk, dv, dg and the gradient of the initial states.
 * The states are recomputed.  The final states count as constants (no gradient flows in).
 *
 *   do_       [total, Hv, V] bf16, strided.
 *   initial_state, state_indices, S, status_dev: as the forward read them.  A negative or
 *             out-of-range slot reads as zeros; repeated slots are read as they are.
 *   dq, dk    [total, Hk, K], dv [total, Hv, V] bf16; dg [total, Hv] fp32; contiguous outputs,
 *             16-byte aligned.
 *   d_initial_state  [nseq, Hv, K, V] fp32 output (one per sequence, also with indices), or NULL.
 */
CCONV_API int cattn_linear_bwd(const void* q, int64_t sqt, int64_t sqh, const void* k,
                               int64_t skt, int64_t skh, const void* v, int64_t svt, int64_t svh,
                               const float* g, int64_t sgt, int64_t sgh, const void* do_,
                               int64_t sot, int64_t soh, int64_t total, int64_t Hk, int64_t Hv,
                               int64_t K, int64_t V, const int32_t* cu_seqlens, int64_t nseq,
                               float scale, const float* initial_state,
                               const int32_t* state_indices, int64_t S, int32_t* status_dev,
                               void* dq, void* dk, void* dv, float* dg, float* d_initial_state,
                               void* workspace, size_t workspace_bytes, cconv_stream_t stream);

/*
 * cattn_linear_update -- one token for each of N sequences, on a pooled state.
 *
 *   q, k      [N, Hk, K], v [N, Hv, V] bf16, strided; g [N, Hv] fp32, strided.
 *   state     [S, Hv, K, V] fp32 contiguous pool, 16-byte aligned, updated in place.
 *   state_indices, pad_rows, status_dev: as cconv_update_ex: int32[N] slots or NULL (row i uses
 *             slot i; needs S >= N); with pad_rows, -1 marks a padding row, which reads and
 *             writes no state and whose o row is not written; on an invalid vector NOTHING but
 *             status_dev is written.
 *   o         [N, Hv, V] bf16 contiguous output, 16-byte aligned.
 *   The limits on Hk, Hv, K, V and on S are cattn_linear_fwd's; 1 <= N < 2^31 - 16.
 */
CCONV_API int cattn_linear_update(const void* q, int64_t sqt, int64_t sqh, const void* k,
                                  int64_t skt, int64_t skh, const void* v, int64_t svt,
                                  int64_t svh, const float* g, int64_t sgt, int64_t sgh,
                                  int64_t N, int64_t Hk, int64_t Hv, int64_t K, int64_t V,
                                  float scale, float* state, int64_t S,
                                  const int32_t* state_indices, int pad_rows, void* o,
                                  int32_t* status_dev, cconv_stream_t stream);

/* Launch descriptions of this library's calls; as cconv_describe_begin / cconv_describe_end. */
CCONV_API int cattn_describe_begin(void);
CCONV_API int cattn_describe_end(cconv_kernel_desc* out, int max, int* count);

/*
 * cattn_device_fault -- reads (and clears) this library's device fault word on the current
 * device after synchronising it: 0, or an OR of 1 = a linear-attention kernel gave up a
 * bounded wait (its outputs are unspecified), 4 = an ill-formed cu_seqlens, 8 = a position
 * outside its table.  Returns CCONV_OK or CCONV_ERR_CUDA.
 */
CCONV_API int cattn_device_fault(int32_t* fault);

#ifdef __cplusplus
}
#endif

#endif /* CATTN_H */

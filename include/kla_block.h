/*
 * kla_block.h -- C ABI of what a block around the recurrences of kla.h and kla_layer.h needs on
 * NVIDIA GB300 (sm_103a): the gated scan (a recurrence with a gate and a state per channel: prompts,
 * single tokens, gradients), rotary positions of queries and keys, the norms after and before a block
 * with its gate and its residual (forward, gradients), and the verification of drafted tokens.
 *
 * The conventions of kla.h hold: device pointers, caller-owned buffers, calls asynchronous on
 * `stream` (whose device has to be the current one), argument errors found on the host before
 * anything is launched (KLA_ERR_INVALID_ARG / KLA_ERR_UNSUPPORTED, nothing written), bounded device
 * waits reported by kla_device_status.
 * Outputs and workspaces must not overlap each other or any input unless said otherwise; a workspace
 * serves one call at a time, whatever stream it runs on.
 */
#ifndef KLA_BLOCK_H
#define KLA_BLOCK_H

#include <stddef.h>
#include <stdint.h>

#include "kla.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---------------------------------------------------------------------------------- gated scan
 * Equal calls give equal bits.
 *
 * For every sequence b and channel c, a state h that starts as h0 (zero where NULL):
 *
 *     KLA_SCAN_SIGMOID   h_t = a_t h_{t-1} + (1 - a_t) x_t,   a_t = 1 / (1 + exp(-gate_t))
 *     KLA_SCAN_LOG       h_t = a_t h_{t-1} + x_t,             a_t = exp(gate_t)
 *
 * A gate is at most 0 in KLA_SCAN_LOG, as a decay's is. Larger ones are taken as they are as long as fp32 holds the
 * products of neighbouring a_t, of 256 tokens at most; where one that is formed passes that range, states may be NaN that
 * are not, and kla_device_status reports KLA_ERR_INVALID_ARG, of this call as of kla_gated_scan_bwd (and of gates that are
 * NaN). Which products are formed is not said: what is not reported is as the definition has it.
 *
 * y_t = h_t, for t = 0 .. n_b - 1, where n_b = lengths[b] (T when lengths is NULL). Tokens
 * t >= n_b are masked: whatever x and gate hold there (NaN included) they leave the state as it is,
 * and y_t = 0. A gate of -inf forgets the state (a_t = 0), one of +inf keeps it in KLA_SCAN_SIGMOID (to
 * 2^-100 of x). A channel whose state is infinite or NaN stays one or the other from there on, whatever
 * its gates, and which of the two is not said; what is less than 2^-126 of a state may count as nothing.
 *
 *   x, gate  [B, T, C] dtype, last axis contiguous. `strides` gives the element strides of the batch
 *            and token axes of x, then of gate (4 values, none negative); NULL means contiguous
 *   lengths  int32 [B] or NULL; values are taken into [0, T]
 *   h0       fp32 [B, C] or NULL (zeros)
 *   y        [B, T, C] dtype, contiguous, written (rounded once from the fp32 state)
 *   h_T      fp32 [B, C] or NULL: the state after the last valid token; may be h0 itself
 *   states   fp32 [B, ceil(T / KLA_SCAN_SPAN), C] or NULL: what kla_gated_scan_bwd needs of this call,
 *            the state before every KLA_SCAN_SPAN-th token (not written past a sequence's end)
 *   sizes    B, C >= 1, 0 <= T <= 2^31 - 1 - 65536 (T = 0 writes h_T only)
 *   alignment: x, gate, y their element; fp32 tensors 4 bytes; workspace 16 bytes
 */
#define KLA_SCAN_SPAN 128

typedef enum { KLA_SCAN_SIGMOID = 0, KLA_SCAN_LOG = 1 } kla_scan_mode;

kla_status kla_gated_scan_fwd(const void *x, const void *gate, const int64_t *strides, const int *lengths,
                              const float *h0, void *y, float *h_T, float *states, int B, int T, int C,
                              kla_dtype dtype, kla_scan_mode mode, void *workspace, size_t workspace_bytes,
                              void *stream);

/* Bytes of device scratch for kla_gated_scan_fwd, and for kla_gated_scan_bwd (0 if none). */
size_t kla_gated_scan_workspace_size(int B, int T, int C, kla_dtype dtype);

/*
 * Gradients of a loss through kla_gated_scan_fwd with the same inputs, given dy = dL/dy, the
 * forward's `states` and dh_T = dL/dh_T (NULL: zero). With dh_t = dy_t + a_{t+1} dh_{t+1} (the last
 * valid token: dy_t + dh_T):
 *     KLA_SCAN_SIGMOID   dx_t = (1 - a_t) dh_t,   dgate_t = a_t (1 - a_t) (h_{t-1} - x_t) dh_t
 *     KLA_SCAN_LOG       dx_t = dh_t,             dgate_t = a_t h_{t-1} dh_t
 * and dh0 = a_0 dh_0. Masked tokens have zero gradients, whatever dy holds there.
 *   strides     batch and token of x, gate, dy (6 values) or NULL
 *   dx, dgate   [B, T, C] dtype, contiguous, written (rounded once); dh0 fp32 [B, C] or NULL
 */
kla_status kla_gated_scan_bwd(const void *x, const void *gate, const void *dy, const int64_t *strides,
                              const int *lengths, const float *states, const float *dh_T, void *dx, void *dgate,
                              float *dh0, int B, int T, int C, kla_dtype dtype, kla_scan_mode mode, void *workspace,
                              size_t workspace_bytes, void *stream);

/*
 * One token for B sequences: h (fp32 [B, C]) is updated in place, y [B, C] dtype is written.
 *   x, gate  [B, C] dtype, rows x_stride and gate_stride elements apart (>= C)
 */
kla_status kla_gated_scan_step(const void *x, int64_t x_stride, const void *gate, int64_t gate_stride, float *h,
                               void *y, int B, int C, kla_dtype dtype, kla_scan_mode mode, void *stream);

/*
 * Self-test of the scan's bounded waits, as kla_selftest_wait_timeout of kla.h: kla_gated_scan_fwd, or
 * with `backward` kla_gated_scan_bwd, in KLA_SCAN_SIGMOID with x as the gate (and as dy), of which the
 * first sequence's first tile (backward: its last) of the first channels is left out, so that the tiles
 * that it would tell its state wait for nothing. After `limit_polls` questions (1 .. 2^21, the calls'
 * own limit, a second or two) they give up, which calls every other wait of the call off; all outputs
 * are undefined then. The next kla_device_status() returns KLA_ERR_TIMEOUT.
 *   out, out2   y (out2 unused), or dx and dgate;  T > 256;  the rest as the calls have it
 */
kla_status kla_selftest_scan_timeout(unsigned limit_polls, int backward, const void *x, float *states, void *out,
                                     void *out2, int B, int T, int C, kla_dtype dtype, void *workspace,
                                     size_t workspace_bytes, void *stream);

/* ------------------------------------------------------------------------------------- rotary
 *
 * The first `rot` of the d values of every head are turned by their token's position: pair i of
 * values (u, v) with angle t = position freqs[i] becomes
 *
 *     u' = scale (u cos t - v sin t),    v' = scale (v cos t + u sin t)
 *
 * with `inverse` by -t, which is the gradient's way back. The other d - rot values are copied.
 *   layout     KLA_ROTARY_HALF: pair i is values i and i + rot / 2; KLA_ROTARY_INTERLEAVED: 2 i, 2 i + 1
 *   q, k       [B, T, Hq, d] and [B, T, Hk, d] dtype, last axis contiguous; k may be NULL (Hk = 0)
 *   q_out, k_out  the same shapes
 *   strides    element strides of the batch, token and head axes of q, k, q_out, k_out (12 values,
 *              none negative); NULL means contiguous tensors. An output may be its own input in place
 *              (the same address and strides; q and k share no value then), else it shares no value with an
 *              input or the other output: slices of one tensor, of equal strides, may reach over each other
 *   freqs      fp32 [rot / 2], finite
 *   positions  [B, T] int64 (positions_are_64 != 0) or int32, contiguous, or NULL: token t has position t
 *   scale      finite
 *   sizes      B, T, Hk >= 0, Hq >= 1, 1 <= d <= 1024, rot even, 0 <= rot <= d
 * Angles are held as a 64-bit fraction of a turn, so that they do not lose bits with the position
 * (2^-24 of a turn at most for frequencies up to 4 at positions up to 2^28, in proportion to both
 * beyond); only sine and cosine are taken in fp32.
 */
typedef enum { KLA_ROTARY_HALF = 0, KLA_ROTARY_INTERLEAVED = 1 } kla_rotary_layout;

kla_status kla_rotary(const void *q, const void *k, void *q_out, void *k_out, const int64_t *strides,
                      const float *freqs, const void *positions, int positions_are_64, int B, int T, int Hq, int Hk,
                      int d, int rot, kla_rotary_layout layout, kla_dtype dtype, float scale, int inverse,
                      void *stream);

/* ----------------------------------------------------------------------------- a block's norms
 *
 * Norms over the last axis, in fp32: xh = (x - mean) rstd with KLA_NORM_LAYER, xh = x rstd with
 * KLA_NORM_RMS (rstd = 1 / sqrt(mean of squares + eps); squares are summed of differences, never of
 * values, in KLA_NORM_LAYER). n >= 3, as for kla_layer_norm_fwd, and n <= 65536.
 */
typedef enum { KLA_NORM_RMS = 0, KLA_NORM_LAYER = 1 } kla_norm_kind;
typedef enum { KLA_ACT_SILU = 0, KLA_ACT_SIGMOID = 1 } kla_activation;

/*
 * After a block's heads: y = xh weight act(gate), act(z) = z / (1 + exp(-z)) or 1 / (1 + exp(-z)).
 *   x, y    [rows, groups, n] dtype, contiguous
 *   gate    the same, rows gate_stride >= groups n elements apart (a slice of a packed projection)
 *   weight  fp32 [n], or [groups, n] where weight_groups != 0, or NULL (1)
 *   mean    fp32 [rows, groups], written, or NULL (not wanted; always NULL with KLA_NORM_RMS)
 *   rstd    fp32 [rows, groups], written, or NULL
 */
kla_status kla_gated_norm_fwd(const void *x, const void *gate, int64_t gate_stride, const float *weight,
                              int weight_groups, void *y, float *mean, float *rstd, int64_t rows, int groups, int n,
                              kla_dtype dtype, kla_norm_kind norm, kla_activation act, float eps, void *stream);

/*
 * Its gradients given dy [rows, groups, n] and the forward's mean (NULL: KLA_NORM_RMS) and rstd: dx,
 * dgate (dtype, contiguous) and dweight (fp32, shaped like weight; NULL: not wanted). The sums over
 * the rows are taken in a fixed order: equal calls give equal bits.
 */
kla_status kla_gated_norm_bwd(const void *dy, const void *x, const void *gate, int64_t gate_stride,
                              const float *weight, int weight_groups, const float *mean, const float *rstd, void *dx,
                              void *dgate, float *dweight, int64_t rows, int groups, int n, kla_dtype dtype,
                              kla_activation act, void *workspace, size_t workspace_bytes, void *stream);
size_t kla_gated_norm_bwd_workspace_size(int64_t rows, int groups, int n, kla_dtype dtype, int weight_groups);

/*
 * Between two blocks: sum = residual + scale x, y = xh(sum) weight. The norm is taken of the sum
 * before it is rounded to dtype.
 *   x, residual, sum, y  [rows, n] dtype, contiguous; sum may be residual itself
 *   weight, scale        fp32 [n] or NULL (1)
 *   mean, rstd           fp32 [rows], written, as above
 */
kla_status kla_add_norm_fwd(const void *x, const void *residual, const float *weight, const float *scale, void *y,
                            void *sum, float *mean, float *rstd, int64_t rows, int n, kla_dtype dtype,
                            kla_norm_kind norm, float eps, void *stream);

/*
 * Its gradients given dy, dsum (what reaches the sum from further on; NULL: nothing), the forward's x,
 * residual, mean (NULL: KLA_NORM_RMS) and rstd: dresidual = dsum + the norm's gradient, dx = scale
 * dresidual, dscale = sum over the rows of x dresidual. The sum is formed again from x and residual, as
 * a rounded one would cost dweight all but 9 of its bits: a forward call that is followed by this one
 * does not write its sum over the residual. Equal calls give equal bits.
 *   dx        NULL where scale is: then dresidual is the gradient of x too
 *   dweight, dscale  fp32 [n] or NULL (not wanted; dscale is NULL where scale is)
 */
kla_status kla_add_norm_bwd(const void *dy, const void *dsum, const void *x, const void *residual,
                            const float *weight, const float *scale, const float *mean, const float *rstd, void *dx,
                            void *dresidual, float *dweight, float *dscale, int64_t rows, int n, kla_dtype dtype,
                            void *workspace, size_t workspace_bytes, void *stream);
size_t kla_add_norm_bwd_workspace_size(int64_t rows, int n, kla_dtype dtype);

/* ------------------------------------------------------------------------- drafted tokens
 *
 * Speculative decoding's verification: sequence b has n_b = lengths[b] drafted tokens (K when lengths
 * is NULL). Draft i is accepted if every one before it was and uniforms[b, i] q(token) < p(token),
 * with p = target[b, i, :] and q = draft_probs[b, i, :]; the product is exact. After `a` accepted
 * drafts the next token is drawn by uniforms[b, K]: from target[b, n_b, :] where all were accepted,
 * else from max(p - q, 0) at position a (from p where that is zero everywhere): the lowest token
 * whose running sum, held to 2^-39 of the whole or better, is above uniforms[b, K] times the whole. Tokens are thus distributed
 * as the target's, whatever the draft. Rows need not sum to one; values that are not above zero (NaN
 * among them) count as zero, +inf (in bf16 too) as the largest finite value of fp32.
 *   draft        int32 [B, K]; a token outside [0, V) is not accepted, and has q = 0
 *   draft_probs  [B, K, V] dtype, or NULL: the draft was sure of its tokens (q = 1 there, 0 elsewhere)
 *   target       [B, K + 1, V] dtype
 *   strides      element strides of the batch and row axes of draft_probs, then of target (4 values,
 *                none negative), or NULL: contiguous. The last axis is contiguous
 *   uniforms     fp32 [B, K + 1] in [0, 1)
 *   lengths      int32 [B] or NULL; values are taken into [0, K]
 *   accepted     int32 [B], written: the accepted drafts, 0 .. n_b
 *   tokens       int32 [B, K + 1], written: the accepted drafts, the next token, then -1. A target row
 *                without a value above zero has no next token: -1
 *   sizes        B >= 1, 0 <= K <= 1024, 1 <= V <= 2^24
 */
kla_status kla_verify_draft(const int *draft, const void *draft_probs, const void *target, const int64_t *strides,
                            const float *uniforms, const int *lengths, int *accepted, int *tokens, int B, int K,
                            int V, kla_dtype dtype, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* KLA_BLOCK_H */

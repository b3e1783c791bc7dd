/*
 * kla_layer.h -- C ABI of what a layer and a decoding loop need next to the recurrence of kla.h on
 * NVIDIA GB300 (sm_103a): linear attention with one decay per head (prompts, single tokens,
 * gradients), layer norm (forward, gradients) and beam search's selection with the states
 * following their beams.
 *
 * The conventions of kla.h hold: device pointers, caller-owned buffers, calls asynchronous on
 * `stream` (whose device has to be the current one), argument errors found on the host before
 * anything is launched (KLA_ERR_INVALID_ARG / KLA_ERR_UNSUPPORTED, nothing written), bounded device
 * waits reported by kla_device_status.
 * Outputs and workspaces must not overlap each other or any input unless said otherwise.
 */
#ifndef KLA_LAYER_H
#define KLA_LAYER_H

#include <stddef.h>
#include <stdint.h>

#include "kla.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ------------------------------------------------------- linear attention, one decay per head
 *
 * For every sequence b and head h, with g = decay[h] and a state S (d_k x d_v):
 *
 *     S_t = g S_{t-1} + k_t v_t^T,        o_t = s S_t^T q_t      (the read follows the write)
 *
 * for t = 0 .. n_b - 1, where n_b = lengths[b] (T when lengths is NULL). Tokens t >= n_b are
 * masked: whatever q, k, v hold there (NaN included) they leave the state as it is, and o_t = 0.
 * A valid token that holds an infinity or a NaN spoils the state from there on, and, since tokens
 * meet in products of 64 or 128, the outputs of up to 127 tokens before it.
 *
 *   q, k     [B, T, H, d_k] dtype, v [B, T, H, d_v] dtype; last axis contiguous. `strides` gives
 *            the element strides of the batch, token and head axes of q, then k, then v (9
 *            values, none negative); NULL means contiguous tensors
 *   decay    fp32 [H], values in [0, 1]
 *   lengths  int32 [B] or NULL; values are taken into [0, T]
 *   S0       fp32 [B, H, d_k, d_v] or NULL (zeros)
 *   o        [B, T, H, d_v] dtype, contiguous, written
 *   S_T      fp32 [B, H, d_k, d_v] or NULL; may be S0 itself
 *   q_scale  the finite scale s
 *   sizes    d_k, d_v in {16, 32, 64, 128}; 0 <= T <= 2^31 - 1 - 65536 (T = 0 writes S_T only)
 *   alignment: q, k, v, o their element; S0, S_T, workspace 16 bytes
 *
 * bf16 with d_k = d_v = 128 and 16-byte aligned rows runs on the tensor cores (bf16 operands, fp32
 * accumulation and state; the state's update is split into two bf16 terms, so that S_T and
 * kla_linear_bwd's dS0 are off by about 4e-6 of their norm, by 1.1e-5 at most for few tokens);
 * every other call in fp32 on the CUDA cores.
 */
kla_status kla_linear_fwd(const void *q, const void *k, const void *v, const int64_t *strides, const float *decay,
                          const int *lengths, const float *S0, void *o, float *S_T, int B, int T, int H, int d_k,
                          int d_v, kla_dtype dtype, float q_scale, void *workspace, size_t workspace_bytes,
                          void *stream);

/* Bytes of device scratch for kla_linear_fwd (0 if none): the states at which the segments of long
 * sequences start. */
size_t kla_linear_fwd_workspace_size(int B, int T, int H, int d_k, int d_v, kla_dtype dtype);

/*
 * Gradients of a loss through kla_linear_fwd with the same inputs, given dO = dL/do and
 * dS_T = dL/dS_T (NULL: zero):
 *     dS_t = s q_t dO_t^T + g dS_{t+1},   dq_t = s S_t dO_t,   dk_t = dS_t v_t,   dv_t = dS_t^T k_t
 * and dS0 = g dS_0. Masked tokens have zero gradients. `decay` is a constant of the layer and gets
 * none.
 *   strides     batch, token, head of q, k, v, dO (12 values) or NULL
 *   dq, dk, dv  contiguous, in dtype (rounded once); dS0 fp32 or NULL
 */
kla_status kla_linear_bwd(const void *q, const void *k, const void *v, const void *dO, const int64_t *strides,
                          const float *decay, const int *lengths, const float *S0, const float *dS_T, void *dq,
                          void *dk, void *dv, float *dS0, int B, int T, int H, int d_k, int d_v, kla_dtype dtype,
                          float q_scale, void *workspace, size_t workspace_bytes, void *stream);
size_t kla_linear_bwd_workspace_size(int B, int T, int H, int d_k, int d_v, kla_dtype dtype);

/*
 * One token for B sequences: S <- g S + k v^T, o = s S^T q.
 *   q, k [B, H, d_k], v [B, H, d_v] dtype, contiguous; decay fp32 [H]
 *   S        fp32 [n_states, H, d_k, d_v]
 *   parent   NULL: sequence b owns state b (n_states = B), and S_out is S (in place) or a separate
 *            buffer. Else int32 [B]: sequence b goes on from state parent[b] (the reordering of a
 *            beam search at no extra pass over the states); an index outside [0, n_states) starts
 *            from the zero state, and S_out must not overlap S.
 *   S_out    fp32 [B, H, d_k, d_v], written
 */
kla_status kla_linear_step(const void *q, const void *k, const void *v, const float *decay, const int *parent,
                           const float *S, float *S_out, void *o, int B, int H, int d_k, int d_v, int n_states,
                           kla_dtype dtype, float q_scale, void *stream);

/* ---------------------------------------------------------------------------------- layer norm
 *
 * Over the last axis of x [rows, groups, n]: mean, rstd = 1 / sqrt(var + eps),
 * y = (x - mean) rstd w[g] + b[g]. groups = 1 is the plain layer norm; groups = H with n = d_v
 * normalises every head's output with weights of its own.
 *   x, y    dtype, contiguous                      weight, bias  fp32 [groups, n] or NULL (1 / 0)
 *   mean, rstd  fp32 [rows, groups], written (NULL: not wanted)
 *   rows >= 0, groups >= 1, 3 <= n <= 65536 (the normalised values of one or two values do not
 *   depend on them but for eps, and their gradient is what rounding leaves: KLA_ERR_UNSUPPORTED)
 * Statistics are taken in fp32 about the mean: squares are summed of differences, never of values.
 */
kla_status kla_layer_norm_fwd(const void *x, const float *weight, const float *bias, void *y, float *mean,
                              float *rstd, int64_t rows, int groups, int n, kla_dtype dtype, float eps,
                              void *stream);

/*
 * Gradients of kla_layer_norm_fwd given dy [rows, groups, n] and the forward's mean and rstd:
 * dx (dtype), dweight and dbias (fp32 [groups, n]; NULL: not wanted). The sums over the rows are
 * taken in a fixed order: equal calls give equal bits. The workspace may be NULL where n <= 8192 and
 * neither dweight nor dbias is wanted.
 */
kla_status kla_layer_norm_bwd(const void *dy, const void *x, const float *weight, const float *mean,
                              const float *rstd, void *dx, float *dweight, float *dbias, int64_t rows, int groups,
                              int n, kla_dtype dtype, void *workspace, size_t workspace_bytes, void *stream);
size_t kla_layer_norm_bwd_workspace_size(int64_t rows, int groups, int n, kla_dtype dtype);

/* ---------------------------------------------------------------------------------- beam search
 *
 * One selection over beams and vocabulary. With lp = log_softmax(logits[b, w, :]), a candidate
 * (w, token) has the score scores[b, w] + lp[token]; a finished beam goes on with the token `eos`
 * alone, at no cost. Each beam ranks its tokens by logit (equal logits: the lower token first); the
 * ranked lists are merged by score (equal scores: the lower beam, then the better rank), and the
 * W best are taken. NaN logits count as -inf and +inf as the largest finite value; a beam whose
 * score is -inf or NaN, or whose logits are all -inf, has only candidates of score -inf, which are
 * taken when nothing else is left.
 *   logits      [B, W, V] dtype; rows row_stride >= V elements apart
 *   scores      fp32 [B, W]            finished  uint8 [B, W] (0 / 1) or NULL (none)
 *   eos         token that finishes a beam, or -1 (then `finished` must be NULL)
 *   new_scores  fp32 [B, W], parents, tokens int32 [B, W], new_finished uint8 [B, W] or NULL: written
 *   1 <= W <= 16, 1 <= V <= 2^21, B W <= 65535
 */
kla_status kla_beam_select(const void *logits, int64_t row_stride, const float *scores, const unsigned char *finished,
                           int eos, float *new_scores, int *parents, int *tokens, unsigned char *new_finished, int B,
                           int W, int V, kla_dtype dtype, void *workspace, size_t workspace_bytes, void *stream);
size_t kla_beam_select_workspace_size(int B, int W, int V, kla_dtype dtype);

/*
 * out[b, w] = S[b, parents[b, w]] for B x W states of `bytes` bytes each (a multiple of 16; the
 * states of kla_decode_step and kla_linear_step alike); a parent outside [0, W) gives zeros. out
 * must not overlap S.
 */
kla_status kla_reorder_states(const void *S, const int *parents, void *out, int B, int W, size_t bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* KLA_LAYER_H */

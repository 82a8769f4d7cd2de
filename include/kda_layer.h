/*
 * kda_layer.h -- C ABI of the operators around the Kimi Delta Attention
 * forward that libkda.so offers besides it (include/kda.h): the gated delta
 * rule with one decay per head (chunked prefill and single-token step), the
 * residual's addition with the RMS norm, and products with 4-bit weights for
 * few tokens.
 *
 * The rules of kda.h hold here too.  Device pointers are HIP device memory on
 * the current device; the caller owns every buffer and the library allocates
 * nothing.  Work is queued on `stream` (NULL = default stream) and the call
 * returns without waiting: no host synchronisation, no device-to-host copy,
 * so every call can be captured into a HIP graph.  All argument checks happen
 * before any HIP call; on an error nothing is launched.  A launch that fails
 * gives KDA_ERR_HIP, with its detail in kda_last_hip_error().  Results do not
 * depend on the schedule: the same call gives the same bits.  Rounding to
 * bf16 and e4m3 is to nearest, ties to even.
 */
#ifndef KDA_LAYER_H_
#define KDA_LAYER_H_

#include "kda.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * The gated delta rule with one decay per value head.  For every sequence and
 * value head h, with key head hk = h / (value_heads / key_heads), head_dim
 * D = 128 and a D x D state S[key][value]:
 *
 *     q~_t, k~_t <- x / sqrt(sum_c x[c]^2 + 1e-6)
 *     beta_t     =  1 / (1 + exp(-beta_logit_t))
 *     log a_t    =  -exp(A_log[h]) * softplus(a_t + dt_bias[h])
 *     S_t        =  a_t (I - beta_t k~_t k~_t^T) S_{t-1} + beta_t k~_t v_t^T
 *     o_t        =  scale * S_t^T q~_t
 *
 * The decay is one number per token and head and is not bounded below (decays
 * under e^-120 count as e^-120, which is 0 in fp32); kda_chunk_prefill_fwd has
 * a bounded decay per key channel instead.
 *
 * Element strides of the per-token tensors: row (t, h) of q starts at q + t *
 * q_token + h * q_head and holds its 128 channels contiguously (k, v and out
 * likewise); a and beta_logits of (t, h) are at t * x_token + h * x_head.  The
 * dense layout has x_token = heads * 128 and x_head = 128, and heads and 1
 * for a and beta.  Strides are non-negative; those of q, k and v are multiples
 * of 8, those of out are positive multiples of 8.  Rows of out that overlap
 * give undefined results.
 */
typedef struct {
  int64_t q_token, q_head;
  int64_t k_token, k_head;
  int64_t v_token, v_head;
  int64_t a_token, a_head;
  int64_t beta_token, beta_head;
  int64_t out_token, out_head;
} kda_gdr_strides_t;

/*
 * Bytes of device workspace kda_gdr_prefill_fwd needs for any call with at
 * most max_tokens tokens, these head counts and at most max_seqs sequences.
 * Pure, host-only, monotone in every argument; 0 for arguments below zero or
 * head counts the call refuses.
 */
size_t kda_gdr_get_workspace_size(int64_t max_tokens, int32_t key_heads, int32_t value_heads,
                                  int32_t max_seqs);

/*
 * Prefill over a packed varlen batch.
 *
 *   q, k           bf16 [num_tokens, key_heads, 128] (device)
 *   v, out         bf16 [num_tokens, value_heads, 128]; rows of out that
 *                  belong to no sequence are not touched
 *   a, beta_logits bf16 [num_tokens, value_heads]; raw
 *   A_log, dt_bias fp32 [value_heads]
 *   initial_state  [num_seqs, value_heads, 128, 128] in state_dtype (row = key
 *                  channel, column = value channel); NULL = zeros
 *   cu_seqlens     int32 [num_seqs + 1]: cu[0] = 0, non-decreasing,
 *                  cu[num_seqs] <= num_tokens.  Read on the device only;
 *                  offsets are clamped to [0, num_tokens] there.
 *   final_state    as initial_state; may be the same pointer (in-place
 *                  update), any other overlap is undefined.  An empty sequence
 *                  ends with the state it starts from.
 *   workspace      at least kda_gdr_get_workspace_size(num_tokens, key_heads,
 *                  value_heads, num_seqs) bytes, 256-byte aligned; written
 *                  before it is read (no initialisation, no status word).
 *                  Calls that may overlap need workspaces of their own, two
 *                  captured graphs that may run at once among them.
 *   strides        host pointer, or NULL for the dense layout
 *
 * q, k, v and out are 16-byte aligned, the states 16-byte, a and beta_logits
 * 2-byte.  value_heads is a multiple of key_heads, at most 65536;
 * num_seqs * value_heads < 2^21; (num_tokens / 64 + num_seqs) * value_heads <
 * 2^24; token strides of q, k, v and out at most 2^24, other strides 2^30.  q, k, v, a, beta_logits
 * and out may be NULL when num_tokens is 0, workspace too when the size query
 * gives 0.
 *
 * Numerics.  Sums, decays and the state are fp32 (sums of log decays fp64).
 * Factors of matrix products keep 22 bits with an fp32 state and 11 bits with
 * a bf16 state (out, which is bf16, 11 bits either way), relative to the
 * largest element of their column, so that out is off by a share of scale times
 * the state, also where a query is far below 1e-3 and its row of out with it.
 * Finite q, k, v, gates and states of any size are taken, as long as fp32 holds
 * the norm of a state's column and |scale| times it.  The final state and out are
 * rounded once, at the end.
 * An input that is not finite makes the rows of its sequence and of the value
 * heads that read it undefined from its chunk of 64 tokens on, and their
 * final states; other sequences and heads are not affected.
 *
 * Calls with at most 8 tokens per sequence on average run token after token,
 * others in chunks.  The lengths are on the device, so the average decides, and
 * one long sequence among many of a token or two takes about 2.3 us a token (255
 * of one token and one of 1500, 32 heads: 3.6 ms, in calls of their own 60 us and
 * 76 us): give it a call of its own.  Up to 32 (sequence, value head) pairs with
 * at least 2048 tokens per sequence on average (4096 above 8 pairs) run in
 * segments at once.  These forms agree within the bounds above, not bit for bit.
 */
kda_status_t kda_gdr_prefill_fwd(const void* q, const void* k, const void* v, const void* a,
                                 const void* beta_logits, const float* A_log, const float* dt_bias,
                                 float scale, const void* initial_state, const int32_t* cu_seqlens,
                                 void* out, void* final_state, void* workspace, void* stream,
                                 int64_t num_tokens, int32_t key_heads, int32_t value_heads,
                                 int32_t num_seqs, kda_state_dtype_t state_dtype,
                                 size_t workspace_bytes, const kda_gdr_strides_t* strides);

/*
 * One token for each of num_seqs sequences whose states live in a pool: the
 * recurrence above for row n of q, k, v, a, beta_logits and out ([num_seqs,
 * heads, ...]) on slot state_indices[n], read and written in place.
 *
 *   state_pool     [num_slots, value_heads, 128, 128] in state_dtype,
 *                  16-byte aligned
 *   state_indices  device int32 [num_seqs].  An index outside [0, num_slots)
 *                  marks a padding row: nothing of it is read or written, its
 *                  row of out keeps what it held.  A slot named twice gives
 *                  undefined values in that slot and those rows.
 *
 * Everything is fp32; a bf16 state is widened exactly and rounded once.  No
 * workspace.  Limits, strides and alignments as in the prefill.
 */
kda_status_t kda_gdr_decode_step(const void* q, const void* k, const void* v, const void* a,
                                 const void* beta_logits, const float* A_log, const float* dt_bias,
                                 float scale, void* state_pool, int64_t num_slots,
                                 const int32_t* state_indices, void* out, void* stream,
                                 int32_t num_seqs, int32_t key_heads, int32_t value_heads,
                                 kda_state_dtype_t state_dtype, const kda_gdr_strides_t* strides);

typedef enum { KDA_OUT_BF16 = 0, KDA_OUT_E4M3 = 1 } kda_out_dtype_t;

/*
 * Residual addition and RMS norm, row by row:
 *
 *     s = x + residual (fp32; s = x if residual is NULL)
 *     residual <- bf16(s), in place
 *     y = s / sqrt(mean(s^2) + eps) * weight
 *     out = bf16(y), or for KDA_OUT_E4M3
 *     out_scale = max|y| / 448 and out = e4m3(y / out_scale)
 *
 * with one scale per row (group_size 0) or per group_size = 128 channels (the
 * last group of a row may be shorter).  A group that is zero throughout gets
 * scale 0 and zeros, a row of zeros zeros (eps = 0 included).  y is formed from
 * the unrounded s.  Sums are fp32, of a scaled row where squares would leave its
 * range: finite s of any size are taken.  Where s is infinite y is NaN, and 0 in
 * the rest of its row; in e4m3 the scale over an infinity is NaN, and groups
 * beside it get scale 0 and zeros.  A NaN makes its row's bf16 output, or all of
 * its row's scales, NaN.
 *
 *   x, residual  bf16 [num_rows, dim], rows x_row and residual_row elements
 *                apart, dim contiguous
 *   weight       bf16 [dim]
 *   out          bf16 or e4m3 (OCP, 448 the largest) [num_rows, dim], rows
 *                out_row elements apart.  It may be x itself (bf16, same row
 *                stride); other overlaps of x, residual and out are undefined.
 *   out_scale    fp32 [num_rows, ceil(dim / 128)] or [num_rows], dense;
 *                NULL for bf16
 *
 * 1 <= dim <= 32768, 0 <= num_rows < 2^31, row strides >= dim (for one row
 * any).  No alignment beyond the element's is needed.
 */
kda_status_t kda_add_rms_norm(const void* x, void* residual, const void* weight, float eps,
                              void* out, float* out_scale, void* stream, int64_t num_rows,
                              int32_t dim, int64_t x_row, int64_t residual_row, int64_t out_row,
                              kda_out_dtype_t out_dtype, int32_t group_size);

/*
 * Products of few tokens (a decode step) with 4-bit weights:
 *
 *     y[m, n] = bf16( sum_k x[m, k] * (w[n, k] - z[n, g]) * scales[n, g] ),  g = k / group_size
 *
 *   x       bf16 [num_tokens, k], rows x_row elements apart (a multiple of
 *           8, at most 2^24)
 *   w       uint8 [n, k / 2], dense: byte j of a row holds w[n, 2 j] in its
 *           low and w[n, 2 j + 1] in its high four bits, each 0..15
 *   scales  bf16 [n, k / group_size], dense
 *   zeros   bf16 [n, k / group_size], dense, or NULL: z = 8
 *   y       bf16 [num_tokens, n], rows y_row elements apart
 *
 * group_size is 32, 64 or 128, k a positive multiple of it (at most 2^20),
 * 1 <= n <= 2^24, 0 <= num_tokens <= 64; x and w are 16-byte aligned.  Sums
 * are fp32, of exact products; a group's is formed as sum (128 + w) x - (128 + z)
 * sum x, which costs about five of the sum's 24 bits.  Sums up to 2^143 are held
 * on the way to y, and so is every finite x (z from 0 to 15).  A value of x that
 * is not finite makes its row of y NaN; other rows are not affected.  A token's
 * sums may be taken in another order in a call with another number of tokens.
 * No workspace.  x may be NULL when num_tokens is 0.
 */
kda_status_t kda_w4_proj(const void* x, const void* w, const void* scales, const void* zeros,
                         void* y, void* stream, int32_t num_tokens, int32_t k, int32_t n,
                         int32_t group_size, int64_t x_row, int64_t y_row);

#ifdef __cplusplus
}
#endif

#endif /* KDA_LAYER_H_ */

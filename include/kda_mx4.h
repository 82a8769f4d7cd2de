/*
 * kda_mx4.h -- C ABI of the operators of libkda.so on microscaled 4-bit numbers:
 * quantisation and its inverse, products with weights in that format, and a
 * mixture-of-experts layer for few tokens whose experts are in it.
 *
 * The rules of kda.h and kda_layer.h hold here too: device pointers on the
 * current device, work queued on `stream`, no allocation, no synchronisation,
 * every call can be captured into a HIP graph, all argument checks before any
 * HIP call, the same call gives the same bits.
 *
 * The format.  A row of k elements, k a multiple of 32, is
 *
 *   codes   uint8 [k / 2]: byte j holds element 2 j in its low and 2 j + 1 in its
 *           high four bits; e2m1: a sign bit above 0, 0.5, 1, 1.5, 2, 3, 4, 6
 *   scales  uint8 [k / 32]: e8m0, 2^(s - 127) for the 32 elements they belong to,
 *           s = 255: NaN
 *
 * and rows are dense: codes and scales of row r begin at r * k / 2 and r * k / 32.
 */
#ifndef KDA_MX4_H_
#define KDA_MX4_H_

#include "kda_layer.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Quantisation: for each 32 adjacent elements of a row with largest magnitude m
 *
 *     s     = max(0, floor(log2 m) - 2 + 127), 0 where m = 0
 *     codes = e2m1(x 2^(127 - s)), to nearest, ties to even, at most 6 in magnitude
 *
 * which is exact arithmetic: one right answer for every input.  Elements between
 * 7 / 8 and all of the next power of two of m are cut to 6 2^(s - 127).  32
 * elements with an infinity or a NaN among them get s = 255 and codes 0.
 *
 *   x       bf16 [num_rows, k], rows x_row elements apart
 *   codes, scales  as above; codes 4-byte aligned
 *
 * k is a positive multiple of 32, at most 2^20; 0 <= num_rows < 2^31, num_rows * k
 * below 2^36; x 16-byte aligned, x_row a multiple of 8 between k and 2^30 (for one
 * row any).  Nothing overlaps.
 */
kda_status_t kda_mx4_quant(const void* x, void* codes, void* scales, void* stream, int64_t num_rows,
                           int32_t k, int64_t x_row);

/*
 * The values of codes and scales as bf16 [num_rows, k], rows out_row elements
 * apart.  Exact, except that values of 2^128 and more (s = 253 and 254) are
 * infinite.  Limits as for the quantisation; out 16-byte, codes 4-byte aligned.
 */
kda_status_t kda_mx4_dequant(const void* codes, const void* scales, void* out, void* stream,
                             int64_t num_rows, int32_t k, int64_t out_row);

/*
 * Products with weights w [n, k] in the format:  y[m, j] = bf16(sum_k x[m, k] w[j, k]).
 *
 *   x         x_scales NULL: bf16 [num_tokens, k], rows x_row elements apart,
 *             at most 64 of them.  Otherwise codes [num_tokens, k / 2], any
 *             number of rows below 2^31, dense (x_row is not read)
 *   w, w_scales    codes and scales of n rows
 *   y         bf16 [num_tokens, n], rows y_row elements apart
 *
 * k is a positive multiple of 32, at most 2^20; 1 <= n <= 2^24; x and w are
 * 16-byte aligned; x_row a multiple of 8 between k and 2^24, y_row between n and
 * 2^30 (for one row any); ceil(num_tokens / 256) * ceil(n / 256) < 2^23.  y must
 * not overlap x or w.
 *
 * Products and sums are fp32: every product between 2^-126 and 2^128 in magnitude is
 * exact, what is smaller may count as 0, and what is larger is infinite, as are, with
 * bf16 x, weights of 2^128 and more (s = 253 and 254).  Up to 128 products at a time
 * are added in one instruction, whose own sum is off by less than 2^-24 of their
 * magnitudes.  A value of x that is not finite, or a scale of NaN, makes its token's
 * row of y, or its weight row's column, NaN or infinite; others are not affected.
 * The order of a sum may depend on num_tokens, and on nothing else of the other
 * tokens.  Of the scales the whole aligned 4-byte words may be read in which those of
 * an operand begin and end; what else is in them has no effect.  No workspace.  x and
 * y may be NULL when num_tokens is 0.
 */
kda_status_t kda_mx4_proj(const void* x, const void* x_scales, const void* w, const void* w_scales,
                          void* y, void* stream, int64_t num_tokens, int32_t k, int32_t n,
                          int64_t x_row, int64_t y_row);

typedef enum { KDA_ROUTE_SIGMOID = 0, KDA_ROUTE_SOFTMAX = 1 } kda_route_t;

/*
 * A mixture-of-experts layer for a decode step's tokens.  For every token x:
 *
 *     l_e   =  sum_k x[k] router[e, k]
 *     p_e   =  1 / (1 + exp(-l_e)), or exp(l_e) / sum_f exp(l_f)
 *     ids   =  the top_k experts with the largest p_e + router_bias[e], largest
 *              first, of equal ones the lowest index (see below)
 *     gate_j = route_scale * p_(ids j) [ / sum_i p_(ids i) with renormalise ]
 *     f_e(x) =  W_down,e (silu(G_e x) * (U_e x)),  silu(a) = a / (1 + exp(-a))
 *     out   =  bf16( sum_j gate_j f_(ids j)(x) + sum_s f_(experts + s)(x) )
 *
 * where G_e are the first `inter` rows of w_up's expert e and U_e the others, and
 * the last sum runs over `shared` experts that every token goes through.
 *
 *   x            bf16 [num_tokens, k], rows x_row elements apart
 *   router       bf16 [experts, k], dense
 *   router_bias  fp32 [experts] or NULL (zeros); counts for the choice alone
 *   w_up, w_up_scales      [experts + shared, 2 inter, k] in the format
 *   w_down, w_down_scales  [experts + shared, k, inter] in the format
 *   state_indices  device int32 [num_tokens] or NULL: an index below zero marks a
 *                padding row, as for kda_gdr_decode_step: its row of out keeps
 *                what it held, its ids are -1 and its gates 0
 *   out          bf16 [num_tokens, k], rows out_row elements apart; must not
 *                overlap another operand
 *   expert_ids   int32 [num_tokens, top_k], written
 *   expert_gates fp32 [num_tokens, top_k], written
 *   workspace    at least kda_mx4_moe_workspace_size(num_tokens, k, inter, experts,
 *                shared, top_k) bytes, 256-byte aligned; written before it is read.
 *                Calls that may overlap need workspaces of their own, two captured
 *                graphs that may run at once among them.
 *
 * 0 <= num_tokens <= 64; k and inter positive multiples of 32, at most 2^16;
 * 1 <= experts <= 1024; 0 <= shared <= 16; 1 <= top_k <= min(experts, 32); x,
 * router, w_up, w_down and out 16-byte aligned, x_row and out_row multiples of 8
 * between k and 2^24 (for one row any).
 *
 * Numerics.  The router's products, sums and scores are fp64, so that the choice is
 * that of the formula for scores that differ by more than about 1e-15 of the
 * logits' terms, and a token's ids and gates do not depend on the other tokens.
 * Where fp64 holds two finite sums p_e + router_bias[e] as the same (scores of
 * sigmoid that are 1 to the last bit, those beside a bias of 1e30), the larger
 * logit comes first, and of equal logits the lowest index; of infinite sums the
 * lowest index.  A sum of NaN comes behind all others.  G x and U x are fp32 sums,
 * with the range of kda_mx4_proj for bf16 x; gate silu(G x) (U x) is an fp32 number
 * that enters W_down with all of its bits (as three bf16 pieces; what of it is
 * below 2^-133 is lost); sums over inter and over experts are fp32, in an order
 * that depends on which experts the other tokens take (the last bits of out do,
 * too), and out is rounded once.  An infinity or a NaN in x or in an expert's
 * weights leaves the choice well defined and makes the rows of out that read it NaN
 * or infinite; it does not enter other rows.  Where the chosen scores add up to 0,
 * renormalise gives NaN.
 */
size_t kda_mx4_moe_workspace_size(int32_t max_tokens, int32_t k, int32_t inter, int32_t experts,
                                  int32_t shared, int32_t top_k);
kda_status_t kda_mx4_moe(const void* x, const void* router, const float* router_bias,
                         const void* w_up, const void* w_up_scales, const void* w_down,
                         const void* w_down_scales, const int32_t* state_indices, void* out,
                         int32_t* expert_ids, float* expert_gates, void* workspace, void* stream,
                         int32_t num_tokens, int32_t k, int32_t inter, int32_t experts,
                         int32_t shared, int32_t top_k, int64_t x_row, int64_t out_row,
                         kda_route_t scoring, int32_t renormalise, float route_scale,
                         size_t workspace_bytes);

#ifdef __cplusplus
}
#endif

#endif /* KDA_MX4_H_ */

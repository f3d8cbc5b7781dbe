/*
 * msb_dense.h -- the dense MoE block for prompts, and the operators it is made of.
 *
 * The block of msb.h reads k channels per (token, expert) for a decode step of up to
 * MSB_MAX_BATCH tokens.  A prompt's tokens together read every channel of every routed
 * expert, so a prompt is better served by the dense block (k = I, rank 0) as matrix
 * products grouped by expert.  The entry points here take any number of tokens and read
 * the same packed weights (router_t, records) as moe_sparse_block, or 8-bit weights:
 *
 *   msb_route            top-K experts of each token, and the rows sorted by expert
 *   msb_grouped_matmul   products of ragged groups of rows with their group's weight
 *   msb_grouped_swiglu   the same for gate and up, with SwiGLU
 *   msb_int8_quantize    rows to 8-bit integers with one scale each
 *   msb_int8_matmul, msb_int8_swiglu, msb_int8_linear   the products in 8-bit integers
 *   msb_combine          a token's expert rows summed by router weight
 *   msb_block_norm       norms before and after a block with its gate and residual scale
 *   moe_dense_block, moe_dense_block_int8   the whole block
 *
 * Conventions are those of msb.h (device pointers of the current device, caller-owned
 * buffers, asynchronous on `stream`, MSB_OK or a negative code, argument errors before
 * anything is enqueued).  Row pitches are in elements, 0 .. 2^28 - 1.  Nothing here keeps
 * state between calls except one error word per device, set when a bounded wait inside a
 * kernel runs out: msb_dense_check reads it.
 * Calls may overlap on the GPU (other streams, captured graphs) as long as their output and
 * workspace buffers differ.
 */
#ifndef MSB_DENSE_H_
#define MSB_DENSE_H_

#include <stddef.h>
#include <stdint.h>

#include "msb.h"

#ifdef __cplusplus
extern "C" {
#endif

#define MSB_DENSE_MAX_TOKENS 1048576 /* tokens of a route or a dense block */
#define MSB_GROUPED_MAX_NK 1048576   /* n and k of a grouped product */
#define MSB_GROUPED_MAX_ROWS 1073741824 /* output rows of a grouped product */
#define MSB_NORM_MAX_D 16384         /* row length of msb_block_norm */
#define MSB_INT8_MAX_K 131056        /* inner length of an 8-bit product: the int32 sum of
                                        k products of at most 128^2 stays below 2^31 */

/* Element types of an operand that may have either. */
#define MSB_BF16 0
#define MSB_F32 1

/* Synchronises `stream`, reads and clears the current device's error word of the entry
 * points of this header.  MSB_OK, MSB_ETIMEOUT (a bounded wait of some call since the last
 * check ran out: that call's output is undefined), or MSB_ECUDA. */
int32_t msb_dense_check(void* stream);

/* ------------------------------------------------------------------ routing
 * For each token the top_e experts of highest logit (ties: lower index), their combine
 * weights, and the (token, expert) pairs sorted by expert and token:
 *   ids      int32 [tokens][top_e]  highest logit first; -1 where no candidate is left
 *   weights  float [tokens][top_e]  exp(l - max), divided by the sum over the kept experts
 *                                   (renorm = 1) or over all candidates (renorm = 0); 0 for -1
 *   offsets  int32 [experts + 1]    expert e has the rows offsets[e] .. offsets[e + 1] - 1
 *   rows     int32 [tokens * top_e] token of each row, ascending within an expert; -1 behind
 *                                   the last row
 *   pos      int32 [tokens][top_e]  row of each pair; -1 for -1
 * A logit that is NaN or -infinity is no candidate; +infinity counts as the largest finite
 * float.  mask (optional, uint8 [tokens]): a token whose mask is 0 has no candidates.
 *  logits   logits_type (MSB_F32, MSB_BF16), row t at logits + t * ld elements, ld >= experts.
 *  tokens   0..MSB_DENSE_MAX_TOKENS; experts 1..MSB_MAX_EXPERTS; top_e 1..min(experts, 16).
 *  workspace, workspace_bytes: msb_route_workspace_size(tokens, experts) bytes of scratch, no
 *           initial contents needed. */
size_t msb_route_workspace_size(int32_t tokens, int32_t experts);
int32_t msb_route(const void* logits, int32_t logits_type, int64_t ld, const uint8_t* mask,
                  int32_t tokens, int32_t experts, int32_t top_e, int32_t renorm, int32_t* ids,
                  float* weights, int32_t* offsets, int32_t* rows, int32_t* pos, void* workspace,
                  size_t workspace_bytes, void* stream);

/* ------------------------------------------------------------------ grouped products
 * Weights of `groups` groups, read where they lie; strides in elements.  Element (n, k) of
 * group e (and part p, for SwiGLU: 0 = gate, 1 = up) is at
 *   data + e * stride_group + p * stride_part + n * stride_n + k * stride_k.
 * stride_k = 1, or (bf16 matmul only) stride_n = 1; the other strides positive multiples of
 * 16 bytes; data 16-byte aligned.  The channel records of msb_pack are such weights: gate and
 * up {records, 3 d I, d, 3 d, 1}, down {records + 2 d, 3 d I, 0, 1, 3 d}. */
typedef struct msb_group_weights {
  const void* data;
  int64_t stride_group, stride_part, stride_n, stride_k;
} msb_group_weights;

/* out[p][j] = sum_i x[row(p)][i] * w[e][j][i] for the rows p of group e,
 * offsets[e] <= p < offsets[e + 1]; rows that belong to no group are left as they are.
 *  x        bf16, x_rows rows ldx elements apart; 16-byte aligned, ldx * 2 a positive multiple
 *           of 16.
 *  rows     row of x for each output row (int32 [out_rows]), or NULL: row(p) = p (x_rows >=
 *           out_rows).  x_rows is at least 1 where out_rows is.  A row outside 0..x_rows-1 reads as zeros.
 *  offsets  int32 [groups + 1] on the device, ascending, within 0..out_rows; NULL with
 *           groups = 1: all rows.  (An offset that is not is moved to the nearest that is.)
 *  out_rows rows of out, up to MSB_GROUPED_MAX_ROWS; 0 is allowed and does nothing.
 *  groups   1..MSB_MAX_EXPERTS; n, k 1..MSB_GROUPED_MAX_NK.
 *  out      out_type (MSB_BF16 or MSB_F32), row p at out + p * ldo elements, ldo >= n; must
 *           not overlap x or the weights.
 * Sums in FP32, rounded once to out_type.  The matrix unit cuts off its additions towards zero
 * instead of rounding them: bf16 outputs whose products are all of one sign come out up to
 * 7.5e-9 k too small, relative, and 2.4e-4 at most (a sixteenth of the largest rounding error of
 * bf16), those of mixed signs far less; float outputs keep to about 1e-6. */
int32_t msb_grouped_matmul(const void* x, int64_t ldx, int32_t x_rows, const int32_t* rows,
                           const int32_t* offsets, int32_t groups, int32_t out_rows,
                           const msb_group_weights* w, int32_t n, int32_t k, void* out,
                           int32_t out_type, int64_t ldo, void* stream);

/* out[p][j] = silu(sum_i x[row(p)][i] * w[e][0][j][i]) * sum_i x[row(p)][i] * w[e][1][j][i];
 * bf16 out; everything else as msb_grouped_matmul.  silu is within (5 + 1.2 |g|) 2^-23 of its
 * value for gates g down to -87, and zero below -87.4. */
int32_t msb_grouped_swiglu(const void* x, int64_t ldx, int32_t x_rows, const int32_t* rows,
                           const int32_t* offsets, int32_t groups, int32_t out_rows,
                           const msb_group_weights* w, int32_t n, int32_t k, void* out,
                           int64_t ldo, void* stream);

/* ------------------------------------------------------------------ 8-bit integers
 * Rows of x in 8 bits: scale = max |x| / 127, q = the integer nearest to x * (127 / max |x|)
 * (FP32 steps, ties to even).  A row whose largest magnitude is below 2^-119 becomes zeros
 * with scale 0; a row with a NaN or infinity becomes zeros with scale NaN.
 *  x        x_type (MSB_BF16 or MSB_F32), rows ldx elements apart.
 *  q        int8, rows ldq bytes apart (ldq >= k); scale float [rows].
 *  rows 0..; k 1..2^28 - 1. */
int32_t msb_int8_quantize(const void* x, int32_t x_type, int64_t ldx, int32_t rows, int32_t k,
                          int8_t* q, int64_t ldq, float* scale, void* stream);

/* msb_grouped_matmul / msb_grouped_swiglu on 8-bit integers: every product is
 *   (float)(sum_i q[row(p)][i] * w[e][j][i]) * q_scale[row(p)] * w_scale[e][j],
 * the sum exact in int32.  q int8, 16-byte aligned, ldq a multiple of 16; w int8 with
 * stride_k = 1; w_scale float [groups][n] (SwiGLU: [groups][2][n]); k <= MSB_INT8_MAX_K. */
int32_t msb_int8_matmul(const int8_t* q, int64_t ldq, const float* q_scale, int32_t x_rows,
                        const int32_t* rows, const int32_t* offsets, int32_t groups,
                        int32_t out_rows, const msb_group_weights* w, const float* w_scale,
                        int32_t n, int32_t k, void* out, int32_t out_type, int64_t ldo,
                        void* stream);
int32_t msb_int8_swiglu(const int8_t* q, int64_t ldq, const float* q_scale, int32_t x_rows,
                        const int32_t* rows, const int32_t* offsets, int32_t groups,
                        int32_t out_rows, const msb_group_weights* w, const float* w_scale,
                        int32_t n, int32_t k, void* out, int64_t ldo, void* stream);

/* msb_int8_quantize of x, then msb_int8_matmul (swiglu = 0) or msb_int8_swiglu (swiglu = 1,
 * out_type MSB_BF16): the same results.  workspace: msb_int8_linear_workspace_size(x_rows, k)
 * bytes (at least 16; 0 for sizes out of range), 16-byte aligned, no initial contents needed;
 * must not overlap x or out. */
size_t msb_int8_linear_workspace_size(int32_t x_rows, int32_t k);
int32_t msb_int8_linear(const void* x, int32_t x_type, int64_t ldx, int32_t x_rows,
                        const int32_t* rows, const int32_t* offsets, int32_t groups,
                        int32_t out_rows, const msb_group_weights* w, const float* w_scale,
                        int32_t n, int32_t k, int32_t swiglu, void* out, int32_t out_type,
                        int64_t ldo, void* workspace, size_t workspace_bytes, void* stream);

/* ------------------------------------------------------------------ combine
 * out[t] = sum over k of weights[t][k] * y[pos[t][k]], in the order of k, in FP32, rounded
 * once; pairs whose pos is outside 0..y_rows-1 are left out (a token without any: zeros).
 *  y        y_type (MSB_BF16 or MSB_F32) [y_rows], rows ldy elements apart.
 *  out      bf16 [tokens], rows ldo elements apart; must not overlap y.
 *  tokens 0..; top_e, d 1..2^28 - 1, and below 2^31 blocks: tokens * ceil(d / 256) < 2^31 is
 *  enough (MSB_EUNSUPPORTED else). */
int32_t msb_combine(const void* y, int32_t y_type, int64_t ldy, int32_t y_rows, const int32_t* pos,
                    const float* weights, int32_t tokens, int32_t top_e, int32_t d, void* out,
                    int64_t ldo, void* stream);

/* ------------------------------------------------------------------ block norm
 * The glue around a block: the norm after it, its gate, the residual scale, and the norm
 * before the next one.  With rms(v) = v / sqrt(mean(v^2) + eps), per row:
 *   b = post_norm ? rms(y) * post_weight : y
 *   h' = skip_scale * h + residual_scale * gate * b
 *   x = rms(h') * pre_weight
 * in FP32; h' is rounded once to h_type when stored, x once to bf16 (from the unrounded h').
 *  h        h_type (MSB_BF16 or MSB_F32), rows ldh elements apart.
 *  y        y_type, rows ldy apart, or NULL: h' = skip_scale * h.
 *  pre_weight, post_weight  weight_type [d], or NULL: ones.
 *  gate     gate_type, element (t, i) at gate + t * gate_row + i * gate_col elements (strides
 *           >= 0: 0 broadcasts), or NULL: ones.
 *  h_out    h_type, rows ldh_out apart; may be h itself (same pitch); NULL: h' is not stored.
 *  x        bf16, rows ldx apart, or NULL: not computed (h_out and x must not both be NULL).
 * Outputs must not overlap inputs or each other, but for h_out = h.
 *  rows 0..; d 1..MSB_NORM_MAX_D. */
int32_t msb_block_norm(const void* h, int32_t h_type, int64_t ldh, const void* y, int32_t y_type,
                       int64_t ldy, const void* pre_weight, const void* post_weight,
                       int32_t weight_type, int32_t post_norm, const void* gate,
                       int32_t gate_type, int64_t gate_row, int64_t gate_col, float skip_scale,
                       float residual_scale, float eps, void* h_out, int64_t ldh_out, void* x,
                       int64_t ldx, int32_t rows, int32_t d, void* stream);

/* ------------------------------------------------------------------ the dense block
 * out[t] = sum over the top_e routed experts e of w_te * down_e (silu(gate_e x_t) * up_e x_t),
 * routed by the softmax over x_t W_router as moe_sparse_block (msb_route's rules).  What
 * moe_sparse_block computes with k = I and rank 0, for any number of tokens: dims->rank is
 * not used.  The hidden values, the 8-bit form's inputs and the experts' output rows are
 * rounded to bf16 between the products.
 *  x        bf16 [tokens][d], 16-byte aligned; out bf16 [tokens][d], must not overlap x.
 *  mask     optional uint8 [tokens]: tokens with mask 0 take no part and get zeros.
 *  router_t, records: packed weights (msb_pack).
 *  gate_up  int8 [E][2][I][d] and gate_up_scale float [E][2][I]; down int8 [E][d][Ipad] (Ipad =
 *           I rounded up to 16; the padding is not read) and down_scale float [E][d].
 *  workspace: msb_dense_workspace_size bytes, 16-byte aligned, no initial contents needed. */
size_t msb_dense_workspace_size(const msb_dims* dims, int32_t tokens, int32_t int8);
int32_t moe_dense_block(const void* x, int32_t tokens, const uint8_t* mask, const void* router_t,
                        const void* records, void* out, const msb_dims* dims, void* workspace,
                        size_t workspace_bytes, void* stream);
int32_t moe_dense_block_int8(const void* x, int32_t tokens, const uint8_t* mask,
                             const void* router_t, const int8_t* gate_up,
                             const float* gate_up_scale, const int8_t* down,
                             const float* down_scale, void* out, const msb_dims* dims,
                             void* workspace, size_t workspace_bytes, void* stream);

#ifdef __cplusplus
} /* extern "C" */
#endif

#endif /* MSB_DENSE_H_ */

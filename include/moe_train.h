/*
 * moe_train.h - the part of libmoe's C ABI that a training step of the MoE
 * expert layer needs beside moe.h: the router with its balance loss, the
 * combine over partly routed tokens and its backward pass, the expert
 * activation with an MXFP8 checkpoint of its input, and the weight gradient
 * over MXFP8 rows. The conventions of moe.h hold for every entry point here
 * (caller-owned device memory, host validation before any launch, nothing
 * allocated or synchronized, MOE_* status codes, slot s = t * top_k + j).
 * Ranges "overlap" when they share a byte: matrices may be columns of one
 * buffer, and an array may lie in a gap between rows. Only matrices whose row
 * strides differ in bytes must lie apart, from their first byte to their last.
 *
 * One step of a layer, forward:
 *   moe_route -> moe_align -> moe_grouped_gemm (no epilogue) -> moe_act_mxfp8
 *   -> moe_grouped_gemm (a_row_div 1) -> moe_combine_routed
 * keeping x as MXFP8 (moe_quantize_mxfp8) and the checkpoint; backward:
 *   moe_combine_backward -> moe_grouped_gemm with W2^T -> moe_act_mxfp8_backward
 *   -> moe_wgrad (second weights) and moe_wgrad_mxfp8 (first weights)
 *   -> moe_grouped_gemm with W1^T -> moe_combine_routed, and moe_route_backward.
 */
#ifndef MOE_TRAIN_H
#define MOE_TRAIN_H

#include "moe.h"

#ifdef __cplusplus
extern "C" {
#endif

/* How the router turns logits into scores. */
typedef enum {
  MOE_SCORE_SOFTMAX = 0,
  MOE_SCORE_SIGMOID = 1
} moe_score;

/* ------------------------------------------------------------------------
 * The router: top-k experts, their weights, and the balance statistics.
 * For every token t with token_mask[t] != 0 (every token without a mask) and
 * at least one logit other than -inf (a "routed" token), with z = logits[t]:
 *   a = z (softmax) or log sigmoid(z) (sigmoid);  q = softmax(a) over E
 *   topk_ids[t][0..k) = the top_k experts by z, largest first, equal logits
 *                       lowest expert first; -inf logits (masked experts)
 *                       and NaN are never chosen, places left over hold -1
 *   topk_w[t][j] = scale * v_j, with for the chosen experts i_j
 *     renormalize: v_j = exp(a[i_j]) / sum over the chosen of exp(a[i])
 *     otherwise:   v_j = q[i_j] (softmax) or sigmoid(z[i_j]) (sigmoid)
 *   topk_w of a place holding -1 is 0.
 * Every other token (padding): ids -1, weights 0, its logits not read when
 * masked. Such slots are routed nowhere by moe_align, the grouped GEMMs,
 * moe_combine_routed and moe_combine_backward.
 * Over the n routed tokens (the statistics, computed when stats is not 0):
 *   counts[e]   = number of slots routed to e   (int32)
 *   num_routed  = n                              (int32)
 *   prob_sum[e] = sum_t q[t][e]                  (fp32)
 *   losses[0]   = E / (top_k n^2) * sum_e counts[e] * prob_sum[e]: the balance
 *                 loss E * sum_e f_e P_e with f_e the share of slots and P_e
 *                 the mean probability of expert e; 1 when balanced
 *   losses[1]   = (1/n) sum_t (log sum_e exp z[t][e])^2 for softmax scores, 0
 *                 for sigmoid scores;  both 0 when n = 0.
 * A NaN logit, or +inf with softmax scores, makes its token's q NaN, which
 * reaches prob_sum, the losses and, for softmax scores without
 * renormalization, all its weights. The other weights depend on the chosen
 * experts' logits alone, which are never NaN; a chosen +inf makes renormalized
 * softmax weights NaN.
 *
 * logits (device) MOE_FP32 or MOE_BF16 [T][E], row stride logits_ld elements;
 * token_mask (device) uint8 [T] or NULL; topk_ids (device) int32 [T][top_k];
 * topk_w (device) fp32 [T][top_k]. Scores, sums and weights are fp32; the
 * sums over tokens run in one fixed order, so repeated calls give equal bits.
 * Without statistics the four outputs and workspace may be NULL.
 * workspace (device, 8-byte aligned): moe_route_workspace_bytes(T, E) bytes,
 * not kept between calls; calls that may run at the same time (other streams,
 * graphs replayed side by side) each need their own.
 * Requirements: 1 <= num_experts <= 1024; 1 <= top_k <= min(num_experts, 64);
 * logits_ld >= num_experts; num_tokens * top_k <= 2^31 - 2^16 (as moe_align);
 * finite scale; pointers aligned to their elements; outputs and workspace must
 * not overlap each other or the inputs. */
moe_status moe_route(const void* logits, int32_t logits_dtype, int64_t logits_ld, const uint8_t* token_mask,
                     int64_t num_tokens, int32_t num_experts, int32_t top_k, int32_t score, int32_t renormalize,
                     float scale, int32_t* topk_ids, float* topk_w, int32_t stats, int32_t* counts,
                     int32_t* num_routed, float* prob_sum, float* losses, void* workspace,
                     int64_t workspace_bytes, moe_stream_t stream);

/* Bytes of moe_route's workspace with statistics; -1 on bad sizes. */
int64_t moe_route_workspace_bytes(int64_t num_tokens, int32_t num_experts);

/* The router's gradient: dlogits = d(sum dtopk_w * topk_w + dlosses . losses) / dlogits,
 * the chosen experts (topk_ids, counts, num_routed, as moe_route wrote them)
 * held constant. With g_j = scale * dtopk_w[t][j], v_j as above and
 *   u_j = v_j (g_j - sum_m g_m v_m) (renormalized) or v_j g_j,
 *   U   = sum_j u_j for softmax scores without renormalization, else 0,
 *   c_e = dlosses[0] * E / (top_k n^2) * counts[e],
 *   da[e] = q_e (c_e - sum_i q_i c_i + 2 dlosses[1] lse / n - U) + sum_{j: i_j = e} u_j
 * (the lse term for softmax scores only), dlogits[t][e] = da[e] for softmax,
 * da[e] * (1 - sigmoid(z_e)) for sigmoid scores.
 * Every row of dlogits is written (in logits' type, rounded once); a token
 * whose first id is negative gets zeros, whatever its logits hold. Ids
 * outside [0, E) past the first contribute nothing; an expert named twice gets
 * both terms.
 * dtopk_w (device) fp32 [T][top_k]; entries at ids of -1 are ignored. dlosses
 * (device) fp32 [2] or NULL (no losses; counts and num_routed may then be
 * NULL). dlogits must not overlap the inputs. Requirements as for moe_route;
 * dlogits_ld >= num_experts. No workspace. */
moe_status moe_route_backward(const void* logits, int32_t logits_dtype, int64_t logits_ld, int64_t num_tokens,
                              int32_t num_experts, int32_t top_k, int32_t score, int32_t renormalize, float scale,
                              const int32_t* topk_ids, const float* dtopk_w, const int32_t* counts,
                              const int32_t* num_routed, const float* dlosses, void* dlogits, int64_t dlogits_ld,
                              moe_stream_t stream);

/* ------------------------------------------------------------------------
 * moe_combine over tokens some of whose slots are routed nowhere:
 *   y[t][n] = bf16( sum_{j < top_k, 0 <= topk_ids[t][j] < E, ascending} topk_w[t][j] * C[t*top_k + j][n] )
 * in fp32. The other slots' rows of C (which the grouped GEMM leaves as they
 * were) and weights are not read; a token without a routed slot gets zeros.
 * topk_ids (device) int32 [T][top_k]; everything else as for moe_combine,
 * whose bits this gives when every slot is routed; y must not overlap the
 * inputs. */
moe_status moe_combine_routed(const void* c, int64_t c_ld, const float* topk_w, const int32_t* topk_ids,
                              int64_t num_tokens, int32_t top_k, int32_t num_experts, int64_t n, void* y,
                              int64_t y_ld, moe_stream_t stream);

/* ------------------------------------------------------------------------
 * Backward pass of the combine. For every slot s = t * top_k + j that is
 * routed (topk_ids NULL, or 0 <= topk_ids[s] < num_experts):
 *   dC[s][n]   = bf16( topk_w[s] * dy[t][n] )
 *   dtopk_w[s] = sum_n dy[t][n] * C[s][n]   (fp32, one fixed order)
 * An unrouted slot gets a dC row of zeros and dtopk_w 0; its row of C is not
 * read. dy (device) bf16 [T][n]; c, dc (device) bf16 [T*top_k][n]; topk_w,
 * dtopk_w (device) fp32 [T][top_k]. Every row and weight is written. dc and
 * dtopk_w must not overlap the inputs or each other. num_experts is read with
 * topk_ids only.
 * n % 8 == 0; dy_ld, c_ld, dc_ld >= n and multiples of 8; dy, c, dc 16-byte
 * aligned. No workspace. */
moe_status moe_combine_backward(const void* dy, int64_t dy_ld, const void* c, int64_t c_ld, const float* topk_w,
                                const int32_t* topk_ids, int64_t num_tokens, int32_t top_k, int32_t num_experts,
                                int64_t n, void* dc, int64_t dc_ld, float* dtopk_w, moe_stream_t stream);

/* ------------------------------------------------------------------------
 * The expert activation with an 8-bit checkpoint of its input. For every row
 * r < rows of pre (the first GEMM's output, bf16, width n):
 *   h[r] = bf16( act(pre[r]) ), act MOE_EPILOGUE_SWIGLU (width n / 2) or
 *          MOE_EPILOGUE_RELU2 (width n), the formulas of moe_grouped_gemm's
 *          epilogues (SwiGLU not bit for bit: that one divides)
 *   q[r], scales[r] = moe_quantize_mxfp8 of pre[r]
 * so a training step keeps n (1 + 1/32) bytes a row for the backward pass in
 * place of 2n for pre and more for h. Rows are independent; rows that no slot
 * uses may hold anything.
 * pre, h bf16; q uint8; scales uint8, with row strides pre_ld, h_ld
 * (elements), q_ld, scales_ld (bytes).
 * Requirements: n a positive multiple of 32 (64 for SwiGLU: both halves are
 * whole blocks); pre_ld >= n, h_ld >= the width of h, multiples of 8;
 * q_ld >= n, a multiple of 16; scales_ld >= n / 32; pre, h, q 16-byte
 * aligned. Outputs must not overlap pre or each other. No workspace. */
moe_status moe_act_mxfp8(int32_t act, const void* pre, int64_t pre_ld, int64_t rows, int64_t n, void* h, int64_t h_ld,
                         void* q, int64_t q_ld, uint8_t* scales, int64_t scales_ld, moe_stream_t stream);

/* Its backward pass from the checkpoint: v = dec(q) * 2^(scale - 127), and
 *   dpre[r] = bf16( dh[r] * act'(v) ),  h[r] = bf16( act(v) ) when h != NULL:
 *   SwiGLU, v = (g, u), s = sigmoid(g): dg = dh u s (1 + g (1 - s)), du = dh g s
 *   squared ReLU: dv = 2 max(v, 0) dh
 * h is what the second weights' gradient (moe_wgrad) reads. A NaN block
 * (scale byte 0xFF) gives NaN for SwiGLU and for squared ReLU as the GEMM's
 * epilogue treats NaN (0). Layouts and requirements as above, dh and h
 * with the width of h, dpre with n. Outputs must not overlap inputs. */
moe_status moe_act_mxfp8_backward(int32_t act, const void* q, int64_t q_ld, const uint8_t* scales, int64_t scales_ld,
                                  const void* dh, int64_t dh_ld, int64_t rows, int64_t n, void* dpre, int64_t dpre_ld,
                                  void* h, int64_t h_ld, moe_stream_t stream);

/* ------------------------------------------------------------------------
 * moe_wgrad over MXFP8 activations (moe_quantize_mxfp8's codes and scales,
 * the form in which a training step keeps them):
 *   dW[e][n][k] = sum_{slots s routed to e} grad[s][n] * xhat[s / top_k][k]
 *   xhat[t][k] = dec(xq[t][k]) * 2^(xs[t][k / 32] - 127)
 * in fp32, xhat exact in bf16 (values below bf16's subnormal range round to
 * zero). xq (device) uint8 E4M3 [T][K], row stride xq_ld bytes, a multiple of
 * 16, 16-byte aligned; xs (device) uint8 E8M0 [T][K/32], row stride xs_ld
 * bytes >= K / 32. dw must not overlap the inputs. Everything else as for
 * moe_wgrad. No workspace. */
moe_status moe_wgrad_mxfp8(const void* xq, int64_t xq_ld, const uint8_t* xs, int64_t xs_ld, const void* grad,
                           int64_t grad_ld, const int32_t* sorted_token_ids, const int32_t* expert_ids,
                           const int32_t* num_tokens_post_pad, int64_t num_tokens, int32_t top_k,
                           int32_t num_experts, int64_t n, int64_t k, int32_t block_m, int64_t max_blocks, float* dw,
                           moe_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_TRAIN_H */

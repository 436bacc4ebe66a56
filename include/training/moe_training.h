/*
 * moe_training.h — C ABI of the gradients of the routed expert path on MI355X (gfx950):
 *
 *   moe_silu_mul_dropout    SiLU(gate) * up with dropout from a counter-based generator
 *   moe_silu_mul_backward   its backward, with the router weight of the row
 *   moe_grouped_gemm_dgrad  grouped products for the gradients of the experts' inputs
 *   moe_grouped_gemm_wgrad  grouped products for the gradients of the experts' weights
 *   moe_route_backward      gradient of the router's logits
 *
 * The conventions of moe_mi355x.h hold here as well: device pointers owned by the caller and 16-byte
 * aligned, row-major contiguous layouts, bf16 as uint16_t bit patterns, no allocation, no
 * synchronisation, work on `stream` only, launches that depend on host scalars only (so that every
 * call can be captured in a HIP graph), host-checkable arguments checked before anything is enqueued.
 * No result depends on the order in which workgroups finish.
 *
 * With x [T, H], pairs p = t * top_k + j in the sorted layout of moe_align and w[p] the router weight,
 * a layer's training step is
 *   g, u = x Wg^T, x Wu^T           moe_grouped_gemm(MOE_OP_GATHER), bf16 [max_pad, I]
 *   h = SiLU(g) * u * mask          moe_silu_mul_dropout
 *   out = combine(h Wd^T, w)        moe_grouped_gemm(MOE_OP_DOWN), moe_combine
 * and its backward, from d_out [T, H],
 *   d = d_out Wd                    moe_grouped_gemm_dgrad, d_out by token: the gradient of h before w
 *   dg, du, w h, dw                 moe_silu_mul_backward
 *   dWd = d_out^T (w h)             moe_grouped_gemm_wgrad, d_out by token
 *   dWg, dWu = dg^T x, du^T x       moe_grouped_gemm_wgrad, x by token
 *   dx = dg Wg + du Wu              moe_grouped_gemm_dgrad with two pairs, then moe_combine with weights 1
 *   dlogits                         moe_route_backward
 * The expert outputs are not needed for it: dw[p] = d_out[t] . (h Wd^T) = (d_out[t] Wd) . h.
 */
#ifndef MOE_TRAINING_H
#define MOE_TRAINING_H

#include "../moe_mi355x.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Dropout.  A hidden value of pair p and column c is dropped (0) or kept and multiplied by 1 / (1 - p_drop).
 * The decision is a function of (seed, offset, p, c) alone, computed again by the backward and never stored:
 *   words[4] = Philox 4x32-10, key = seed (low word first), counter = (c / 8, p, offset low, offset high)
 *   r = 16 bits of words[(c % 8) / 2]: the low half for even c, the high half for odd c
 *   kept when r >= round(65536 * p_drop), capped at 65535
 * so p_drop is taken to a multiple of 2^-16, and the factor is 1 / (1 - that multiple).
 * `rng` holds seed and offset (two int64) in device memory, so that a captured graph can be replayed with
 * other numbers; the backward has to find what the forward found.  Steps use different offsets. */

/* h[r] = bf16(SiLU(gate[r]) * up[r] * mask), in fp32, for the rows r with sorted_ids[r] in [0, num_pairs); other
 * rows are not written.  Without sorted_ids every row r is pair r.
 *   gate, up, out  bf16 [rows, n]; out may be gate or up, else it is apart from both
 *   p_drop         in [0, 1); rng may be NULL where it is 0
 * n % 8 == 0, rows * n up to 2^35 (MOE_EUNSUPPORTED above).  rows == 0, or num_pairs == 0 with sorted_ids,
 * enqueues nothing. */
moe_status moe_silu_mul_dropout(const uint16_t* gate, const uint16_t* up, uint16_t* out, const int32_t* sorted_ids,
                                int64_t num_pairs, int64_t rows, int32_t n, double p_drop, const int64_t* rng,
                                moe_stream stream);

/* Backward of moe_silu_mul_dropout for rows whose result is multiplied by a router weight later on:
 * d [rows, n] is the gradient of the row's h for weight 1 (d_out[t] Wd), w[p] the weight of the row's pair.
 *   h          = SiLU(g) * u * mask
 *   d_gate     = bf16(w * d * mask * u * sigmoid(g) * (1 + g * (1 - sigmoid(g))))
 *   d_up       = bf16(w * d * mask * SiLU(g))
 *   h_weighted = bf16(w * h)            the x of moe_grouped_gemm_wgrad for the down projection
 *   d_topk_w[p] = sum over columns of d * h, in fp32, h not rounded
 *   topk_w fp32 [num_pairs]; without sorted_ids every row r is pair r, and num_pairs >= rows.
 * Each of d_gate, d_up and h_weighted may be one of gate, up and d, else it is apart from them; the outputs are
 * apart from each other.
 * Rows without a pair are not written, nor are the d_topk_w of pairs without a row (an expert id out of
 * range).  n % 8 == 0, rows below 2^24 (MOE_EUNSUPPORTED above).  rows == 0, or num_pairs == 0 with sorted_ids,
 * enqueues nothing. */
moe_status moe_silu_mul_backward(const uint16_t* gate, const uint16_t* up, const uint16_t* d, const float* topk_w,
                                 const int32_t* sorted_ids, int64_t num_pairs, int64_t rows, int32_t n,
                                 double p_drop, const int64_t* rng, uint16_t* d_gate, uint16_t* d_up,
                                 uint16_t* h_weighted, float* d_topk_w, moe_stream stream);

/* dx[r, k] = sum_n dy0(r, n) * W0[e, n, k] (+ dy1(r, n) * W1[e, n, k]) for every real sorted row r of every expert
 * e: the gradient of the input of y = x W^T.  Exact bf16 products, fp32 sums, one rounding to bf16.
 *   dy0, dy1   bf16 [max_pad, N] by sorted row, or (by_token) [num_pairs / top_k, N] by token
 *   w0, w1     MOE_W_BF16 weights [E, N, K]; w1 and dy1 are NULL without a second pair
 *   dx         bf16 [max_pad, K], apart from every operand; sentinel and padding rows are not written
 * N and K multiples of 8, up to 2^20, num_experts <= 256, max_pad < 2^31 - 1024 (MOE_EUNSUPPORTED above).
 * workspace: NULL, or one of moe_grouped_gemm (the same buffer, zero-filled before its first use; every call
 * leaves its counters at zero; calls that share one must not overlap).  With it, launches of few tiles divide
 * the sum over n among workgroups.  num_pairs == 0 enqueues nothing. */
moe_status moe_grouped_gemm_dgrad(const uint16_t* dy0, const moe_weight* w0, const uint16_t* dy1, const moe_weight* w1,
                                  uint16_t* dx, const int32_t* sorted_ids, const int32_t* expert_offsets,
                                  int64_t num_pairs, int32_t top_k, int32_t num_experts, int32_t n, int32_t k,
                                  int32_t block_size, int64_t max_pad, int32_t by_token, void* workspace,
                                  int64_t workspace_bytes, moe_stream stream);

/* dw[e, n, k] = base[e, n, k] + sum over the real sorted rows r of expert e of dy(r, n) * x(r, k): the gradient of
 * the weights of y = x W^T.  Exact bf16 products, fp32 sums.  Experts without rows get base, or zeros.
 *   dy         bf16 [max_pad, N] by sorted row, or (dy_by_token) [num_pairs / top_k, N] by token
 *   x          bf16 [max_pad, K] by sorted row, or (x_by_token) [num_pairs / top_k, K] by token
 *   dw         [E, N, K], bf16 (one rounding, after base is added) or, with dw_fp32, fp32; apart from dy and x
 *   base       NULL, or of dw's type and shape; dw (gradients summed over batches), or apart from it
 * N and K multiples of 8, up to 2^20, num_experts <= 256, max_pad < 2^31 - 1024 (MOE_EUNSUPPORTED above).  workspace: as for
 * moe_grouped_gemm_dgrad; with it, launches of few tiles divide long sums over rows among workgroups.
 * num_pairs == 0 writes base or zeros. */
moe_status moe_grouped_gemm_wgrad(const uint16_t* dy, const uint16_t* x, void* dw, const void* base, int32_t dw_fp32,
                                  const int32_t* sorted_ids, const int32_t* expert_offsets, int64_t num_pairs,
                                  int32_t top_k, int32_t num_experts, int32_t n, int32_t k, int32_t block_size,
                                  int64_t max_pad, int32_t dy_by_token, int32_t x_by_token, void* workspace,
                                  int64_t workspace_bytes, moe_stream stream);

/* Gradient of the router's logits from that of the weights that moe_route returned, in fp64, rounded to fp32:
 *   logits NULL (weights renormalised over the chosen):
 *     d_logits[t, ids[t, j]] = w_j * (d_w_j - sum_i w_i d_w_i), 0 for the experts not chosen
 *   logits fp32 [T, E] (not renormalised), p = softmax(logits[t]):
 *     d_logits[t, e] = p_e * (sum of d_w_j with ids[t, j] == e - sum_i w_i d_w_i)
 *   topk_ids i32, topk_w and d_topk_w fp32 [T, top_k]; pairs with an id outside [0, E) count as d_w = 0, and
 *   their d_topk_w is not read
 *   d_logits fp32 [T, E], every entry written; apart from topk_ids, topk_w and d_topk_w (where top_k == E it may
 *   be one of them), and logits or apart from it
 * num_experts and top_k <= 256 (MOE_EUNSUPPORTED above).  num_tokens == 0 enqueues nothing. */
moe_status moe_route_backward(const int32_t* topk_ids, const float* topk_w, const float* d_topk_w,
                              const float* logits, int32_t num_tokens, int32_t num_experts, int32_t top_k,
                              float* d_logits, moe_stream stream);

#ifdef __cplusplus
}
#endif
#endif /* MOE_TRAINING_H */

/*
 * megamoe/half.h -- C ABI of the unquantised experts of the MegaMoE pipeline, in fp16
 * or bf16, and of what training takes: the gradients of the products, of SwiGLU and
 * of the router, and the norms around the layer with theirs.
 *
 * The conventions, dims, limits, types and errors are those of megamoe.h.  `type` is
 * MEGAMOE_FP16 or MEGAMOE_BF16, one for all 16-bit tensors of a call; sums and
 * statistics are in fp32 and rounded once, at the end.  (In the products' sums a
 * subnormal fp16 value counts, to the accuracy that 2^-14 in its place would have.)
 * No result depends on timing.  Rows of the expert-major order at and past the last
 * element of expert_cumsum are left as they are.  Weights are rows over the forward's
 * reduction, with no further layout:
 *   w1 [E, 2I, K]  rows [0, I) feed silu, [I, 2I) the gate
 *   w2 [E, K, I]
 */
#ifndef MEGAMOE_HALF_H_
#define MEGAMOE_HALF_H_

#include "../megamoe.h"

#ifdef __cplusplus
extern "C" {
#endif


/* The sort of megamoe_permute alone: its index outputs, no quantised rows.
 * workspace >= megamoe_permute_workspace_bytes(); megamoe_last_error reads the
 * dropped routes from it. */
int megamoe_sort_routes(const megamoe_dims *d, const int32_t *expert_idx,
                        int32_t *expanded_row_idx, int32_t *sorted_route,
                        int32_t *tokens_per_expert, int32_t *expert_cumsum, void *workspace,
                        size_t workspace_bytes, void *stream);

/* The grouped products.  For sorted row d of expert e's group, of route
 * q = sorted_route[d] and token t = q / top_k:
 *   megamoe_half_gmm1         c[d, n] = sum_k x[t, k] w1[e, n, k]
 *   megamoe_half_gmm1_swiglu  y[d, i] = probs[q] silu(c[d, i]) c[d, I + i], with c in fp32
 *                             (probs nullable: 1)
 *   megamoe_half_gmm2         gmm2_out[d, k] = sum_i y[d, i] w2[e, k, i]
 *   x [M, K], c [R, 2I], y [R, I], gmm2_out [R, K]
 * The route's weight is applied to y, so a token's output is the plain sum of
 * its rows of gmm2_out (megamoe_norm with rows alone). */
int megamoe_half_gmm1(const megamoe_dims *d, const uint16_t *x, int type,
                      const int32_t *sorted_route, const int32_t *expert_cumsum,
                      const uint16_t *w1, uint16_t *c, void *stream);
int megamoe_half_gmm1_swiglu(const megamoe_dims *d, const uint16_t *x, int type,
                             const int32_t *sorted_route, const int32_t *expert_cumsum,
                             const float *probs, const uint16_t *w1, uint16_t *y, void *stream);
int megamoe_half_gmm2(const megamoe_dims *d, const uint16_t *y, int type,
                      const int32_t *expert_cumsum, const uint16_t *w2, uint16_t *gmm2_out,
                      void *stream);

/* Gradients of the products' rows, from those of their results:
 *   megamoe_half_gmm1_dgrad  dx_rows[d, k] = sum_n dc[d, n] w1[e, n, k]
 *                            (a token's gradient is the sum of its rows)
 *   megamoe_half_gmm2_dgrad  dy[d, i] = sum_k dout[t, k] w2[e, k, i]
 *   dc [R, 2I], dx_rows [R, K], dout [M, K] (that of the tokens' sums), dy [R, I] */
int megamoe_half_gmm1_dgrad(const megamoe_dims *d, const uint16_t *dc, int type,
                            const int32_t *expert_cumsum, const uint16_t *w1, uint16_t *dx_rows,
                            void *stream);
int megamoe_half_gmm2_dgrad(const megamoe_dims *d, const uint16_t *dout, int type,
                            const int32_t *sorted_route, const int32_t *expert_cumsum,
                            const uint16_t *w2, uint16_t *dy, void *stream);

/* Gradients of the weights, over the rows d of each expert:
 *   megamoe_half_gmm1_wgrad  dw1[e, n, k] = sum_d dc[d, n] x[t, k]
 *   megamoe_half_gmm2_wgrad  dw2[e, k, i] = sum_d dout[t, k] y[d, i]
 * dw_type: type or MEGAMOE_FP32.  accumulate nonzero: added to what dw holds (in
 * fp32, then rounded); zero: dw is written, 0 for an expert without rows.  Their
 * limit is (R + 64) * max(K, 2I) < 2^31 (else MEGAMOE_EUNSUPPORTED). */
int megamoe_half_gmm1_wgrad(const megamoe_dims *d, const uint16_t *dc, const uint16_t *x, int type,
                            const int32_t *sorted_route, const int32_t *expert_cumsum, void *dw1,
                            int dw_type, int accumulate, void *stream);
int megamoe_half_gmm2_wgrad(const megamoe_dims *d, const uint16_t *dout, const uint16_t *y,
                            int type, const int32_t *sorted_route, const int32_t *expert_cumsum,
                            void *dw2, int dw_type, int accumulate, void *stream);

/* SwiGLU weighted by the route's probability, as in megamoe_half_gmm1_swiglu but from
 * c as stored, and its gradient: dc [R, 2I], and
 *   dprobs[q] = sum_i dy[d, i] silu(c[d, i]) c[d, I + i], 0 for a route without a row
 * probs nullable (1), dprobs nullable. */
int megamoe_half_swiglu(const megamoe_dims *d, const uint16_t *c, int type,
                        const int32_t *sorted_route, const int32_t *expert_cumsum,
                        const float *probs, uint16_t *y, void *stream);
int megamoe_half_swiglu_grad(const megamoe_dims *d, const uint16_t *c, const uint16_t *dy,
                             int type, const int32_t *sorted_route,
                             const int32_t *expanded_row_idx, const int32_t *expert_cumsum,
                             const float *probs, uint16_t *dc, float *dprobs, void *stream);

/* The norms after and before the layer, with the gate and the residual between:
 *   s[t] = sum over the token's slots of rows[expanded_row_idx[t * top_k + slot]]
 *          (slots without a row are skipped), or rows[t] where expanded_row_idx is null
 *   n    = s / sqrt(mean s^2 + eps) * w_after, or s where w_after is null
 *   r    = x + alpha * gate * n; x null: 0, rows null: r = x, gate null: 1
 *   h    = r / sqrt(mean r^2 + eps) * w_before
 * Each of s, r, h is rounded from fp32 values that were not rounded before; every
 * one may be null (h exactly where w_before is), not all of them.  Squares are in
 * fp32 too: where a row's mean square passes its range (values of some 1e19), the
 * norm of that row is 0.  With rows alone r
 * is the plain combine, with x and w_before alone h is the norm before a layer.
 *   x, r      x_type [M, K]; r may be x's own memory
 *   rows, s   rows_type [R, K] with expanded_row_idx [R], else [M, K]
 *   h         h_type [M, K]
 *   gate      gate_type [gate_rows, gate_cols], broadcast: rows 1 or M, columns 1 or K
 *   w_after, w_before fp32 [K]; eps > 0
 * Reads M, K and top_k of the dims; K <= 32768. */
int megamoe_norm(const megamoe_dims *d, const void *x, int x_type, const void *rows, int rows_type,
                 const int32_t *expanded_row_idx, const float *w_after, const void *gate,
                 int gate_type, int64_t gate_rows, int64_t gate_cols, float alpha,
                 const float *w_before, float eps, void *s, void *r, void *h, int h_type,
                 void *stream);

/* The gradients of megamoe_norm, from s and r as it wrote them and the gradients dr
 * (nullable: 0) and dh of r and h.  dh is [M, K], or with expanded_row_idx [R, K], the
 * gradients of the rows that h was gathered to, which are summed.
 *   dx   x_type [M, K]: the whole gradient of r, which is x's
 *   ds   rows_type [M, K]: that of s, which is every gathered row's; exactly where s is given
 *   dw_after, dw_before fp32 [K], dgate like gate: exactly where w_after, w_before and
 *   gate are given; dh and r exactly where w_before is
 * Sums over tokens have a fixed order.  workspace: device,
 * megamoe_norm_grad_workspace_bytes(), no clearing. */
int megamoe_norm_grad_workspace_bytes(const megamoe_dims *d, size_t *bytes);
int megamoe_norm_grad(const megamoe_dims *d, const void *dr, const void *r, int x_type,
                      const void *dh, int h_type, const int32_t *expanded_row_idx, const void *s,
                      int rows_type, const float *w_after, const void *gate, int gate_type,
                      int64_t gate_rows, int64_t gate_cols, float alpha, const float *w_before,
                      float eps, void *dx, void *ds, float *dw_after, float *dw_before,
                      void *dgate, void *workspace, size_t workspace_bytes, void *stream);

/* The gradient of megamoe_route's probs with respect to its logits, with logits, bias
 * and renormalize as given to it and expert_idx and probs as it wrote them:
 *   dlogits[t, e] = w[e] (g[e] - sum_e w[e] g[e])
 * w: the softmax over the chosen experts or over all that take part; g[e]: dprobs of
 * expert e's slot, 0 where it was not chosen.  0 for an expert that takes no part.
 * Slots whose expert is outside [0, E) are skipped.
 *   dprobs fp32 [M, top_k], dlogits logits_type [M, E] */
int megamoe_route_grad(const megamoe_dims *d, const void *logits, int logits_type,
                       const float *bias, int renormalize, const int32_t *expert_idx,
                       const float *probs, const float *dprobs, void *dlogits, void *stream);

/* The whole layer with 16-bit experts: megamoe_sort_routes, megamoe_half_gmm1_swiglu,
 * megamoe_half_gmm2 and the plain combine of megamoe_norm, the same bits.  x [M, K] and
 * out [M, K] of `type`, expert_idx and probs as in megamoe_forward, dropped routes
 * through megamoe_last_error. */
int megamoe_half_workspace_bytes(const megamoe_dims *d, size_t *bytes);
int megamoe_forward_half(const megamoe_dims *d, const uint16_t *x, int type,
                         const int32_t *expert_idx, const float *probs, const uint16_t *w1,
                         const uint16_t *w2, uint16_t *out, void *workspace,
                         size_t workspace_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* MEGAMOE_HALF_H_ */

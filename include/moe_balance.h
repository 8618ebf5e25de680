/*
 * Balance loss of the router (libmoe, AMD MI355X / gfx950), the counts it is
 * made of, its gradient, and the router's backward from dense logit gradients.
 *
 * With p[t] = softmax(logits[t]) over all E experts, N the number of counted
 * tokens (those whose mask is not 0), c[e] the number of counted tokens that
 * chose e and P[e] the sum of p[t, e] over the counted tokens,
 *   loss = coef * E / (k N^2) * sum_e c[e] P[e],
 * coef for an even load, more for an uneven one. The counts are piecewise
 * constant, the gradient flows through p:
 *   dlogits[t, e] = dloss coef E / (k N^2) p[t, e] (c[e] - sum_i p[t, i] c[i]).
 * All sums are linear in c, P and N: ranks that share a loss add up counts,
 * tokens and prob_sum (all-reduce) and hand the sums to the backward; then
 * each rank's dlogits are the gradients of the loss of the whole batch.
 *
 * Conventions as in moe.h: caller-owned DEVICE memory, work enqueued on
 * `stream`, host-side argument checks before any HIP call, moe_status codes.
 * No output may overlap an input.
 */
#ifndef MOE_BALANCE_H
#define MOE_BALANCE_H

#include "moe.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * moe_balance_loss - counts, probability sums and the loss. Softmax in fp32,
 * sums over tokens in fp32 within a workgroup and fp64 across them, in an
 * order that depends on the sizes alone: the same bits every call.
 *
 *  T        tokens, 0 .. INT32_MAX (0: zero counts, sums and loss)
 *  E, k     1 .. MOE_MAX_EXPERTS, 1 .. min(E, MOE_MAX_TOPK)
 *  dtype    MOE_F32, MOE_BF16 or MOE_F16: that of the logits
 *  logits   [T, E] dtype (those of moe_route or moe_route_typed). -inf is an
 *           expert that is not offered (p = 0); a row of -inf alone adds
 *           nothing to P. Rows that are not counted are not looked at.
 *  topk_idx [T, k] int32; entries outside [0, E) are dropped slots
 *  mask     [T] uint8 | NULL (every token counts)
 *  coef     finite
 *  counts   [E] int32 out, tokens [1] int32 out, prob_sum [E] fp32 out
 *  loss     [1] fp32 out (0 when no token counts)
 *  ws       workspace of at least moe_balance_loss_workspace_size() bytes
 * Errors: INVALID_ARG (sizes, coef, NULL), UNSUPPORTED (dtype, E or k above
 * the limits), WORKSPACE.
 */
moe_status moe_balance_loss(int32_t T, int32_t E, int32_t k, int32_t dtype, const void* logits,
                            const int32_t* topk_idx, const uint8_t* mask, float coef,
                            int32_t* counts, int32_t* tokens, float* prob_sum, float* loss,
                            void* ws, size_t ws_bytes, void* stream);
/* Host arithmetic; 0 for sizes the call rejects. */
size_t moe_balance_loss_workspace_size(int32_t T, int32_t E);

/*
 * moe_balance_loss_backward - the gradient of the logits, dense. With dlogit
 * (the gradient through the routing weights, from moe_combine_backward) each
 * token's values are added at its chosen experts, counted or not, so that
 * dlogits is the router's whole gradient.
 *
 *  T, E, k, dtype, logits, mask, coef   as for moe_balance_loss (k is in the
 *           loss's factor)
 *  dlogit   [T, k] fp32 | NULL (nothing is added)
 *  topk_idx [T, k] int32, looked at with dlogit (NULL without): slots outside
 *           [0, E) add nothing, an expert named twice gets both
 *  counts   [E] int32, tokens [1] int32: of moe_balance_loss (or their sums
 *           over ranks; no token: the balance term is 0)
 *  dloss    [1] fp32 | NULL (1): the gradient of the loss
 *  dlogits  [T, E] fp32 out
 * Errors: as moe_balance_loss.
 */
moe_status moe_balance_loss_backward(int32_t T, int32_t E, int32_t k, int32_t dtype,
                                     const void* logits, const int32_t* topk_idx,
                                     const uint8_t* mask, float coef, const int32_t* counts,
                                     const int32_t* tokens, const float* dloss,
                                     const float* dlogit, float* dlogits, void* stream);

/*
 * moe_router_backward_dense - gradients of logits = x W_r^T from dense dlogits:
 *   dx[t]     = sum_e dlogits[t, e] w_router[e]   (added to dx if accumulate)
 *   dw_router = dlogits^T x
 * with products and sums as exact as fp32's (on the bf16 matrix cores, fp32
 * operands as the sum of three bf16 parts; an infinite operand gives NaN),
 * summed over tokens in an order that depends on the sizes alone.
 *
 *  T, E, D    0 .. INT32_MAX; 1 .. MOE_MAX_EXPERTS; a positive multiple of
 *             64, at most MOE_MAX_WIDTH
 *  dtype      MOE_F32 or MOE_BF16: that of x
 *  dlogits    [T, E] fp32, x [T, D] dtype, w_router [E, D] fp32
 *  accumulate 1: dx += (dx_shared of the shared expert, say), 0: dx =
 *  dx         [T, D] fp32 out | NULL (not wanted)
 *  dw_router  [E, D] fp32 out | NULL (zeros when T is 0)
 *  ws         workspace of at least moe_router_backward_dense_workspace_size()
 *             bytes; may be NULL when dw_router is
 * x, w_router, dx, dw_router and ws are aligned to 16 bytes. Errors:
 * INVALID_ARG (sizes, accumulate, NULL, alignment), UNSUPPORTED (dtype, limits,
 * ceil(T / 64) * (D / 64) of 2^23 or more), WORKSPACE.
 */
moe_status moe_router_backward_dense(int32_t T, int32_t E, int32_t D, int32_t dtype,
                                     const float* dlogits, const void* x, const float* w_router,
                                     int32_t accumulate, float* dx, float* dw_router, void* ws,
                                     size_t ws_bytes, void* stream);
size_t moe_router_backward_dense_workspace_size(int32_t T, int32_t E, int32_t D);

#ifdef __cplusplus
}
#endif

#endif /* MOE_BALANCE_H */

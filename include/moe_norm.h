/*
 * Layer norm in front of the MoE layer (libmoe, AMD MI355X / gfx950) and its
 * gradient. The MoE layer of moe.h takes its hidden states as they are; in a
 * pre-norm block they are the layer norm of the block's input, and the block's
 * input gradient is the layer's, taken back through the norm, plus the
 * residual branch's. (LayerTrain has that block; moe_layer_forward adds the
 * tensor it routes as the residual, which there is the norm's output. Norms
 * without a mean are not covered.)
 *
 * Conventions as in moe.h: caller-owned DEVICE memory, work enqueued on
 * `stream`, host-side argument checks before any HIP call, moe_status codes.
 * `dtype` is a moe_dtype of the activations (MOE_F32 or MOE_BF16); gamma,
 * beta, mean, rstd and the parameter gradients are fp32. Rows may have any
 * width and any alignment their type allows. No output may overlap an input.
 * NaN and infinite values follow the formulas: a row that holds one becomes
 * NaN, other rows do not change.
 */
#ifndef MOE_NORM_H
#define MOE_NORM_H

#include "moe.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * moe_layer_norm - for every row of D values
 *   mean = sum(x) / D,  rstd = 1 / sqrt(sum((x - mean)^2) / D + eps),
 *   y = (x - mean) rstd gamma + beta,
 * in fp32 (the sum of x in fp64, the variance from centred values), y rounded
 * once to nearest even.
 *
 *  rows   >= 0 (0: nothing is done)
 *  D      1 .. MOE_MAX_WIDTH
 *  dtype  MOE_F32 or MOE_BF16
 *  x      [rows, D] dtype
 *  gamma  [D] fp32 | NULL (ones), beta [D] fp32 | NULL (zeros)
 *  eps    >= 0, finite
 *  y      [rows, D] dtype   out
 *  mean   [rows] fp32 | NULL, rstd [rows] fp32 | NULL   out: for the backward
 * Errors: INVALID_ARG (sizes, eps, NULL x or y), UNSUPPORTED (dtype, D above
 * MOE_MAX_WIDTH, rows * D of 2^40 or more).
 */
moe_status moe_layer_norm(int64_t rows, int32_t D, int32_t dtype, const void* x,
                          const float* gamma, const float* beta, float eps, void* y, float* mean,
                          float* rstd, void* stream);

/*
 * moe_layer_norm_backward - gradients of moe_layer_norm. With
 * h = (x - mean) rstd and g = dy gamma, row by row
 *   dx = rstd (g - sum(g) / D - h sum(g h) / D) + dres
 *   dgamma = sum over rows of dy h,  dbeta = sum over rows of dy,
 * in fp32, dx rounded once to nearest even. The sums over rows are taken in
 * a fixed order that depends on the sizes alone: the same bits every call.
 *
 *  x, dy   [rows, D] dtype
 *  gamma   [D] fp32 | NULL (ones)
 *  mean, rstd  [rows] fp32 from moe_layer_norm
 *  dres    [rows, D] dtype | NULL   added to dx (the residual's gradient)
 *  dx      [rows, D] dtype   out
 *  dgamma, dbeta  [D] fp32 | NULL   out (zeros when rows is 0)
 *  ws      workspace of at least moe_layer_norm_backward_workspace_size()
 *          bytes; may be NULL when dgamma and dbeta are
 * Errors: as moe_layer_norm (with rows 0 only dgamma and dbeta are written);
 * WORKSPACE if ws_bytes is smaller.
 */
moe_status moe_layer_norm_backward(int64_t rows, int32_t D, int32_t dtype, const void* x,
                                   const void* dy, const float* gamma, const float* mean,
                                   const float* rstd, const void* dres, void* dx, float* dgamma,
                                   float* dbeta, void* ws, size_t ws_bytes, void* stream);
/* Host arithmetic; 0 for sizes the call rejects. */
size_t moe_layer_norm_backward_workspace_size(int64_t rows, int32_t D);

#ifdef __cplusplus
}
#endif

#endif /* MOE_NORM_H */

/*
 * Optimiser step for the expert matrices (libmoe, AMD MI355X / gfx950): the
 * Newton-Schulz orthogonalisation of a momentum, and the Muon update built on
 * it (K. Jordan et al., "Muon: An optimizer for hidden layers in neural
 * networks", 2024), batched over the experts' stacked matrices.
 *
 * Conventions as in moe.h: caller-owned DEVICE memory, work enqueued on
 * `stream`, host-side argument checks before any HIP call, moe_status codes.
 * The library keeps no state: momentum and workspace are the caller's.
 */
#ifndef MOE_UPDATE_H
#define MOE_UPDATE_H

#include "moe.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Most Newton-Schulz steps of one call. */
#define MOE_MAX_ORTH_STEPS 16

/*
 * n matrices of [rows, cols] values (sizes are arguments of the call), row
 * major: element (i, r, c) is data[i stride + r ld + c]. ld >= cols; with
 * n > 1, stride >= cols, and the matrices must not share elements. So the
 * gate and the up columns of gate_up tensors [n, D, 2I] are two such batches
 * (ld = 2I, stride = 2 D I, the up columns' data I elements further on).
 * Elements between the rows are neither read nor written.
 */
typedef struct {
  void* data;
  int32_t dtype; /* MOE_F32 or MOE_BF16 */
  int64_t ld, stride;
} moe_matrices;

/*
 * moe_orthogonalize - for each matrix G, with m = min(rows, cols),
 *   X_0 = G / (||G||_F + eps)   (transposed when rows > cols, so X is m x max)
 *   A = X X^T;  X <- (3.4445 I - 4.7750 A + 2.0315 A^2) X,   `steps` times,
 * and out = X (transposed back), rounded once. The quintic drives singular
 * values above about 0.01 ||G||_F into [0.68, 1.21] within five steps. A
 * zero matrix gives zeros; a matrix with a NaN or an infinite value gives NaN
 * throughout; the other matrices do not change.
 * Precision: every product runs on the fp16 matrix cores with each fp32 value
 * held as two fp16 parts (within 2^-22 of it), summed in fp32; the Frobenius
 * norm is summed in fp64. Measured against 64 bits, as a share of ||out||_F,
 * for five steps into an fp32 out: 0.6e-6 to 6e-6 where G has full rank, 4e-6 to
 * 1.5e-4 for ranks from 64 down to 1 (fp32 arithmetic, measured the same way:
 * 1.3e-6 to 4e-6, and 3e-6 to 2.6e-4). A bf16 out, whose own rounding is 1.7e-3,
 * takes more of its steps between two products X X^T: up to 1e-5 at full rank.
 * Steps past five: outside the range of a G of low rank every step multiplies
 * rounding errors by 3.4445, in this as in any arithmetic. At ranks 1 and 8 the
 * error is 1e-3 to 4e-3 after 8 steps, 0.1 to 0.6 after 12, and after 16 the
 * result has directions that G does not have.
 *
 *  n      matrices (>= 0; 0: nothing is done), at most 65535
 *  rows, cols   1 .. MOE_MAX_WIDTH; the smaller one at most 32768;
 *         n ceil(rows / 64) ceil(cols / 64) below 2^23
 *  g      dtype MOE_F32 or MOE_BF16
 *  steps  1 .. MOE_MAX_ORTH_STEPS
 *  eps    >= 0, finite (0 makes a zero matrix NaN)
 *  out    dtype MOE_F32 or MOE_BF16; may be g itself (same data, ld, stride
 *         and dtype), otherwise it must not overlap g
 *  ws     workspace of at least moe_orthogonalize_workspace_size() bytes
 *         (with R, C and M the sizes rows, cols and m rounded up to multiples
 *         of 32: at most 12 n R C + 20 n M^2 + 8 n KB, for m up to 128 at most
 *         12 n R C + the larger of 26 MB and 96 n KB; thin matrices take far
 *         more than their values), 256-byte aligned
 * Errors: INVALID_ARG (sizes, NULL pointers, ld, stride, eps, steps, a
 * misaligned ws), UNSUPPORTED (dtype, sizes past the limits), WORKSPACE.
 */
moe_status moe_orthogonalize(int32_t n, int32_t rows, int32_t cols, const moe_matrices* g,
                             int32_t steps, float eps, const moe_matrices* out, void* ws,
                             size_t ws_bytes, void* stream);
/* Bytes for moe_orthogonalize and moe_muon_update; host arithmetic; 0 for
 * sizes the calls reject. */
size_t moe_orthogonalize_workspace_size(int32_t n, int32_t rows, int32_t cols, int32_t steps);

/*
 * Scalars of moe_muon_update. lr, mu, weight_decay and scale are finite;
 * they are read by the host during the call, so a captured graph keeps the
 * ones it was captured with.
 */
typedef struct {
  float lr;           /* learning rate                                        */
  float mu;           /* momentum                                             */
  float weight_decay; /* decoupled: w shrinks by lr weight_decay              */
  float scale;        /* factor of the orthogonal update (for instance
                         0.2 sqrt(max(rows, cols)))                           */
  float eps;          /* as for moe_orthogonalize                             */
  int32_t nesterov;   /* 1: U = G + mu M; 0: U = M                            */
  int32_t steps;      /* Newton-Schulz steps, 1 .. MOE_MAX_ORTH_STEPS         */
} moe_muon_desc;

/*
 * moe_muon_update - one Muon step for each matrix, in place:
 *   M <- mu M + G;  U = G + mu M (nesterov) or M;
 *   W <- (1 - lr weight_decay) W - lr scale O,  O = moe_orthogonalize(U).
 * fp32, with the products of moe_orthogonalize in O, before and in the last one
 * alike; W is rounded once to its type (to nearest even: with bf16 weights, steps
 * below half a unit in W's last place leave W as it is). A matrix without
 * gradient (G = 0, M = 0) is only decayed.
 *
 *  g         dtype MOE_F32 or MOE_BF16 (LayerTrain's gradients are fp32)
 *  momentum  dtype MOE_F32   in and out
 *  w         dtype MOE_F32 or MOE_BF16   in and out
 *  g, momentum and w must not overlap; each has its own ld and stride.
 *  n, rows, cols, ws  as for moe_orthogonalize
 * Errors: as moe_orthogonalize; INVALID_ARG for a NULL or non-finite desc,
 * UNSUPPORTED for a momentum that is not fp32.
 */
moe_status moe_muon_update(int32_t n, int32_t rows, int32_t cols, const moe_muon_desc* desc,
                           const moe_matrices* g, const moe_matrices* momentum,
                           const moe_matrices* w, void* ws, size_t ws_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_UPDATE_H */

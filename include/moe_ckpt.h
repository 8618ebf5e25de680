/*
 * Activation checkpoints in 8 bits (libmoe, AMD MI355X / gfx950): what a
 * training step keeps from its forward for its backward, in 8.5 bits a value,
 * and the backward of the gated expert layer from it. The fp32 pre-activations
 * G | U that moe_expert_ffn_train keeps are the largest thing a layer holds
 * between the two passes (cap_rows * 2 inter * 4 bytes; here 17/64 of them).
 *
 * Format. Blocks of 32 columns of a row share a scale s =
 * bf16_up(max(amax * fp32(1/127), 2^-126)), amax the largest magnitude in the
 * block, the product in fp32, rounded up to bf16. A value's code is the
 * integer nearest to v * fp32(1/s), ties to even, in -127 .. 127; it comes
 * back as code * s, off by at most s / 2: 1/254 of the block's largest
 * magnitude (and 2^-7 of that from the scale's rounding). The scale is at most
 * 2^121, so that no value becomes infinite, in bf16 neither; with that scale
 * codes are those of v * fp32(127/128 2^-121) and values off by up to 1.5 s. An equal step
 * over the block suits values that are summed into gradients better than a
 * floating-point code, whose step grows with the value: for normally
 * distributed values the error is 0.5 % of the standard deviation, that of
 * E4M3 2.6 %. A block that holds a NaN or an infinity comes back as NaN
 * throughout.
 *
 *   codes [rows, D] int8, scales [rows, D / 32] bf16 (raw 16-bit words)
 *
 * Conventions as in moe.h: caller-owned DEVICE memory, work enqueued on
 * `stream`, host-side argument checks before any HIP call, moe_status codes.
 * No output may overlap an input.
 */
#ifndef MOE_CKPT_H
#define MOE_CKPT_H

#include "moe_backward.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * moe_ckpt_save_rows - x to codes and scales.
 *
 *  rows    >= 0 (0: nothing is done)
 *  D       a positive multiple of 32, at most 2 MOE_MAX_WIDTH
 *  dtype   MOE_F32 or MOE_BF16
 *  x       [rows, D] dtype
 *  codes   [rows, D] int8 out, scales [rows, D / 32] bf16 out
 * x and codes are aligned to 16 bytes. Errors: INVALID_ARG (sizes, NULL,
 * alignment), UNSUPPORTED (dtype, D, rows above INT32_MAX, (rows + 16) * D
 * above 2^34).
 */
moe_status moe_ckpt_save_rows(int64_t rows, int32_t D, int32_t dtype, const void* x, void* codes,
                              void* scales, void* stream);

/*
 * moe_ckpt_restore_rows - out[i] = codes[j] * scales[j] with j = index[i] (i
 * without an index), rounded once to dtype: the rows as they were, or in the
 * order of a permute (index = perm_src: x_perm from the kept x).
 *
 *  n       rows of out, >= 0 (0: nothing is done)
 *  rows    rows of codes; without an index at least n
 *  codes, scales, D   as above
 *  index   [n] int32 | NULL; a row whose index is not in [0, rows) stays as
 *          it was
 *  out     [n, D] dtype out
 * codes and out are aligned to 16 bytes. Errors: as moe_ckpt_save_rows;
 * INVALID_ARG also for n > rows without an index.
 */
moe_status moe_ckpt_restore_rows(int64_t n, int64_t rows, int32_t D, int32_t dtype,
                                 const void* codes, const void* scales, const int32_t* index,
                                 void* out, void* stream);

/*
 * moe_expert_ffn_train_ckpt - moe_expert_ffn_train (bf16 layers) with G | U
 * kept in 8 bits: the same y_perm, bit for bit; the GEMM's epilogue makes the
 * codes from its fp32 accumulators.
 * moe_expert_gate_up_train_ckpt - its first half: h [cap_rows, inter] fp16 as
 * moe_expert_gate_up writes it, and the codes.
 *
 *  gu_codes   [cap_rows, 2 inter] int8 out, gu_scales [cap_rows, 2 inter / 32]
 *             bf16 out (rows past offsets[n] untouched)
 *  other arguments and errors as for moe_expert_ffn_train; codes are aligned
 *  to 16 bytes (INVALID_ARG otherwise)
 */
moe_status moe_expert_ffn_train_ckpt(const moe_desc* desc, int32_t n_experts, int32_t inter,
                                     int64_t cap_rows, const void* x_perm, const int32_t* offsets,
                                     const void* w_gate_up, const void* w_down, void* y_perm,
                                     void* gu_codes, void* gu_scales, void* ws, size_t ws_bytes,
                                     void* stream);
moe_status moe_expert_gate_up_train_ckpt(const moe_desc* desc, int32_t n_experts, int32_t inter,
                                         int64_t cap_rows, const void* x_perm,
                                         const int32_t* offsets, const void* w_gate_up, void* h,
                                         void* gu_codes, void* gu_scales, void* stream);

/*
 * moe_expert_gate_up_backward_ckpt - the adjoint of the gated first layer from
 * the kept G | U: with dH = dY W_down^T (in the accumulators), on the values
 * that the codes stand for,
 *   dG = dH U (s + G s (1 - s)), dU = dH G s, H = G s U,  s = sigmoid(G),
 * dgu = dG | dU [cap_rows, 2 inter] bf16, h [cap_rows, inter] bf16 (rows past
 * offsets[n] untouched). H is that of the kept values, not the forward's.
 * moe_expert_ffn_backward_ckpt - moe_expert_ffn_backward from the kept G | U:
 * the call above, then dx_perm, dw_down and dw_gate_up from dgu and h.
 *
 *  other arguments, workspace size and errors as for moe_expert_ffn_backward;
 *  UNSUPPORTED for fp32 layers; codes are aligned to 16 bytes
 */
moe_status moe_expert_gate_up_backward_ckpt(const moe_desc* desc, int32_t n_experts,
                                            int32_t inter, int64_t cap_rows, const void* dy_perm,
                                            const int32_t* offsets, const void* w_down,
                                            const void* gu_codes, const void* gu_scales,
                                            void* dgu, void* h, void* stream);
moe_status moe_expert_ffn_backward_ckpt(const moe_desc* desc, int32_t n_experts, int32_t inter,
                                        int64_t cap_rows, const void* x_perm,
                                        const int32_t* offsets, const void* w_gate_up,
                                        const void* w_down, const void* dy_perm,
                                        const void* gu_codes, const void* gu_scales,
                                        float* dx_perm, float* dw_gate_up, float* dw_down,
                                        void* ws, size_t ws_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_CKPT_H */

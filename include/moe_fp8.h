/*
 * Expert FFN in FP8 with block scales (libmoe, AMD MI355X / gfx950): the
 * format in which fine-grained MoE weights are distributed, 8-bit codes with
 * one fp32 scale for each 128 x 128 block of a weight matrix, and activations
 * quantized on the way with one fp32 scale for each row and 128 columns.
 * (moe_mxfp8.h is the variant with a power of two for each 32 values.)
 *
 * Format. A block's scale is s = max(amax * fp32(1/448), 2^-126), amax the
 * largest magnitude in the block, products in fp32; a value's code is the
 * E4M3 value (OCP FP8: 3 mantissa bits, no infinities, 448 the largest)
 * nearest to v * fp32(1/s), ties to even. The code stands for code * s. A
 * block of zeros has codes 0. A block that holds a NaN or an infinity comes
 * back as NaN throughout. Codes made elsewhere may use any finite scales whose
 * products (a row's times a weight's) are finite; of a product below 2^-126
 * bits are lost.
 *
 * Layouts (all DEVICE memory, caller-owned; B(n) = ceil(n / 128)):
 *   activation rows   codes [rows, K] uint8, scales [B(K), rows] fp32
 *                     (a block's scales of all rows adjacent)
 *   weights           codes [n, N, K] uint8 (output column c of expert e
 *                     holds its K values contiguously), scales
 *                     [n, B(N), B(K)] fp32: for each expert the weight
 *                     [out, in] and its scales [out/128, in/128]
 * The last block of a dimension may be shorter than 128.
 *
 * Conventions as in moe.h: work enqueued on `stream`, host-side argument
 * checks before any HIP call, moe_status codes. No output may overlap an
 * input.
 */
#ifndef MOE_FP8_H
#define MOE_FP8_H

#include "moe.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * moe_fp8_quantize_rows - activation rows to codes and scales.
 *
 *  rows    >= 0 (0: nothing is done)
 *  K       a positive multiple of 64, at most MOE_MAX_WIDTH
 *  dtype   MOE_F32 or MOE_BF16
 *  x       [rows, K] dtype
 *  codes   [rows, K] uint8 out, scales [B(K), rows] fp32 out
 * Pointers are aligned to 16 bytes. Errors: INVALID_ARG (sizes, NULL,
 * alignment), UNSUPPORTED (dtype, K above MOE_MAX_WIDTH, rows above INT32_MAX,
 * (rows + 16) * K above 2^34).
 */
moe_status moe_fp8_quantize_rows(int64_t rows, int32_t K, int32_t dtype, const void* x,
                                 void* codes, float* scales, void* stream);

/*
 * moe_fp8_pack_weights - stacked expert weights to codes and scales, once,
 * when they are loaded: w [n, K, N] is transposed to [n, N, K] and each
 * 128 x 128 block gets its scale.
 *
 *  n       experts, 0 .. MOE_MAX_EXPERTS
 *  K, N    positive multiples of 64, at most 2 MOE_MAX_WIDTH
 *  dtype   MOE_F32 or MOE_BF16
 *  w       [n, K, N] dtype
 *  codes   [n, N, K] uint8 out, scales [n, B(N), B(K)] fp32 out
 * Errors: as moe_fp8_quantize_rows; UNSUPPORTED also for n above
 * MOE_MAX_EXPERTS and for 2^24 blocks or more.
 */
moe_status moe_fp8_pack_weights(int32_t n, int32_t K, int32_t N, int32_t dtype, const void* w,
                                void* codes, float* scales, void* stream);

/*
 * moe_expert_gate_up_fp8, moe_expert_down_fp8 - the two grouped products of
 * the expert FFN:
 *   h[r, c] = SiLU(x[r] . W_gate[c]) * (x[r] . W_up[c])   (bf16)
 *   y[r, c] = h[r] . W_down[c]             (expert_out_dtype: fp32 or fp16)
 * where a product of codes is
 *   sum over blocks b of xs[b, r] ws[c / 128, b] sum over k in b of xq wq.
 * The 128 products of a block are summed inside the FP8 matrix instruction
 * (exact products; its internal sum keeps some 12 bits below the largest
 * product: the error of a block's sum is at most 2^-10 of the sum of the
 * |products|; measured: 2^-19 in the mean and 2^-15 at most for normally
 * distributed values, 2^-15 and 2^-11.7 for codes spread over the format's whole
 * range), the blocks in fp32. A bf16 result of gate_up or an fp16 one of down
 * so rounds now and then to the neighbour of what fp32 sums would give, and
 * fp32 results carry some 16 bits. fp16 outputs saturate at +-65504.
 *
 *  desc        a bf16 layer (act_dtype MOE_BF16; weight_layout and ep_*
 *              are not looked at)
 *  n_experts, inter, cap_rows, offsets   as for moe_expert_ffn (offsets NULL:
 *              one expert owning all rows)
 *  xq, xs      [cap_rows, D] codes, [B(D), cap_rows] scales
 *  w_gu_q, w_gu_s  gate_up_proj: [n, 2 inter, D], [n, B(2 inter), B(D)]
 *  h           [cap_rows, inter] bf16 out (rows past offsets[n] untouched)
 *  hq, hs      [cap_rows, inter], [B(inter), cap_rows]
 *  w_d_q, w_d_s    down_proj: [n, D, inter], [n, B(D), B(inter)]
 *  y_perm      [cap_rows, D] out (rows past offsets[n] untouched)
 * Codes, h and y_perm are aligned to 16 bytes. Errors: as moe_expert_ffn;
 * INVALID_ARG also for another alignment; UNSUPPORTED for a fp32 layer.
 */
moe_status moe_expert_gate_up_fp8(const moe_desc* desc, int32_t n_experts, int32_t inter,
                                  int64_t cap_rows, const void* xq, const float* xs,
                                  const int32_t* offsets, const void* w_gu_q,
                                  const float* w_gu_s, void* h, void* stream);
moe_status moe_expert_down_fp8(const moe_desc* desc, int32_t n_experts, int32_t inter,
                               int64_t cap_rows, const void* hq, const float* hs,
                               const int32_t* offsets, const void* w_d_q, const float* w_d_s,
                               void* y_perm, void* stream);

/*
 * moe_expert_ffn_fp8 - moe_expert_gate_up_fp8, H (rounded to bf16) quantized
 * as moe_fp8_quantize_rows does, moe_expert_down_fp8: the same bits as the
 * three calls one after another.
 *
 *  ws   workspace of at least moe_ffn_fp8_workspace_size() bytes, aligned to
 *       16 bytes (H, its codes and its scales)
 *  other arguments and errors as above; WORKSPACE if ws_bytes is smaller,
 *  UNSUPPORTED also for (cap_rows + 16) * inter above 2^34
 */
moe_status moe_expert_ffn_fp8(const moe_desc* desc, int32_t n_experts, int32_t inter,
                              int64_t cap_rows, const void* xq, const float* xs,
                              const int32_t* offsets, const void* w_gu_q, const float* w_gu_s,
                              const void* w_d_q, const float* w_d_s, void* y_perm, void* ws,
                              size_t ws_bytes, void* stream);
/* Host arithmetic; 0 for sizes the call rejects. */
size_t moe_ffn_fp8_workspace_size(const moe_desc* desc, int32_t inter, int64_t cap_rows);

#ifdef __cplusplus
}
#endif

#endif /* MOE_FP8_H */

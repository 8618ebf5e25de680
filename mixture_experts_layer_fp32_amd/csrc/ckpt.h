// The arithmetic of the 8-bit activation checkpoints (format in moe_ckpt.h),
// shared by the row kernels and the epilogues of the expert GEMMs.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace moe {

// Scale (bf16 bits) of a block whose largest magnitude has these fp32 bits:
// amax / 127 rounded up to bf16, so that every code fits, at most 2^121: the
// largest value, 127 times that, is then finite in bf16 too. A NaN stays one.
constexpr uint32_t kCkptTopScale = 0x7c00u;  // 2^121
__device__ __forceinline__ uint32_t ckpt_scale_bits(uint32_t amax_bits) {
  const float s = __uint_as_float(amax_bits) * (1.0f / 127.0f);
  const uint32_t b = max(__float_as_uint(s) & 0x7fffffffu, 0x00800000u);
  if (b >= 0x7f800000u) return b > 0x7f800000u ? 0x7fc0u : 0x7f80u;
  return min((b + 0xffffu) >> 16, kCkptTopScale);
}
// The factor r of the codes: 1 / s; with the largest scale 127/128 of it, which
// takes the largest fp32 value to 127.
__device__ __forceinline__ float ckpt_factor(uint32_t scale_bits) {
  const float r = 1.0f / __uint_as_float(scale_bits << 16);
  return scale_bits == kCkptTopScale ? 0x1.fcp-122f : r;
}

// Four codes: the nearest integers to v r, in -127 .. 127 since r <= 127 / amax
// up to two roundings. Adding 1.5 * 2^23 rounds to the nearest even integer and
// leaves it in the low byte. (In a block with a NaN or an infinity the codes
// mean nothing: its scale is NaN, or infinite with codes 0.)
__device__ __forceinline__ uint32_t ckpt_codes4(float a, float b, float c, float d, float r) {
#pragma clang fp contract(off)  // the product is rounded before the sum
  const float ar = a * r, br = b * r, cr = c * r, dr = d * r;
  const uint32_t ab = __builtin_amdgcn_perm(__float_as_uint(br + 12582912.f),
                                            __float_as_uint(ar + 12582912.f), 0x0c0c0400);
  const uint32_t cd = __builtin_amdgcn_perm(__float_as_uint(dr + 12582912.f),
                                            __float_as_uint(cr + 12582912.f), 0x04000c0c);
  return ab | cd;
}

// The values of four codes (exact in fp32: 7 bits times 8).
__device__ __forceinline__ void ckpt_values4(uint32_t q, float s, float* f) {
#pragma unroll
  for (int j = 0; j < 4; ++j) f[j] = static_cast<float>(static_cast<int8_t>(q >> (8 * j))) * s;
}

// Two values to bf16 (v_cvt_pk_bf16_f32: to nearest even, NaN kept).
typedef float ckpt_f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 ckpt_bf16x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint32_t cvt_bf16x2(float a, float b) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(ckpt_f32x2{a, b}, ckpt_bf16x2));
}

}  // namespace moe

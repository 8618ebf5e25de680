// The arithmetic of the 8-bit activation checkpoints (format in moe_ckpt.h),
// shared by the row kernels and the epilogues of the expert GEMMs.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace moe {

// Scale (bf16 bits) of a block whose largest magnitude has these fp32 bits:
// amax / 127 rounded up to bf16, so that every code fits. A NaN stays one.
__device__ __forceinline__ uint32_t ckpt_scale_bits(uint32_t amax_bits) {
  const float s = __uint_as_float(amax_bits) * (1.0f / 127.0f);
  const uint32_t b = max(__float_as_uint(s) & 0x7fffffffu, 0x00800000u);
  return b > 0x7f800000u ? 0x7fc0u : (b + 0xffffu) >> 16;
}

// Four codes: the nearest integers to v r, in -127 .. 127 since r <= 127 / amax
// up to one rounding. Adding 1.5 * 2^23 rounds to the nearest even integer and
// leaves it in the low bits. (Blocks with a NaN or an infinity have scale NaN
// or infinity and code * scale is NaN whatever the code, unless it is finite
// times infinity: v r is then 0 or NaN; NaN's bits are replaced by 0.)
__device__ __forceinline__ uint32_t ckpt_code(float v, float r) {
#pragma clang fp contract(off)  // the product is rounded before the sum
  const float t = v * r;
  const float m = t == t ? t : 0.f;
  return __float_as_uint(m + 12582912.f) & 0xffu;
}
__device__ __forceinline__ uint32_t ckpt_codes4(float a, float b, float c, float d, float r) {
  return ckpt_code(a, r) | ckpt_code(b, r) << 8 | ckpt_code(c, r) << 16 | ckpt_code(d, r) << 24;
}

// The values of four codes (exact in fp32: 7 bits times 8).
__device__ __forceinline__ void ckpt_values4(uint32_t q, float s, float* f) {
#pragma unroll
  for (int j = 0; j < 4; ++j)
    f[j] = static_cast<float>(static_cast<int32_t>(q << (24 - 8 * j)) >> 24) * s;
}

}  // namespace moe

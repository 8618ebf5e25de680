// Activation checkpoints in 8 bits: rows to int8 codes with a bf16 scale for
// each 32 columns, and back, through an index if wanted.
//
// Both are bound by memory: (es + 1 + 1/16) bytes a value to save, (1 + 1/16)
// read and es written to restore. A thread takes 8 columns (16 bytes of bf16,
// 8 of codes), the four lanes of a DPP quad one 32-column block.
#include "ckpt.h"
#include "moe_internal.h"

namespace moe {
namespace {

constexpr int kThreads = 256;

template <bool BF16>
__device__ __forceinline__ void load8(const void* p, int64_t vec, float (&f)[8]) {
  if (BF16) {
    const uint4 v = static_cast<const uint4*>(p)[vec];
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      f[2 * j] = __uint_as_float(w[j] << 16);
      f[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
    }
  } else {
    const float4 a = static_cast<const float4*>(p)[2 * vec];
    const float4 b = static_cast<const float4*>(p)[2 * vec + 1];
    const float v[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = v[j];
  }
}

template <bool BF16>
__device__ __forceinline__ void store8(void* p, int64_t vec, const float (&f)[8]) {
  if (BF16) {
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      w[j] = f32_to_bf16(f[2 * j]) | (static_cast<uint32_t>(f32_to_bf16(f[2 * j + 1])) << 16);
    static_cast<uint4*>(p)[vec] = make_uint4(w[0], w[1], w[2], w[3]);
  } else {
    static_cast<float4*>(p)[2 * vec] = make_float4(f[0], f[1], f[2], f[3]);
    static_cast<float4*>(p)[2 * vec + 1] = make_float4(f[4], f[5], f[6], f[7]);
  }
}

template <bool BF16>
__global__ __launch_bounds__(kThreads) void ckpt_save_kernel(const void* __restrict__ x,
                                                             int64_t n_vec,
                                                             uint2* __restrict__ codes,
                                                             uint16_t* __restrict__ scales) {
  const int64_t v = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  float f[8] = {};
  const bool live = v < n_vec;  // n_vec is a multiple of 4: quads live or die together
  if (live) load8<BF16>(x, v, f);
  uint32_t amax = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) amax = max(amax, __float_as_uint(f[j]) & 0x7fffffffu);
  amax = max(amax, static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(amax), 0xB1, 0xF, 0xF, false)));
  amax = max(amax, static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(amax), 0x4E, 0xF, 0xF, false)));
  const uint32_t s = ckpt_scale_bits(amax);
  const float r = 1.0f / __uint_as_float(s << 16);
  if (live) {
    codes[v] = make_uint2(ckpt_codes4(f[0], f[1], f[2], f[3], r),
                          ckpt_codes4(f[4], f[5], f[6], f[7], r));
    if ((threadIdx.x & 3) == 0) scales[v >> 2] = static_cast<uint16_t>(s);
  }
}

// vecs: 8-column vectors of a row.
template <bool BF16>
__global__ __launch_bounds__(kThreads) void ckpt_restore_kernel(
    const uint2* __restrict__ codes, const uint16_t* __restrict__ scales,
    const int32_t* __restrict__ index, int64_t n_vec, int64_t rows, int vecs,
    void* __restrict__ out) {
  const int64_t v = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  if (v >= n_vec) return;
  const int64_t i = v / vecs;
  const int64_t j = index ? static_cast<int64_t>(index[i]) : i;
  if (j < 0 || j >= rows) return;
  const int64_t src = j * vecs + (v - i * vecs);
  const uint2 q = codes[src];
  const float s = __uint_as_float(static_cast<uint32_t>(scales[src >> 2]) << 16);
  float f[8];
  ckpt_values4(q.x, s, f);
  ckpt_values4(q.y, s, f + 4);
  store8<BF16>(out, v, f);
}

}  // namespace

hipError_t launch_ckpt_save(bool bf16, int64_t rows, int D, const void* x, void* codes,
                            void* scales, hipStream_t s) {
  const int64_t n_vec = rows * D / 8;
  if (n_vec == 0) return hipSuccess;
  const unsigned grid = static_cast<unsigned>((n_vec + kThreads - 1) / kThreads);
  auto* k = bf16 ? ckpt_save_kernel<true> : ckpt_save_kernel<false>;
  k<<<grid, kThreads, 0, s>>>(x, n_vec, static_cast<uint2*>(codes),
                              static_cast<uint16_t*>(scales));
  return hipGetLastError();
}

hipError_t launch_ckpt_restore(bool bf16, int64_t n, int64_t rows, int D, const void* codes,
                               const void* scales, const int32_t* index, void* out,
                               hipStream_t s) {
  const int64_t n_vec = n * D / 8;
  if (n_vec == 0) return hipSuccess;
  const unsigned grid = static_cast<unsigned>((n_vec + kThreads - 1) / kThreads);
  auto* k = bf16 ? ckpt_restore_kernel<true> : ckpt_restore_kernel<false>;
  k<<<grid, kThreads, 0, s>>>(static_cast<const uint2*>(codes),
                              static_cast<const uint16_t*>(scales), index, n_vec, rows, D / 8,
                              out);
  return hipGetLastError();
}

}  // namespace moe

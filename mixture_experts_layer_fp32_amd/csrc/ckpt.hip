// Activation checkpoints in 8 bits: rows to int8 codes with a bf16 scale for
// each 32 columns, and back, through an index if wanted.
//
// Both are bound by memory: (es + 1 + 1/16) bytes a value to save, (1 + 1/16)
// read and es written to restore. To save, a thread takes 16 adjacent columns at
// a time (a 16-byte store of codes), two lanes share a scale: 16384 x 2048 bf16
// in 16 us; 131072 rows of them restored in 111 us, 5.2 TB/s.
#include <type_traits>

#include "ckpt.h"
#include "moe_internal.h"

namespace moe {
namespace {

constexpr int kThreads = 256;

// Sixteen values, at 16-column vector vec.
template <bool BF16>
__device__ __forceinline__ void load16(const void* p, int64_t vec, uint4 (&w)[BF16 ? 2 : 4]) {
#pragma unroll
  for (int i = 0; i < (BF16 ? 2 : 4); ++i)
    w[i] = static_cast<const uint4*>(p)[vec * (BF16 ? 2 : 4) + i];
}
template <bool BF16>
__device__ __forceinline__ void values16(const uint4 (&w)[BF16 ? 2 : 4], float (&f)[16]) {
#pragma unroll
  for (int i = 0; i < (BF16 ? 2 : 4); ++i) {
    const uint32_t u[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (BF16) {
        f[8 * i + 2 * j] = __uint_as_float(u[j] << 16);
        f[8 * i + 2 * j + 1] = __uint_as_float(u[j] & 0xffff0000u);
      } else {
        f[4 * i + j] = __uint_as_float(u[j]);
      }
    }
  }
}

// kSaveVecs vectors a thread, their loads in flight together (two: 30 us for
// 16384 x 2048 bf16, four: 16).
constexpr int kSaveVecs = 4;
template <bool BF16>
__global__ __launch_bounds__(kThreads) void ckpt_save_kernel(const void* __restrict__ x,
                                                             int64_t n_vec,
                                                             uint4* __restrict__ codes,
                                                             uint16_t* __restrict__ scales) {
  const int64_t v0 = static_cast<int64_t>(blockIdx.x) * (kThreads * kSaveVecs) + threadIdx.x;
  uint4 w[kSaveVecs][BF16 ? 2 : 4];
#pragma unroll
  for (int i = 0; i < kSaveVecs; ++i) {
    // (n_vec is even: both lanes of a block are past the end, or none)
    const int64_t v = v0 + i * kThreads;
    if (v < n_vec) load16<BF16>(x, v, w[i]);
  }
#pragma unroll
  for (int i = 0; i < kSaveVecs; ++i) {
    const int64_t v = v0 + i * kThreads;
    float f[16] = {};
    if (v < n_vec) values16<BF16>(w[i], f);
    uint32_t amax = 0;
#pragma unroll
    for (int j = 0; j < 16; ++j) amax = max(amax, __float_as_uint(f[j]) & 0x7fffffffu);
    amax = max(amax, static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(amax), 0xB1, 0xF, 0xF, false)));
    const uint32_t s = ckpt_scale_bits(amax);
    const float r = ckpt_factor(s);
    if (v < n_vec) {
      codes[v] = make_uint4(ckpt_codes4(f[0], f[1], f[2], f[3], r),
                            ckpt_codes4(f[4], f[5], f[6], f[7], r),
                            ckpt_codes4(f[8], f[9], f[10], f[11], r),
                            ckpt_codes4(f[12], f[13], f[14], f[15], r));
      if ((threadIdx.x & 1) == 0) scales[v >> 1] = static_cast<uint16_t>(s);
    }
  }
}

// A thread restores 16 bytes of a row, so that a wave's store is adjacent:
// 2^lanes_log threads take a row's vecs vectors of kCols columns, a workgroup
// kThreads >> lanes_log rows at a time, kRestoreRows times. (With 16 columns a
// thread, two stores of alternating 16 bytes, 129 us for 131072 x 2048 bf16.)
// The stores stream past the caches: a restore writes more than they hold,
// and its reads, up to k times the same rows, then stay there.
constexpr int kRestoreRows = 4;
typedef unsigned u32x4 __attribute__((ext_vector_type(4)));
template <bool BF16>
__global__ __launch_bounds__(kThreads) void ckpt_restore_kernel(
    const uint8_t* __restrict__ codes, const uint16_t* __restrict__ scales,
    const int32_t* __restrict__ index, int64_t n, int64_t rows, int vecs, int lanes_log,
    u32x4* __restrict__ out) {
  constexpr int kCols = BF16 ? 8 : 4;
  typedef typename std::conditional<BF16, uint2, uint32_t>::type Codes;
  const int lane = threadIdx.x & ((1 << lanes_log) - 1);
  const int per = kThreads >> lanes_log;
  const int64_t i0 = static_cast<int64_t>(blockIdx.x) * (per * kRestoreRows) + (threadIdx.x >> lanes_log);
  int64_t src[kRestoreRows];  // first vector of the row of codes, -1: none
#pragma unroll
  for (int r = 0; r < kRestoreRows; ++r) {
    const int64_t i = i0 + r * per;
    const int64_t j = i < n ? (index ? static_cast<int64_t>(index[i]) : i) : -1;
    src[r] = j >= 0 && j < rows ? j * vecs : -1;
  }
  for (int c = lane; c < vecs; c += 1 << lanes_log) {
    Codes q[kRestoreRows];
    uint32_t s[kRestoreRows];
#pragma unroll
    for (int r = 0; r < kRestoreRows; ++r)
      if (src[r] >= 0) {
        q[r] = reinterpret_cast<const Codes*>(codes)[src[r] + c];
        s[r] = scales[(src[r] + c) / (32 / kCols)];
      }
#pragma unroll
    for (int r = 0; r < kRestoreRows; ++r)
      if (src[r] >= 0) {
        const float sv = __uint_as_float(s[r] << 16);
        float f[8];
        u32x4 w;
        if constexpr (BF16) {
          ckpt_values4(q[r].x, sv, f);
          ckpt_values4(q[r].y, sv, f + 4);
#pragma unroll
          for (int j = 0; j < 4; ++j) w[j] = cvt_bf16x2(f[2 * j], f[2 * j + 1]);
        } else {
          ckpt_values4(q[r], sv, f);
#pragma unroll
          for (int j = 0; j < 4; ++j) w[j] = __float_as_uint(f[j]);
        }
        __builtin_nontemporal_store(w, out + (i0 + r * per) * vecs + c);
      }
  }
}

}  // namespace

hipError_t launch_ckpt_save(bool bf16, int64_t rows, int D, const void* x, void* codes,
                            void* scales, hipStream_t s) {
  const int64_t n_vec = rows * D / 16;
  if (n_vec == 0) return hipSuccess;
  constexpr int kPer = kThreads * kSaveVecs;
  const unsigned grid = static_cast<unsigned>((n_vec + kPer - 1) / kPer);
  auto* k = bf16 ? ckpt_save_kernel<true> : ckpt_save_kernel<false>;
  k<<<grid, kThreads, 0, s>>>(x, n_vec, static_cast<uint4*>(codes),
                              static_cast<uint16_t*>(scales));
  return hipGetLastError();
}

hipError_t launch_ckpt_restore(bool bf16, int64_t n, int64_t rows, int D, const void* codes,
                               const void* scales, const int32_t* index, void* out,
                               hipStream_t s) {
  if (n == 0) return hipSuccess;
  const int vecs = D / (bf16 ? 8 : 4);
  int lanes_log = 0;  // a power of two of at most vecs lanes a row
  while (lanes_log < 8 && (2 << lanes_log) <= vecs) ++lanes_log;
  const int64_t per = static_cast<int64_t>(kThreads >> lanes_log) * kRestoreRows;
  const unsigned grid = static_cast<unsigned>((n + per - 1) / per);
  auto* k = bf16 ? ckpt_restore_kernel<true> : ckpt_restore_kernel<false>;
  k<<<grid, kThreads, 0, s>>>(static_cast<const uint8_t*>(codes),
                              static_cast<const uint16_t*>(scales), index, n, rows, vecs,
                              lanes_log, static_cast<u32x4*>(out));
  return hipGetLastError();
}

}  // namespace moe

// FP8 quantization with block scales: activation rows (a scale for each row
// and 128 columns) and packed expert weights (a scale for each 128 x 128
// block).
//
//   s = max(amax * (1/448), 2^-126),  code = e4m3_rne(v * (1 / s))
// with the two quotients as fp32 constants or one correctly rounded division
// per block: a division for each value would cost more than its memory
// traffic. |v (1/s)| <= 448 (1 + 2^-22), which rounds to 448, so the hardware
// conversion (round to nearest even, NaN above 464) never overflows on finite
// blocks; a block with a NaN or an infinity gets s NaN or infinite, v * (1/s)
// is NaN or 0 and code * s is NaN everywhere. amax is taken on the bits of
// |v|, which order as the values do, with NaN above everything.
#include "moe_internal.h"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kRows = 16;    // rows per workgroup: 64-byte runs of scales
constexpr int kCols = 512;   // columns per workgroup: four blocks, 1 KB of bf16 a row
constexpr uint32_t kTinyBits = 0x00800000u;  // 2^-126

__device__ __forceinline__ uint32_t abs_bits(float f) { return __float_as_uint(f) & 0x7fffffffu; }

__device__ __forceinline__ float block_scale(uint32_t amax_bits) {
  const float s = __uint_as_float(amax_bits) * (1.0f / 448.0f);
  return __uint_as_float(max(__float_as_uint(s) & 0x7fffffffu, kTinyBits));
}

// Four values to four codes.
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d, float r) {
  int v = __builtin_amdgcn_cvt_pk_fp8_f32(a * r, b * r, 0, false);
  v = __builtin_amdgcn_cvt_pk_fp8_f32(c * r, d * r, v, true);
  return static_cast<uint32_t>(v);
}

// Maximum over the 16 lanes of a DPP row.
__device__ __forceinline__ uint32_t row16_max(uint32_t v) {
#define MOE_DPP_MAX(ctrl) \
  v = max(v, static_cast<uint32_t>( \
                 __builtin_amdgcn_mov_dpp(static_cast<int>(v), ctrl, 0xF, 0xF, false)))
  MOE_DPP_MAX(0xB1);   // lane ^ 1
  MOE_DPP_MAX(0x4E);   // lane ^ 2
  MOE_DPP_MAX(0x141);  // mirrored half row (7 - lane)
  MOE_DPP_MAX(0x140);  // mirrored row (15 - lane)
#undef MOE_DPP_MAX
  return v;
}

// 16 lanes hold one 128-column block of a row, a wave four blocks of it; wave
// w takes rows w, w + 4, ... of the workgroup's 16. The scales of the 16 rows
// are gathered in LDS and leave as 64-byte runs. Bound by memory: 16384 x 4096
// bf16 in 39.8 us, 5.1 TB/s, what a copy reaches.
template <bool BF16>
__global__ __launch_bounds__(kThreads) void fp8_quantize_rows_kernel(
    const void* __restrict__ xv, int64_t rows, int K, int col_tiles, uint8_t* __restrict__ codes,
    float* __restrict__ scales) {
  __shared__ float s_scale[kCols / 128][kRows];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int64_t row0 = static_cast<int64_t>(blockIdx.x / col_tiles) * kRows;
  const int c0 = static_cast<int>(blockIdx.x % col_tiles) * kCols;
  const int blk = lane >> 4, l = lane & 15;
  // bf16: 8 adjacent columns; fp32: 4 in each half of the block, so that the
  // loads of 16 lanes are adjacent.
  const int col = c0 + 128 * blk + (BF16 ? 8 * l : 4 * l);
  float f[4][8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t row = row0 + wave + 4 * i;
    const int64_t o = row * K + col;
#pragma unroll
    for (int j = 0; j < 8; ++j) f[i][j] = 0.f;
    if (BF16) {
      if (row < rows && col < K) {
        const uint4 v = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(xv) + o);
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          f[i][2 * j] = __uint_as_float(w[j] << 16);
          f[i][2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
        }
      }
    } else {
#pragma unroll
      for (int h = 0; h < 2; ++h)
        if (row < rows && col + 64 * h < K) {
          const float4 v = *reinterpret_cast<const float4*>(static_cast<const float*>(xv) + o + 64 * h);
          f[i][4 * h] = v.x;
          f[i][4 * h + 1] = v.y;
          f[i][4 * h + 2] = v.z;
          f[i][4 * h + 3] = v.w;
        }
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t row = row0 + wave + 4 * i;
    uint32_t amax = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) amax = max(amax, abs_bits(f[i][j]));
    const float s = block_scale(row16_max(amax));
    const float r = 1.0f / s;
    const uint32_t lo = e4m3x4(f[i][0], f[i][1], f[i][2], f[i][3], r);
    const uint32_t hi = e4m3x4(f[i][4], f[i][5], f[i][6], f[i][7], r);
    if (l == 0) s_scale[blk][wave + 4 * i] = s;
    if (row < rows) {
      uint8_t* dst = codes + row * K + col;
      if (BF16) {
        if (col < K) *reinterpret_cast<uint2*>(dst) = make_uint2(lo, hi);
      } else {
        if (col < K) *reinterpret_cast<uint32_t*>(dst) = lo;
        if (col + 64 < K) *reinterpret_cast<uint32_t*>(dst + 64) = hi;
      }
    }
  }
  __syncthreads();
  if (threadIdx.x < (kCols / 128) * kRows) {
    const int b = threadIdx.x / kRows, i = threadIdx.x % kRows;
    if (row0 + i < rows && c0 + 128 * b < K)
      scales[static_cast<int64_t>(c0 / 128 + b) * rows + row0 + i] = s_scale[b][i];
  }
}

// One 128 x 128 block of w [K][N] per workgroup: thread t reads the rows
// t / 16 + 16 i at columns 8 (t % 16), the block's maximum goes through LDS,
// and the codes leave transposed, 16 bytes of K a thread. Runs once per
// weight load.
constexpr int kPitch = 144;  // bytes of an LDS row of 128 codes (K), 16-byte aligned
template <bool BF16>
__global__ __launch_bounds__(kThreads) void fp8_pack_weights_kernel(
    const void* __restrict__ wv, int K, int N, int kb, int nb, uint8_t* __restrict__ codes,
    float* __restrict__ scales) {
  __shared__ __attribute__((aligned(16))) uint8_t tile[128 * kPitch];
  __shared__ uint32_t s_max[kThreads / 64];
  const int t = threadIdx.x;
  const int bk = static_cast<int>(blockIdx.x) % kb;
  const int rest = static_cast<int>(blockIdx.x) / kb;
  const int bn = rest % nb, e = rest / nb;
  const int n0 = bn * 128 + 8 * (t & 15), k0 = bk * 128 + (t >> 4);
  float f[8][8];
  uint32_t amax = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int k = k0 + 16 * i;
#pragma unroll
    for (int j = 0; j < 8; ++j) f[i][j] = 0.f;
    if (k < K && n0 < N) {
      const int64_t o = (static_cast<int64_t>(e) * K + k) * N + n0;
      if (BF16) {
        const uint4 v = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(wv) + o);
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          f[i][2 * j] = __uint_as_float(w[j] << 16);
          f[i][2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
        }
      } else {
        const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(wv) + o);
        const float4 a = p[0], b = p[1];
        const float v[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
        for (int j = 0; j < 8; ++j) f[i][j] = v[j];
      }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) amax = max(amax, abs_bits(f[i][j]));
  }
#pragma unroll
  for (int off = 32; off > 0; off >>= 1)
    amax = max(amax, static_cast<uint32_t>(__shfl_xor(static_cast<int>(amax), off, 64)));
  if ((t & 63) == 0) s_max[t >> 6] = amax;
  __syncthreads();
  amax = max(max(s_max[0], s_max[1]), max(s_max[2], s_max[3]));
  const float s = block_scale(amax), r = 1.0f / s;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t q[2] = {e4m3x4(f[i][0], f[i][1], f[i][2], f[i][3], r),
                           e4m3x4(f[i][4], f[i][5], f[i][6], f[i][7], r)};
#pragma unroll
    for (int j = 0; j < 8; ++j)
      tile[(8 * (t & 15) + j) * kPitch + (t >> 4) + 16 * i] =
          static_cast<uint8_t>(q[j >> 2] >> (8 * (j & 3)));
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int n = (t >> 3) + 32 * i, k = 16 * (t & 7);
    if (bn * 128 + n < N && bk * 128 + k < K)
      *reinterpret_cast<uint4*>(codes + (static_cast<int64_t>(e) * N + bn * 128 + n) * K +
                                bk * 128 + k) =
          *reinterpret_cast<const uint4*>(tile + n * kPitch + k);
  }
  if (t == 0) scales[(static_cast<int64_t>(e) * nb + bn) * kb + bk] = s;
}

}  // namespace

hipError_t launch_fp8_quantize_rows(bool bf16, int64_t rows, int K, const void* x, void* codes,
                                    float* scales, hipStream_t s) {
  if (rows == 0) return hipSuccess;
  const int ct = (K + kCols - 1) / kCols;
  const unsigned grid = static_cast<unsigned>((rows + kRows - 1) / kRows * ct);
  auto* k = bf16 ? fp8_quantize_rows_kernel<true> : fp8_quantize_rows_kernel<false>;
  k<<<grid, kThreads, 0, s>>>(x, rows, K, ct, static_cast<uint8_t*>(codes), scales);
  return hipGetLastError();
}

hipError_t launch_fp8_pack_weights(bool bf16, int n, int K, int N, const void* w, void* codes,
                                   float* scales, hipStream_t s) {
  if (n == 0) return hipSuccess;
  const int kb = (K + 127) / 128, nb = (N + 127) / 128;
  const unsigned grid = static_cast<unsigned>(static_cast<int64_t>(n) * kb * nb);
  auto* k = bf16 ? fp8_pack_weights_kernel<true> : fp8_pack_weights_kernel<false>;
  k<<<grid, kThreads, 0, s>>>(w, K, N, kb, nb, static_cast<uint8_t*>(codes), scales);
  return hipGetLastError();
}

}  // namespace moe

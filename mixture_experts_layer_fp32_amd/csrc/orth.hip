// Newton-Schulz orthogonalisation and the Muon update (include/moe_update.h).
//
//   X_0 = U / (||U||_F + eps),  X <- P(A) X,  A = X X^T,
//   P(A) = a I + b A + c A^2
//
// X is m x k with m <= k (the transposed matrix when U is taller than wide).
//
// Steps on the short side. P(A) X has the Gram matrix P A P, because A and P
// commute; so after one product A = X X^T several steps can be taken on m x m
// matrices alone (P_1, A_2 = P_1 A P_1, P_2, ...), their product
// Q = ... P_2 P_1 kept, and X <- Q X done once. A segment of L steps costs
// 3 k m^2 + (4 L - 3) m^3 multiply-adds instead of L (3 k m^2 + m^3) (every
// m x m result is symmetric: half a product). Rounding errors of A in
// directions of small singular values grow by a^2 = 11.9 a step until A is
// formed from X again, so segments are short, and the longest comes first,
// where X's singular values are far below 1. Five steps in one segment end in
// NaN on low-rank matrices (simulated). segment_rule() has the lengths and
// the errors measured with them.
//
// Products. Each fp32 value v is held as two fp16 numbers, hi = fp16(v s) and
// lo = fp16(v s - hi), s a power of two per matrix: 22 bits and the sign of
// lo. x y = hi hi + hi lo + lo hi on the fp16 matrix cores, summed in fp32;
// lo lo (2^-24 of the product, typically) is left out: in the simulations
// keeping it changed the error by less than 4 %. Three matrix instructions
// at the fp16 rate stand for one fp32 product, against a 16th of that rate
// for fp32 instructions. The scales keep every operand in fp16's range: X
// entries are at most 1.21, A's 1.46, P's 3.45 and Q's 41 (the largest
// singular value bounds an entry), while s = 2^12 puts fp16's smallest step
// (2^-24) at 2^-36 of unit.
//
// Layout. A matrix operand [R][K] is stored in matrix-core fragments: 32-row
// block rb, 16-deep slice ks, part (hi, lo), lane l, 8 values:
//   ((rb KS + ks) 2 + part) 512 + l 8 + j  holds  (32 rb + l % 32,
//                                                  16 ks + 8 (l / 32) + j),
// KS = 2 ceil(K / 32), zeros past R and K. A workgroup's copies are runs of
// 4 KB, a fragment is 16 bytes a lane in LDS order, so there are no bank
// conflicts and no swizzle.
#include <algorithm>

#include "moe_internal.h"
#include "moe_update.h"

namespace moe {
namespace {

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef __attribute__((address_space(3))) unsigned char lds_u8;

constexpr float kA = 3.4445f, kB = -4.7750f, kC = 2.0315f;
constexpr float kScaleX = 4096.f, kScaleA = 4096.f, kScaleP = 1024.f;
constexpr int kXcds = 8;

struct Mats {  // moe_matrices on the device side
  void* data;
  int64_t ld, stride;
  int bf16;
};

__device__ __forceinline__ float load_el(const Mats& m, int64_t off) {
  return m.bf16 ? bf16_to_f32(static_cast<const uint16_t*>(m.data)[off])
                : static_cast<const float*>(m.data)[off];
}

// ---- norm: partial sums of squares; the momentum -----------------------------
// Partial sums in fp64 (no overflow or underflow of squares). With mom.data
// the momentum is updated and the norm is that of U.
__global__ __launch_bounds__(256) void orth_norm_kernel(Mats g, Mats mom, float mu, int nesterov,
                                                        int rows, int cols,
                                                        int64_t chunk, double* __restrict__ part) {
  const int b = blockIdx.y;
  const int64_t e0 = blockIdx.x * chunk;
  const int64_t e1 = min(e0 + chunk, static_cast<int64_t>(rows) * cols);
  double s = 0.0;
  for (int64_t e = e0 + threadIdx.x; e < e1; e += 256) {
    const int64_t r = e / cols, c = e - r * cols;
    float u = load_el(g, b * g.stride + r * g.ld + c);
    if (mom.data != nullptr) {
      float* mp = static_cast<float*>(mom.data) + b * mom.stride + r * mom.ld + c;
      const float m = fmaf(mu, *mp, u);
      *mp = m;
      u = nesterov ? fmaf(mu, m, u) : m;
    }
    s += static_cast<double>(u) * u;
  }
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) s += __shfl_xor(s, off, 64);
  __shared__ double red[4];
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = s;
  __syncthreads();
  if (threadIdx.x == 0)
    part[static_cast<int64_t>(b) * gridDim.x + blockIdx.x] = red[0] + red[1] + red[2] + red[3];
}

// v s as two fp16 numbers.
__device__ __forceinline__ void split(float v, uint16_t& hi, uint16_t& lo) {
  const _Float16 h = static_cast<_Float16>(v);
  const _Float16 l = static_cast<_Float16>(v - static_cast<float>(h));
  hi = __builtin_bit_cast(uint16_t, h);
  lo = __builtin_bit_cast(uint16_t, l);
}

// ---- split: U / norm into fragments, both ways round -------------------------
// One 64 x 64 tile of U a workgroup, through LDS.
__global__ __launch_bounds__(256) void orth_split_kernel(
    Mats g, Mats mom, float mu, int nesterov, int rows, int cols, float eps,
    const double* __restrict__ part, int nparts, uint16_t* __restrict__ u_planes,
    uint16_t* __restrict__ ut_planes, int64_t plane_stride, int tiles_c) {
  __shared__ float tile[64][65];
  __shared__ double red[4];
  const int b = blockIdx.y, tid = threadIdx.x;
  const int r0 = (blockIdx.x / tiles_c) * 64, c0 = (blockIdx.x % tiles_c) * 64;
  double s = 0.0;
  for (int i = tid; i < nparts; i += 256) s += part[static_cast<int64_t>(b) * nparts + i];
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) s += __shfl_xor(s, off, 64);
  if ((tid & 63) == 0) red[tid >> 6] = s;
  __syncthreads();
  const double inv =
      static_cast<double>(kScaleX) / (sqrt(red[0] + red[1] + red[2] + red[3]) + eps);
  for (int i = tid; i < 64 * 64; i += 256) {
    const int r = r0 + (i >> 6), c = c0 + (i & 63);
    float u = 0.f;
    if (r < rows && c < cols) {
      u = load_el(g, b * g.stride + r * g.ld + c);
      if (mom.data != nullptr) {
        const float m = static_cast<const float*>(mom.data)[b * mom.stride + r * mom.ld + c];
        u = nesterov ? fmaf(mu, m, u) : m;
      }
      u = static_cast<float>(u * inv);
    }
    tile[i >> 6][i & 63] = u;
  }
  __syncthreads();
  // 8 fragments of each orientation (2 row blocks x 4 slices), 64 lanes each.
  const int rb_u = (rows + 31) / 32, rb_t = (cols + 31) / 32;
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    uint16_t* out = (half == 0 ? u_planes : ut_planes) + b * plane_stride;
    const int nrb = half == 0 ? rb_u : rb_t, ks_n = 2 * (half == 0 ? rb_t : rb_u);
    const int rb0 = (half == 0 ? r0 : c0) / 32, ks0 = (half == 0 ? c0 : r0) / 16;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int f = (tid >> 6) + 4 * i, lane = tid & 63;
      const int rb = f >> 2, ks = f & 3;
      if (rb0 + rb >= nrb || ks0 + ks >= ks_n) continue;
      const int row = 32 * rb + (lane & 31), k = 16 * ks + 8 * (lane >> 5);
      union {
        uint16_t h[8];
        uint4 v;
      } hi, lo;
#pragma unroll
      for (int j = 0; j < 8; ++j)
        split(half == 0 ? tile[row][k + j] : tile[k + j][row], hi.h[j], lo.h[j]);
      uint4* p = reinterpret_cast<uint4*>(
          out + (static_cast<int64_t>(rb0 + rb) * ks_n + ks0 + ks) * 1024 + lane * 8);
      p[0] = hi.v;
      p[64] = lo.v;
    }
  }
}

// ---- products ------------------------------------------------------------------
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
// 16 bytes global -> LDS at lds_base + 16 * lane (M0 holds the LDS base).
// Out-of-range offsets write zeros. Counted by vmcnt.
__device__ __forceinline__ void dma16(__amdgpu_buffer_rsrc_t rsrc, int voff, int soff,
                                      unsigned lds_base) {
  asm volatile("s_mov_b32 m0, %3\n\tbuffer_load_dwordx4 %0, %1, %2 offen lds"
               :: "v"(voff), "s"(rsrc), "s"(soff), "s"(lds_base) : "memory", "m0");
}
#pragma clang diagnostic pop

constexpr int vmcnt_imm(int n) { return (n & 15) | (7 << 4) | (15 << 8) | ((n >> 4) << 14); }

// 4x4 transpose inside each group of 4 lanes: before, lane l's v[s] is row
// 4 (l / 32) + s, column l % 32; after, it is row 4 (l / 32) + l % 4, column
// 4 (l % 32 / 4) + s.
__device__ __forceinline__ void transpose4(float (&v)[4], int quad) {
  float n[4];
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const float x = __builtin_bit_cast(
        float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v[r ^ 1]), 0xB1, 0xF, 0xF, false));
    n[r] = ((r ^ quad) & 1) ? x : v[r];
  }
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const float x = __builtin_bit_cast(
        float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, n[r ^ 2]), 0x4E, 0xF, 0xF, false));
    v[r] = ((r ^ quad) & 2) ? x : n[r];
  }
}

__device__ __forceinline__ void store_parts(uint16_t* frag, int lane, int j, const float (&v)[4]) {
  union {
    uint16_t h[4];
    uint2 w;
  } hi, lo;
#pragma unroll
  for (int s = 0; s < 4; ++s) split(v[s], hi.h[s], lo.h[s]);
  *reinterpret_cast<uint2*>(frag + lane * 8 + j) = hi.w;
  *reinterpret_cast<uint2*>(frag + 512 + lane * 8 + j) = lo.w;
}

// One product D[i][j] = sum_k a[i][k] b[j][k] of n matrices, a of ra 32-row
// blocks, b of rb, both KS slices deep; strides between matrices in values.
struct Product {
  const uint16_t *a, *b;
  int64_t sa, sb;
  uint16_t* out_t;  // operand with rows j and depth i
  uint16_t* out_n;  // operand with rows i and depth j
  int64_t so;
  const uint16_t* aux;  // kSym: symmetric operand added with factor beta
  float alpha, beta, gamma;
};
struct Out {  // kOut: matrix row j, column i
  Mats w;
  int rows, cols;
  float keep, add;  // w <- keep w + add O (muon), or w <- add O
  int muon;
};

enum Epilogue { kSym = 0, kOperand = 1, kOut = 2 };

// kSym: the result is symmetric: tiles on and below the diagonal only;
//   alpha D + beta aux + gamma I is stored into out_t, and its mirror image.
// kOperand: alpha D is stored into out_t and out_n.
// kOut: to the caller's matrices.
// blockIdx.y: one of two independent products.
template <int EPI, int WM, int WN, int WR, int WC>
__global__ __launch_bounds__(64 * WR * WC) void orth_product_kernel(Product p0, Product p1,
                                                                   Out o, int n, int ra, int rb,
                                                                   int KS) {
  constexpr int BA = WR * WM, BB = WC * WN;    // 32-row blocks per tile
  constexpr int NW = WR * WC;
  constexpr int kStage = (BA + BB) * 4096;     // K = 32, both parts
  constexpr int NC = (BA + BB) * 4 / NW;       // 1 KB copies per wave and step
  static_assert((BA + BB) * 4 % NW == 0, "copies are shared out evenly");
  static_assert(EPI != kSym || BA == BB, "symmetric results use square tiles");
  __shared__ __attribute__((aligned(1024))) unsigned char smem[2 * kStage];

  const Product& p = blockIdx.y == 0 ? p0 : p1;
  const int ta = (ra + BA - 1) / BA, tb = (rb + BB - 1) / BB;
  const int per_mat = EPI == kSym ? ta * (ta + 1) / 2 : ta * tb;
  // The tiles in eight runs, one an XCD (workgroup b runs on XCD b % 8).
  const int total = per_mat * n, per = (total + kXcds - 1) / kXcds;
  const int t = (static_cast<int>(blockIdx.x) % kXcds) * per + static_cast<int>(blockIdx.x) / kXcds;
  if (t >= total) return;
  const int mat = t / per_mat, lt = t - mat * per_mat;
  int ti, tj;
  if constexpr (EPI == kSym) {
    ti = static_cast<int>((sqrtf(8.f * lt + 1.f) - 1.f) * 0.5f);
    while (ti * (ti + 1) / 2 > lt) --ti;
    while ((ti + 1) * (ti + 2) / 2 <= lt) ++ti;
    tj = lt - ti * (ti + 1) / 2;
  } else {
    ti = lt / tb;
    tj = lt - ti * tb;
  }
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wr = wave / WC, wc = wave % WC;
  const int a0 = ti * BA, b0 = tj * BB;  // first 32-row blocks

  // ---- copies: piece c of a step is 1 KB, four pieces a row block ----
  const int row_bytes = KS * 2048;
  const __amdgpu_buffer_rsrc_t a_rsrc = __builtin_amdgcn_make_buffer_rsrc(
      (void*)(p.a + mat * p.sa + static_cast<int64_t>(a0) * KS * 1024), 0,
      min(BA, ra - a0) * row_bytes, 0x00020000);
  const __amdgpu_buffer_rsrc_t b_rsrc = __builtin_amdgcn_make_buffer_rsrc(
      (void*)(p.b + mat * p.sb + static_cast<int64_t>(b0) * KS * 1024), 0,
      min(BB, rb - b0) * row_bytes, 0x00020000);
  const unsigned lds0 = (unsigned)(uintptr_t)(lds_u8*)smem;
  auto copy_step = [&](int kt, int slot) {
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int c = wave * NC + i;
      const int blk = c >> 2;
      const unsigned dst = lds0 + slot * kStage + c * 1024;
      if (blk < BA)
        dma16(a_rsrc, blk * row_bytes + (c & 3) * 1024 + lane * 16, kt * 4096, dst);
      else
        dma16(b_rsrc, (blk - BA) * row_bytes + (c & 3) * 1024 + lane * 16, kt * 4096, dst);
    }
  };

  f32x16 acc[WM][WN];
#pragma unroll
  for (int i = 0; i < WM; ++i)
#pragma unroll
    for (int j = 0; j < WN; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;

  const int nk = KS / 2;
  copy_step(0, 0);
  for (int kt = 0; kt < nk; ++kt) {
    // This wave's copies of step kt have landed; after the barrier every
    // wave's have, and every wave is done with the other slot.
    __builtin_amdgcn_s_waitcnt(vmcnt_imm(0));
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");  // no LDS read moves above the barrier
    if (kt + 1 < nk) copy_step(kt + 1, (kt + 1) & 1);
    const unsigned char* s = smem + (kt & 1) * kStage + lane * 16;
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {
      f16x8 fa[WM][2], fb[WN][2];
#pragma unroll
      for (int i = 0; i < WM; ++i)
#pragma unroll
        for (int q = 0; q < 2; ++q)
          fa[i][q] = *reinterpret_cast<const f16x8*>(s + (wr * WM + i) * 4096 + ks * 2048 + q * 1024);
#pragma unroll
      for (int j = 0; j < WN; ++j)
#pragma unroll
        for (int q = 0; q < 2; ++q)
          fb[j][q] = *reinterpret_cast<const f16x8*>(s + (BA + wc * WN + j) * 4096 + ks * 2048 +
                                                     q * 1024);
#pragma unroll
      for (int q = 0; q < 3; ++q)  // lo hi, hi lo, hi hi
#pragma unroll
        for (int i = 0; i < WM; ++i)
#pragma unroll
          for (int j = 0; j < WN; ++j)
            acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(fa[i][q == 0], fb[j][q == 1],
                                                               acc[i][j], 0, 0, 0);
    }
  }

  // ---- epilogue: register 4 q + s of lane l is row 8 q + 4 (l / 32) + s of
  // the a block and row l % 32 of the b block ----
  const int half = lane >> 5, l32 = lane & 31;
#pragma unroll
  for (int i = 0; i < WM; ++i) {
    const int ib = a0 + wr * WM + i;
    if (ib >= ra) continue;
#pragma unroll
    for (int j = 0; j < WN; ++j) {
      const int jb = b0 + wc * WN + j;
      if (jb >= rb) continue;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        float v[4];
#pragma unroll
        for (int s = 0; s < 4; ++s) v[s] = acc[i][j][4 * q + s] * p.alpha;
        if constexpr (EPI == kOut) {
          const int r = jb * 32 + l32, c = ib * 32 + 8 * q + 4 * half;
          if (r >= o.rows) continue;
          const int64_t at = mat * o.w.stride + r * o.w.ld + c;
#pragma unroll
          for (int s = 0; s < 4; ++s) {
            if (c + s >= o.cols) continue;
            float w = o.add * v[s];
            if (o.muon) w = fmaf(o.keep, load_el(o.w, at + s), w);
            if (o.w.bf16)
              static_cast<uint16_t*>(o.w.data)[at + s] = f32_to_bf16(w);
            else
              static_cast<float*>(o.w.data)[at + s] = w;
          }
        } else {
          // Operand with rows j: depth KT slices (that of i's blocks).
          const int64_t ft = (static_cast<int64_t>(jb) * (2 * ra) + 2 * ib + (q >> 1)) * 1024;
          const int lt2 = l32 + 32 * (q & 1);
          if constexpr (EPI == kSym) {
            if (p.aux != nullptr) {
              const uint16_t* x = p.aux + mat * p.so + ft + lt2 * 8 + 4 * half;
              union {
                uint2 w;
                _Float16 h[4];
              } hi, lo;
              hi.w = *reinterpret_cast<const uint2*>(x);
              lo.w = *reinterpret_cast<const uint2*>(x + 512);
#pragma unroll
              for (int s = 0; s < 4; ++s) {
                const float av = static_cast<float>(hi.h[s]) + static_cast<float>(lo.h[s]);
                v[s] = fmaf(p.beta, av, v[s]);
                if (ib == jb && 8 * q + 4 * half + s == l32) v[s] += p.gamma;
              }
            }
          }
          store_parts(p.out_t + mat * p.so + ft, lt2, 4 * half, v);
          if (EPI == kOperand || ti != tj) {
            transpose4(v, lane & 3);
            const int j0 = 4 * (l32 >> 2), row = 8 * q + 4 * half + (lane & 3);
            const int64_t fn = (static_cast<int64_t>(ib) * (2 * rb) + 2 * jb + (j0 >> 4)) * 1024;
            store_parts(p.out_n + mat * p.so + fn, row + 32 * ((j0 >> 3) & 1), j0 & 7, v);
          }
        }
      }
    }
  }
}

int ceil32(int v) { return (v + 31) / 32; }

// Workspace, in values (16 bits) per matrix: X and two X^T (or the other way
// round for tall matrices), five m x m operands; then the norm's partials.
struct Space {
  int64_t x, mm;  // values of one X operand, of one m x m operand
  int64_t part;   // partial sums per matrix
  size_t bytes;
};
int norm_parts(int n, int64_t values) {
  const int64_t most = std::max<int64_t>(1, std::min<int64_t>(1024, 4096 / std::max(n, 1)));
  return static_cast<int>(std::min<int64_t>(most, (values + 4095) / 4096));
}
Space space(int n, int rows, int cols) {
  Space s;
  const int64_t m = ceil32(std::min(rows, cols)), k = ceil32(std::max(rows, cols));
  s.x = m * 2 * k * 1024;
  s.mm = m * 2 * m * 1024;
  s.part = norm_parts(n, static_cast<int64_t>(rows) * cols);
  s.bytes = static_cast<size_t>(n) * ((3 * s.x + 5 * s.mm) * 2 + s.part * 8);
  return s;
}

// Most steps of the first segment and of the later ones. Relative Frobenius
// error of fp32 results against 64 bits (gradients of 1.5 m tokens; plain
// torch fp32 / steps one by one / 2 + 2 + 1 / 3 + 2, in 1e-6):
//   8 x 128 x 512    1.7 / 1.2 / 2.4 / 2.6     4 x 512 x 512     2.1 / 1.8 / 3.4 / 5.2
//   4 x 256 x 1024   2.1 / 1.4 / 3.4 / 2.4     4 x 1024 x 1024   2.7 / 2.3 / 3.4 / 7.7
//   2 x 1024 x 4096  3.5 / 2.6 / 4.1 / 5.3     1 x 2048 x 2048   3.5 / 2.9 / 3.4 / 9.4
// A bf16 result rounds by 1.7e-3, so it takes the fewest operations. An fp32
// result keeps plain fp32's accuracy: single steps, and pairs from m = 1024
// on. In a Muon step with fp32 weights the update is a small part of the
// weight, and with it the error: pairs.
struct Segments {
  int first, later;
};
Segments segment_rule(bool bf16_out, bool muon, int m) {
  if (bf16_out) return {3, 2};
  if (muon || m >= 1024) return {2, 2};
  return {1, 1};
}

template <int EPI>
hipError_t launch_product(const Product& p0, const Product* p1, const Out& o, int n, int ra,
                          int rb, int KS, hipStream_t s) {
  constexpr int B = 4;
  const int ta = (ra + B - 1) / B, tb = (rb + B - 1) / B;
  const int64_t total = static_cast<int64_t>(n) * (EPI == kSym ? ta * (ta + 1) / 2 : ta * tb);
  const int64_t grid = (total + kXcds - 1) / kXcds * kXcds;
  orth_product_kernel<EPI, 2, 2, 2, 2><<<dim3(static_cast<unsigned>(grid), p1 ? 2 : 1), 256, 0, s>>>(
      p0, p1 ? *p1 : p0, o, n, ra, rb, KS);
  return hipGetLastError();
}

}  // namespace

size_t orth_ws_bytes(int n, int rows, int cols) { return space(n, rows, cols).bytes; }

int64_t orth_tiles(int n, int rows, int cols) {
  const int64_t m = (std::min(rows, cols) + 127) / 128, k = (std::max(rows, cols) + 127) / 128;
  return n * m * k;
}

// mom.data NULL: orthogonalise g into w. Otherwise a Muon step.
hipError_t launch_orth(int n, int rows, int cols, const moe_matrices& g, const moe_matrices* mom,
                       const moe_matrices& w, const moe_muon_desc& d, void* ws, hipStream_t s) {
  const Space sp = space(n, rows, cols);
  const bool tall = rows > cols;
  const int rm = ceil32(std::min(rows, cols)), rk = ceil32(std::max(rows, cols));
  char* base = static_cast<char*>(ws);
  auto take = [&](int64_t values) {
    uint16_t* q = reinterpret_cast<uint16_t*>(base);
    base += values * 2 * n;
    return q;
  };
  uint16_t *X = take(sp.x), *XT = take(sp.x), *XT2 = take(sp.x);
  uint16_t *A = take(sp.mm), *U = take(sp.mm), *P = take(sp.mm), *Q = take(sp.mm),
           *Q2 = take(sp.mm);
  double* part = reinterpret_cast<double*>(base);

  const Mats gm{g.data, g.ld, g.stride, g.dtype == MOE_BF16};
  const Mats wm{w.data, w.ld, w.stride, w.dtype == MOE_BF16};
  const Mats mm = mom ? Mats{mom->data, mom->ld, mom->stride, 0} : Mats{nullptr, 0, 0, 0};
  const int nparts = static_cast<int>(sp.part);
  const int64_t values = static_cast<int64_t>(rows) * cols;
  const int64_t chunk = (values + nparts - 1) / nparts;
  orth_norm_kernel<<<dim3(nparts, n), 256, 0, s>>>(gm, mm, d.mu, d.nesterov, rows, cols,
                                                   chunk, part);
  const int tr = (rows + 63) / 64, tc = (cols + 63) / 64;
  orth_split_kernel<<<dim3(tr * tc, n), 256, 0, s>>>(gm, mm, d.mu, d.nesterov, rows, cols, d.eps,
                                                     part, nparts, tall ? XT : X, tall ? X : XT,
                                                     sp.x, tc);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;

  const Out none{};
  // Symmetric m x m product: out = so (a b / (sa sb) + beta aux + gamma I).
  auto sym_args = [&](const uint16_t* a, const uint16_t* b, float sa, float sb, uint16_t* out,
                      float so, float alpha) {
    return Product{a, b, sp.mm, sp.mm, out, out, sp.mm, nullptr, alpha * so / (sa * sb), 0.f, 0.f};
  };
  auto sym = [&](const Product& p) { return launch_product<kSym>(p, nullptr, none, n, rm, rm, 2 * rm, s); };
  auto poly = [&](uint16_t* out) {  // P = aI + bA + cA^2
    Product p = sym_args(A, A, kScaleA, kScaleA, out, kScaleP, kC);
    p.aux = A;
    p.beta = kB * kScaleP / kScaleA;
    p.gamma = kA * kScaleP;
    return sym(p);
  };
  const Segments seg = segment_rule(wm.bf16, mom != nullptr, std::min(rows, cols));
  int left = d.steps;
  for (bool first = true; left > 0; first = false) {
    const int L = std::min(left, first ? seg.first : seg.later);
    left -= L;
    Product gram{X, X, sp.x, sp.x, A, A, sp.mm, nullptr, kScaleA / (kScaleX * kScaleX), 0.f, 0.f};
    if ((e = launch_product<kSym>(gram, nullptr, none, n, rm, rm, 2 * rk, s)) != hipSuccess) return e;
    uint16_t *q = Q, *q2 = Q2;
    if ((e = poly(q)) != hipSuccess) return e;
    const uint16_t* pl = q;  // the last P
    for (int i = 1; i < L; ++i) {
      // U = A P (with the product of the P so far, from the second step on),
      // A <- U P, the next P.
      Product u = sym_args(A, pl, kScaleA, kScaleP, U, kScaleA, 1.f);
      Product qq = sym_args(pl, q, kScaleP, kScaleP, q2, kScaleP, 1.f);
      e = launch_product<kSym>(u, i > 1 ? &qq : nullptr, none, n, rm, rm, 2 * rm, s);
      if (e != hipSuccess) return e;
      if (i > 1) std::swap(q, q2);
      if ((e = sym(sym_args(U, pl, kScaleA, kScaleP, A, kScaleA, 1.f))) != hipSuccess) return e;
      if ((e = poly(P)) != hipSuccess) return e;
      pl = P;
    }
    if (L > 1) {
      if ((e = sym(sym_args(pl, q, kScaleP, kScaleP, q2, kScaleP, 1.f))) != hipSuccess) return e;
      q = q2;
    }
    // X <- Q X: rows i and j of the result such that the caller's rows are j.
    const uint16_t *a = tall ? q : XT, *b = tall ? XT : q;
    Product x{a, b, tall ? sp.mm : sp.x, tall ? sp.x : sp.mm, tall ? XT2 : X, tall ? X : XT2,
              sp.x, nullptr, 0.f, 0.f, 0.f};
    const int ra = tall ? rm : rk, rb = tall ? rk : rm;
    if (left > 0) {
      x.alpha = 1.f / kScaleP;
      e = launch_product<kOperand>(x, nullptr, none, n, ra, rb, 2 * rm, s);
      std::swap(XT, XT2);
    } else {
      x.alpha = 1.f / (kScaleP * kScaleX);
      const Out o{wm, rows, cols, mom ? 1.f - d.lr * d.weight_decay : 0.f,
                  mom ? -d.lr * d.scale : 1.f, mom != nullptr};
      e = launch_product<kOut>(x, nullptr, o, n, ra, rb, 2 * rm, s);
    }
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace moe

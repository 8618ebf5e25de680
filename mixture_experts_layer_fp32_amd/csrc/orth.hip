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
#include <type_traits>

#include "moe_internal.h"
#include "moe_update.h"

namespace moe {
namespace {

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef __attribute__((address_space(3))) unsigned char lds_u8;

constexpr float kA = 3.4445f, kB = -4.7750f, kC = 2.0315f;
constexpr float kScaleX = 4096.f, kScaleA = 4096.f, kScaleP = 1024.f;
constexpr int kXcds = 8;
constexpr int kSmallTiles = 128;

struct Mats {  // moe_matrices on the device side
  void* data;
  int64_t ld, stride;
  int bf16;
};

__device__ __forceinline__ float load_el(const Mats& m, int64_t off) {
  return m.bf16 ? bf16_to_f32(static_cast<const uint16_t*>(m.data)[off])
                : static_cast<const float*>(m.data)[off];
}

// V adjacent values (4: aligned to their size).
template <int V>
__device__ __forceinline__ void load_v(const Mats& m, int64_t off, float (&f)[V]) {
  if constexpr (V == 1) {
    f[0] = load_el(m, off);
  } else if (m.bf16) {
    const uint2 r = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(m.data) + off);
    f[0] = __uint_as_float(r.x << 16);
    f[1] = __uint_as_float(r.x & 0xffff0000u);
    f[2] = __uint_as_float(r.y << 16);
    f[3] = __uint_as_float(r.y & 0xffff0000u);
  } else {
    const float4 r = *reinterpret_cast<const float4*>(static_cast<const float*>(m.data) + off);
    f[0] = r.x; f[1] = r.y; f[2] = r.z; f[3] = r.w;
  }
}

// ---- norm: partial sums of squares; the momentum -----------------------------
// Partial sums in fp64 (no overflow or underflow of squares). With mom.data
// the momentum is updated and the norm is that of U. Bound by memory.
template <int V>
__global__ __launch_bounds__(256) void orth_norm_kernel(Mats g, Mats mom, float mu, int nesterov,
                                                        int rows, int cols, int64_t chunk,
                                                        double* __restrict__ part) {
  const int b = blockIdx.y;
  const int64_t e1 = min((blockIdx.x + 1) * chunk, static_cast<int64_t>(rows) * cols);
  int64_t e = blockIdx.x * chunk + threadIdx.x * V;  // chunk is a multiple of 4
  // Row and column of e, carried along.
  int64_t r = e / cols;
  int c = static_cast<int>(e - r * cols);
  const int step_r = 256 * V / cols, step_c = 256 * V % cols;
  double s = 0.0;
#pragma unroll 4
  for (; e < e1; e += 256 * V) {
    float u[V];
    load_v<V>(g, b * g.stride + r * g.ld + c, u);
    if (mom.data != nullptr) {
      const int64_t at = b * mom.stride + r * mom.ld + c;
      float m[V];
      load_v<V>(mom, at, m);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        m[i] = fmaf(mu, m[i], u[i]);
        u[i] = nesterov ? fmaf(mu, m[i], u[i]) : m[i];
      }
      float* mp = static_cast<float*>(mom.data) + at;
      if constexpr (V == 4)
        *reinterpret_cast<float4*>(mp) = make_float4(m[0], m[1], m[2], m[3]);
      else
        *mp = m[0];
    }
#pragma unroll
    for (int i = 0; i < V; ++i) s += static_cast<double>(u[i]) * u[i];
    r += step_r;
    c += step_c;
    if (c >= cols) {
      c -= cols;
      ++r;
    }
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
// One 64 x 64 tile of U a workgroup, through LDS. Bound by memory.
template <int V>
__global__ __launch_bounds__(256) void orth_split_kernel(
    Mats g, Mats mom, float mu, int nesterov, int rows, int cols, float eps,
    const double* __restrict__ part, int nparts, uint16_t* __restrict__ u_planes,
    uint16_t* __restrict__ ut_planes, int64_t plane_stride, int tiles_c) {
  __shared__ float tile[64][65];
  __shared__ double red[4];
  const int b = gridDim.y - 1 - blockIdx.y, tid = threadIdx.x;
  const int r0 = (blockIdx.x / tiles_c) * 64, c0 = (blockIdx.x % tiles_c) * 64;
  // The tile's values are on their way while the norm is summed.
  constexpr int NL = 64 * 64 / (256 * V);
  float u[NL][V];
#pragma unroll
  for (int i = 0; i < NL; ++i) {
    const int x = (tid + 256 * i) * V, r = r0 + (x >> 6), c = c0 + (x & 63);
#pragma unroll
    for (int k = 0; k < V; ++k) u[i][k] = 0.f;
    if (r < rows && c < cols) {
      load_v<V>(g, b * g.stride + r * g.ld + c, u[i]);
      if (mom.data != nullptr) {
        float m[V];
        load_v<V>(mom, b * mom.stride + r * mom.ld + c, m);
#pragma unroll
        for (int k = 0; k < V; ++k) u[i][k] = nesterov ? fmaf(mu, m[k], u[i][k]) : m[k];
      }
    }
  }
  double s = 0.0;
  for (int i = tid; i < nparts; i += 256) s += part[static_cast<int64_t>(b) * nparts + i];
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) s += __shfl_xor(s, off, 64);
  if ((tid & 63) == 0) red[tid >> 6] = s;
  __syncthreads();
  const double inv =
      static_cast<double>(kScaleX) / (sqrt(red[0] + red[1] + red[2] + red[3]) + eps);
#pragma unroll
  for (int i = 0; i < NL; ++i) {
    const int x = (tid + 256 * i) * V;
#pragma unroll
    for (int k = 0; k < V; ++k) tile[x >> 6][(x & 63) + k] = static_cast<float>(u[i][k] * inv);
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
// Out-of-range offsets write zeros. Counted by vmcnt. (s_nop: a copy needs one
// wait state behind a write of M0, which nobody adds to assembly.)
__device__ __forceinline__ void dma16(__amdgpu_buffer_rsrc_t rsrc, int voff, int soff,
                                      unsigned lds_base) {
  asm volatile("s_mov_b32 m0, %3\n\ts_nop 0\n\tbuffer_load_dwordx4 %0, %1, %2 offen lds"
               :: "v"(voff), "s"(rsrc), "s"(soff), "s"(lds_base) : "memory", "m0");
}
#pragma clang diagnostic pop

// s_waitcnt immediates: at most n vector memory operations outstanding; none,
// and no LDS operation either.
constexpr int vmcnt_imm(int n) { return (n & 15) | (7 << 4) | (15 << 8) | ((n >> 4) << 14); }
constexpr int kVm0Lgkm0 = 7 << 4;
constexpr int kOutOfRange = 0x7FFF0000;  // past every operand tile (below 2^28 bytes)

// Four values as fp16 parts, two packed conversions each (to nearest even).
struct Parts {
  uint2 hi, lo;
};
__device__ __forceinline__ Parts split4(const float (&v)[4]) {
  const f16x2 h0 = __builtin_convertvector(f32x2{v[0], v[1]}, f16x2);
  const f16x2 h1 = __builtin_convertvector(f32x2{v[2], v[3]}, f16x2);
  const f16x2 l0 = __builtin_convertvector(
      f32x2{v[0] - static_cast<float>(h0[0]), v[1] - static_cast<float>(h0[1])}, f16x2);
  const f16x2 l1 = __builtin_convertvector(
      f32x2{v[2] - static_cast<float>(h1[0]), v[3] - static_cast<float>(h1[1])}, f16x2);
  return {uint2{__builtin_bit_cast(uint32_t, h0), __builtin_bit_cast(uint32_t, h1)},
          uint2{__builtin_bit_cast(uint32_t, l0), __builtin_bit_cast(uint32_t, l1)}};
}

// 4x4 transpose inside each group of 4 lanes: before, lane l's v[s] is row s,
// column l % 4; after, it is row l % 4, column s.
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

// The same for four 16-bit values.
__device__ __forceinline__ uint2 transpose4(uint2 w, int quad) {
  auto dpp = [](uint32_t v, auto ctrl) {
    return static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(v),
                                                          decltype(ctrl)::value, 0xF, 0xF, false));
  };
  const bool up = (quad & 2) != 0;
  // Lanes 0, 1 take rows 0, 1 of lanes 2, 3 and give them rows 2, 3.
  uint32_t keep = up ? w.y : w.x;
  uint32_t got = dpp(up ? w.x : w.y, std::integral_constant<int, 0x4E>{});
  // Even lanes take the lower halves of both of the pair, odd lanes the upper.
  const uint32_t sel = (quad & 1) ? 0x03020706u : 0x05040100u;
  keep = __builtin_amdgcn_perm(dpp(keep, std::integral_constant<int, 0xB1>{}), keep, sel);
  got = __builtin_amdgcn_perm(dpp(got, std::integral_constant<int, 0xB1>{}), got, sel);
  return up ? uint2{got, keep} : uint2{keep, got};
}

__device__ __forceinline__ void store_parts(uint16_t* frag, int lane, int j, const Parts& v) {
  *reinterpret_cast<uint2*>(frag + lane * 8 + j) = v.hi;
  *reinterpret_cast<uint2*>(frag + 512 + lane * 8 + j) = v.lo;
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
  int flip;  // each XCD's tiles last to first
};
struct Out {  // kOut: matrix row i, column j
  Mats w;
  int rows, cols;
  float keep, add;  // w <- keep w + add O (muon), or w <- add O
  int muon;
  int vec4;  // groups of four columns are aligned to their size
};

enum Epilogue { kSym = 0, kOperand = 1, kOut = 2 };

// Tile of this workgroup: matrix, first 32-row blocks of a and b; false past
// the last tile. Tiles of B x B blocks in eight runs, one an XCD (workgroup b
// runs on XCD b % 8), matrix by matrix; symmetric results have the tiles on
// and below the diagonal only.
struct Tile {
  int mat, a0, b0;
};
template <int EPI, int BA, int BB>
__device__ __forceinline__ bool find_tile(int n, int ra, int rb, int flip, Tile& t) {
  const int ta = (ra + BA - 1) / BA, tb = (rb + BB - 1) / BB;
  const int per_mat = EPI == kSym ? ta * (ta + 1) / 2 : ta * tb;
  const int total = per_mat * n, per = (total + kXcds - 1) / kXcds;
  const int slot = static_cast<int>(blockIdx.x) / kXcds;
  const int u = (static_cast<int>(blockIdx.x) % kXcds) * per + (flip ? per - 1 - slot : slot);
  if (u >= total) return false;
  t.mat = u / per_mat;
  const int lt = u - t.mat * per_mat;
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
  t.a0 = ti * BA;
  t.b0 = tj * BB;
  return true;
}

// Register groups q0 .. q0 + NQ - 1 of one 32 x 32 block (ib, jb): acc[q][s]
// of lane l is row 8 (q0 + q) + 4 (l / 32) + s of the a block and row l % 32
// of the b block. kSym: blocks above the diagonal are left to their mirror
// images.
template <int EPI, int NQ>
__device__ __forceinline__ void store_block(const Product& p, const Out& o, int mat, int ra,
                                            int rb, int ib, int jb, int q0,
                                            const float (&acc)[NQ][4], int lane) {
  if (EPI == kSym && ib < jb) return;
  const int half = lane >> 5, l32 = lane & 31;
  if constexpr (EPI == kOut) {
    const bool whole = (ib + 1) * 32 <= o.rows && (jb + 1) * 32 <= o.cols;
    if (whole && o.vec4) {
      // Four lanes exchange their values: a lane gets four columns of one row.
      const int64_t at = mat * o.w.stride +
                         static_cast<int64_t>(ib * 32 + 8 * q0 + 4 * half + (lane & 3)) * o.w.ld +
                         jb * 32 + 4 * (l32 >> 2);
      float w[NQ][4];
#pragma unroll
      for (int q = 0; q < NQ; ++q) {
        const int64_t e = at + 8 * q * o.w.ld;
#pragma unroll
        for (int s = 0; s < 4; ++s) w[q][s] = 0.f;
        if (o.muon && o.w.bf16) {
          const uint2 r = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(o.w.data) + e);
          w[q][0] = __uint_as_float(r.x << 16);
          w[q][1] = __uint_as_float(r.x & 0xffff0000u);
          w[q][2] = __uint_as_float(r.y << 16);
          w[q][3] = __uint_as_float(r.y & 0xffff0000u);
        } else if (o.muon) {
          const float4 r = *reinterpret_cast<const float4*>(static_cast<const float*>(o.w.data) + e);
          w[q][0] = r.x; w[q][1] = r.y; w[q][2] = r.z; w[q][3] = r.w;
        }
      }
#pragma unroll
      for (int q = 0; q < NQ; ++q) {
        const int64_t e = at + 8 * q * o.w.ld;
        float v[4] = {acc[q][0], acc[q][1], acc[q][2], acc[q][3]};
        transpose4(v, lane & 3);
#pragma unroll
        for (int s = 0; s < 4; ++s) v[s] = fmaf(o.keep, w[q][s], o.add * (v[s] * p.alpha));
        if (o.w.bf16) {
          const bf16x2 b0 = __builtin_convertvector(f32x2{v[0], v[1]}, bf16x2);
          const bf16x2 b1 = __builtin_convertvector(f32x2{v[2], v[3]}, bf16x2);
          *reinterpret_cast<uint2*>(static_cast<uint16_t*>(o.w.data) + e) =
              uint2{__builtin_bit_cast(uint32_t, b0), __builtin_bit_cast(uint32_t, b1)};
        } else {
          *reinterpret_cast<float4*>(static_cast<float*>(o.w.data) + e) =
              make_float4(v[0], v[1], v[2], v[3]);
        }
      }
      return;
    }
    // Lanes run along the caller's columns.
    const int r0 = ib * 32 + 8 * q0 + 4 * half, c = jb * 32 + l32;
    const int64_t at = mat * o.w.stride + r0 * o.w.ld + c;
    auto ok = [&](int q, int s) { return r0 + 8 * q + s < o.rows && c < o.cols; };
    auto off = [&](int q, int s) { return at + (8 * q + s) * o.w.ld; };
    float w[NQ][4];
#pragma unroll
    for (int q = 0; q < NQ; ++q)
#pragma unroll
      for (int s = 0; s < 4; ++s)
        w[q][s] = o.muon && ok(q, s) ? load_el(o.w, off(q, s)) : 0.f;
#pragma unroll
    for (int q = 0; q < NQ; ++q)
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        const float v = fmaf(o.keep, w[q][s], o.add * (acc[q][s] * p.alpha));
        if (!ok(q, s)) continue;
        if (o.w.bf16)
          static_cast<__bf16*>(o.w.data)[off(q, s)] = static_cast<__bf16>(v);  // to nearest even
        else
          static_cast<float*>(o.w.data)[off(q, s)] = v;
      }
  } else {
    // Operand with rows j, its depth i: four adjacent values a lane.
    auto frag = [&](int q) {
      return (static_cast<int64_t>(jb) * (2 * ra) + 2 * ib + ((q0 + q) >> 1)) * 1024;
    };
    auto slot = [&](int q) { return l32 + 32 * ((q0 + q) & 1); };
    union Half4 {
      uint2 w;
      _Float16 h[4];
    };
    Half4 hi[NQ], lo[NQ];
    const bool add = EPI == kSym && p.aux != nullptr;
    if (add) {
#pragma unroll
      for (int q = 0; q < NQ; ++q) {
        const uint16_t* x = p.aux + mat * p.so + frag(q) + slot(q) * 8 + 4 * half;
        hi[q].w = *reinterpret_cast<const uint2*>(x);
        lo[q].w = *reinterpret_cast<const uint2*>(x + 512);
      }
    }
#pragma unroll
    for (int q = 0; q < NQ; ++q) {
      float v[4];
#pragma unroll
      for (int s = 0; s < 4; ++s) v[s] = acc[q][s] * p.alpha;
      if (add) {
#pragma unroll
        for (int s = 0; s < 4; ++s) {
          const float x = static_cast<float>(hi[q].h[s]) + static_cast<float>(lo[q].h[s]);
          v[s] = fmaf(p.beta, x, v[s]);
          if (ib == jb && 8 * (q0 + q) + 4 * half + s == l32) v[s] += p.gamma;
        }
      }
      Parts w = split4(v);
      store_parts(p.out_t + mat * p.so + frag(q), slot(q), 4 * half, w);
      if (EPI == kOperand || ib != jb) {
        // Operand with rows i, its depth j.
        w.hi = transpose4(w.hi, lane & 3);
        w.lo = transpose4(w.lo, lane & 3);
        const int j0 = 4 * (l32 >> 2), row = 8 * (q0 + q) + 4 * half + (lane & 3);
        const int64_t fn = (static_cast<int64_t>(ib) * (2 * rb) + 2 * jb + (j0 >> 4)) * 1024;
        store_parts(p.out_n + mat * p.so + fn, row + 32 * ((j0 >> 3) & 1), j0 & 7, w);
      }
    }
  }
}

// kSym: the result is symmetric: tiles on and below the diagonal only;
//   alpha D + beta aux + gamma I is stored into out_t, and its mirror image.
// kOperand: alpha D is stored into out_t and out_n.
// kOut: to the caller's matrices (rows i, columns j).
// blockIdx.y: one of two independent products.
// Every product has both fp16 parts, the last one of a bf16 result too: its high
// parts alone (11 bits) put O off by 3e-4 at full rank and by 3.3e-3 below it,
// where Q is near 11.9 I off the gradient's range and all of its diagonal rounds
// the same way, twice bf16's own rounding.
template <int EPI, int WM, int WN, int WR, int WC>
__global__ __launch_bounds__(64 * WR * WC) void orth_product_kernel(Product p0, Product p1,
                                                                   Out o, int n, int ra, int rb,
                                                                   int KS) {
  constexpr int BA = WR * WM, BB = WC * WN;    // 32-row blocks per tile
  constexpr int NW = WR * WC;
  constexpr int SS = 2;                        // slices a step
  constexpr int kStage = (BA + BB) * 4096;
  constexpr int NC = (BA + BB) * 4 / NW;       // 1 KB copies per wave and step
  static_assert((BA + BB) * 4 % NW == 0 && BA * 4 % NC == 0, "copies are shared out evenly");
  static_assert(EPI != kSym || BA == BB, "symmetric results use square tiles");
  __shared__ __attribute__((aligned(1024))) unsigned char smem[2 * kStage];

  const Product& p = blockIdx.y == 0 ? p0 : p1;
  Tile t;
  if (!find_tile<EPI, BA, BB>(n, ra, rb, p.flip, t)) return;
  const int mat = t.mat, a0 = t.a0, b0 = t.b0;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  // Waves w and w + 4 share a SIMD; their regions are paired so that on
  // diagonal tiles of 256, where regions 0 and 5 are half and 1 and 3 not
  // computed, no SIMD has more than one and a half.
  static_assert(NW == 8, "eight regions");
  const int region = (0x31507642 >> (4 * wave)) & 7;
  const int wr = region / WC, wc = region % WC;

  // ---- copies: a step is 4 (BA + BB) pieces of 1 KB, four a row block; each
  // wave copies NC of them, all of one operand ----
  const int row_bytes = KS * 2048;
  const bool copy_a = wave * NC < BA * 4;
  const int piece0 = wave * NC - (copy_a ? 0 : BA * 4);
  const uint16_t* src = copy_a ? p.a + mat * p.sa + static_cast<int64_t>(a0) * KS * 1024
                               : p.b + mat * p.sb + static_cast<int64_t>(b0) * KS * 1024;
  const __amdgpu_buffer_rsrc_t rsrc = __builtin_amdgcn_make_buffer_rsrc(
      (void*)src, 0, (copy_a ? min(BA, ra - a0) : min(BB, rb - b0)) * row_bytes, 0x00020000);
  int voff[NC];
#pragma unroll
  for (int i = 0; i < NC; ++i)
    voff[i] = ((piece0 + i) >> 2) * row_bytes + ((piece0 + i) & 3) * 1024 + lane * 16;
  const unsigned lds_w = (unsigned)(uintptr_t)(lds_u8*)smem + wave * NC * 1024;
  const int nk = KS / SS;  // KS is even
  // A copy past the last slice is still issued, out of range (it writes
  // zeros), so the K loop has no branch around it.
  auto copy = [&](int i, int kt) {
    dma16(rsrc, kt < nk ? voff[i] : kOutOfRange, kt * (SS * 2048),
          lds_w + (kt & 1) * kStage + i * 1024);
  };

  f32x16 acc[WM][WN];
#pragma unroll
  for (int i = 0; i < WM; ++i)
#pragma unroll
    for (int j = 0; j < WN; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;

  // The K loop over the wave's first NJ block columns.
  auto run = [&](auto nj_c) {
    constexpr int NJ = decltype(nj_c)::value;
    // Fragments of half a step: WM of a, then NJ of b, [hi, lo] of one slice each.
    constexpr int NF = NJ > 0 ? 2 * (WM + NJ) : 0, NM = 3 * WM * NJ;
    f16x8 fr[2][NF > 0 ? NF : 1];
    auto read = [&](int f, int kt, int ks) {
      const int blk = f / 2 < WM ? wr * WM + f / 2 : BA + wc * WN + f / 2 - WM;
      fr[ks][f] = *reinterpret_cast<const f16x8*>(smem + (kt & 1) * kStage + blk * 4096 +
                                                  ks * 2048 + (f & 1) * 1024 + lane * 16);
    };
    // Products of half a step, of a slice in the order lo hi, hi lo, hi hi;
    // `side(x)` for x in [0, n) is spread between them.
    auto multiply = [&](int ks, int n, auto side) {
      if constexpr (NM == 0) {
#pragma unroll
        for (int y = 0; y < n; ++y) side(y);
      } else {
#pragma unroll
        for (int x = 0; x < NM; ++x) {
          const int q = x / (WM * NJ), i = x / NJ % WM, j = x % NJ;
#pragma unroll
          for (int y = x * n / NM; y < (x + 1) * n / NM; ++y) side(y);
          __builtin_amdgcn_sched_barrier(0);
          acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(
              fr[ks][2 * i + (q == 0)], fr[ks][2 * (WM + j) + (q == 1)], acc[i][j], 0, 0, 0);
          __builtin_amdgcn_sched_barrier(0);
        }
      }
    };
#pragma unroll
    for (int i = 0; i < NC; ++i) copy(i, 0);
#pragma unroll
    for (int i = 0; i < NC; ++i) copy(i, 1);
    __builtin_amdgcn_s_waitcnt(vmcnt_imm(NC));
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");  // no LDS read moves above the barrier
#pragma unroll
    for (int f = 0; f < NF; ++f) read(f, 0, 0);
    for (int kt = 0; kt < nk; ++kt) {
      // First slice, with the reads of the second in between.
      multiply(0, NF, [&](int f) { read(f, kt, 1); });
      // This wave's reads of the step's slot are done and its copies of the
      // next step have landed; after the barrier every wave's. The slot takes
      // step kt + 2, a whole step before it is needed, while the second slice
      // is multiplied and the next step's first slice is read.
      __builtin_amdgcn_s_waitcnt(kVm0Lgkm0);
      __builtin_amdgcn_s_barrier();
      asm volatile("" ::: "memory");
      multiply(1, NF + NC, [&](int y) {
        if (y < NF)
          read(y, kt + 1, 0);
        else
          copy(y - NF, kt + 2);
      });
    }
    __builtin_amdgcn_s_waitcnt(kVm0Lgkm0);  // no copy is left when the wave ends
  };
  // Symmetric results, tiles on the diagonal: a wave whose blocks all lie above
  // it only copies, one whose second half does leaves that out. The card's
  // clock is bound by its power here, so work left out is time.
  const int above = EPI == kSym && a0 == b0 ? wr * WM + WM - 1 : BB;  // last row block
  if (EPI == kSym && wc * WN > above)
    run(std::integral_constant<int, 0>{});
  else if (EPI == kSym && WN == 4 && wc * WN + WN / 2 > above)
    run(std::integral_constant<int, EPI == kSym && WN == 4 ? WN / 2 : WN>{});
  else
    run(std::integral_constant<int, WN>{});

#pragma unroll
  for (int i = 0; i < WM; ++i) {
    const int ib = a0 + wr * WM + i;
    if (ib >= ra) continue;
#pragma unroll
    for (int j = 0; j < WN; ++j) {
      const int jb = b0 + wc * WN + j;
      if (jb >= rb) continue;
      float v[4][4];
#pragma unroll
      for (int r = 0; r < 16; ++r) v[r / 4][r % 4] = acc[i][j][r];
      store_block<EPI, 4>(p, o, mat, ra, rb, ib, jb, 0, v, lane);
    }
  }
}

// ---- products with few tiles ---------------------------------------------------
// 64 x 64 tiles whose depth is shared out over the 8 waves of a workgroup,
// slice by slice; each wave reads its fragments straight into registers (two
// buffers of two slices), so there is no barrier until the waves' sums meet
// in LDS, and the time is that of a few loads. Also the more exact sum: eight
// parts instead of one chain. With more tiles than CUs four waves a workgroup,
// two workgroups a CU (6 x 700^2 339 -> 322 us, 64 x 160^2 166 -> 142).

// Slices [ks0, ks1) of the tile whose operand blocks (two of a, two of b; this
// lane's values) begin at src, shared out over NW waves (8 or 4). v: the
// wave's 16 / NW register groups of block 4 wave / NW, summed over the waves.
template <int NW>
using SmallSums = float[NW][4][4][64][4];  // wave, block, register group, lane
template <int NW>
__device__ __forceinline__ void small_tile(const uint16_t* const (&src)[4], int ks0, int ks1,
                                           int wave, int lane, SmallSums<NW>& part,
                                           float (&v)[16 / NW][4]) {
  f32x16 acc[2][2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;
  f16x8 fr[2][2][4][2];  // buffer, slice, operand block, part
  auto load = [&](int buf, int ks) {
#pragma unroll
    for (int u = 0; u < 2; ++u)
      if (ks + NW * u < ks1) {
#pragma unroll
        for (int b = 0; b < 4; ++b)
#pragma unroll
          for (int q = 0; q < 2; ++q)
            fr[buf][u][b][q] = *reinterpret_cast<const f16x8*>(
                src[b] + static_cast<int64_t>(ks + NW * u) * 1024 + q * 512);
      }
  };
  auto multiply = [&](int buf, int ks) {
#pragma unroll
    for (int u = 0; u < 2; ++u)
      if (ks + NW * u < ks1) {
#pragma unroll
        for (int q = 0; q < 3; ++q)
#pragma unroll
          for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j)
              acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(
                  fr[buf][u][i][q == 0], fr[buf][u][2 + j][q == 1], acc[i][j], 0, 0, 0);
      }
  };
  load(0, ks0 + wave);
  load(1, ks0 + wave + 2 * NW);
  for (int ks = ks0 + wave; ks < ks1; ks += 4 * NW) {
    multiply(0, ks);
    load(0, ks + 4 * NW);
    multiply(1, ks + 2 * NW);
    load(1, ks + 6 * NW);
  }
#pragma unroll
  for (int b = 0; b < 4; ++b)
#pragma unroll
    for (int q = 0; q < 4; ++q)
      *reinterpret_cast<float4*>(part[wave][b][q][lane]) =
          make_float4(acc[b / 2][b % 2][4 * q], acc[b / 2][b % 2][4 * q + 1],
                      acc[b / 2][b % 2][4 * q + 2], acc[b / 2][b % 2][4 * q + 3]);
  __syncthreads();
  const int b = 4 * wave / NW, q0 = 16 / NW * wave % 4;
#pragma unroll
  for (int q = 0; q < 16 / NW; ++q)
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      v[q][s] = 0.f;
#pragma unroll
      for (int w = 0; w < NW; ++w) v[q][s] += part[w][b][q0 + q][lane][s];
    }
}

template <int EPI, int NW>
__global__ __launch_bounds__(64 * NW) void orth_product_small_kernel(Product p0, Product p1, Out o,
                                                                 int n, int ra, int rb, int KS) {
  __shared__ __attribute__((aligned(16))) SmallSums<NW> part;
  const Product& p = blockIdx.y == 0 ? p0 : p1;
  Tile t;
  if (!find_tile<EPI, 2, 2>(n, ra, rb, p.flip, t)) return;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  // Row blocks past the last read the last one again (they are not stored).
  const uint16_t* src[4];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    src[i] = p.a + t.mat * p.sa + static_cast<int64_t>(min(t.a0 + i, ra - 1)) * KS * 1024 + lane * 8;
    src[2 + i] = p.b + t.mat * p.sb + static_cast<int64_t>(min(t.b0 + i, rb - 1)) * KS * 1024 + lane * 8;
  }
  float v[16 / NW][4];
  small_tile<NW>(src, 0, KS, wave, lane, part, v);
  const int b = 4 * wave / NW, ib = t.a0 + b / 2, jb = t.b0 + b % 2;
  if (ib >= ra || jb >= rb) return;
  store_block<EPI, 16 / NW>(p, o, t.mat, ra, rb, ib, jb, 16 / NW * wave % 4, v, lane);
}

// ---- short sides up to 128 -------------------------------------------------------
// X X^T of matrices with at most four row blocks: one or three 64 x 64 tiles,
// the depth split over the workgroups too. Sums in fp32, for the next kernel:
// gram[matrix][split][tile][wave][2][lane][4].
constexpr int kGramTile = 4096;  // floats
__global__ __launch_bounds__(512) void orth_gram_kernel(const uint16_t* __restrict__ x, int64_t sx,
                                                        int rm, int KS, int tiles, int splits,
                                                        float* __restrict__ gram) {
  __shared__ __attribute__((aligned(16))) SmallSums<8> part;
  const int sp = blockIdx.x / tiles, tile = blockIdx.x % tiles, mat = blockIdx.y;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int a0 = tile == 0 ? 0 : 2, b0 = tile == 2 ? 2 : 0;  // (0, 0), (2, 0), (2, 2)
  const uint16_t* src[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int rb = min((i < 2 ? a0 : b0) + (i & 1), rm - 1);
    src[i] = x + mat * sx + static_cast<int64_t>(rb) * KS * 1024 + lane * 8;
  }
  float v[2][4];
  small_tile<8>(src, KS * sp / splits, KS * (sp + 1) / splits, wave, lane, part, v);
  float* out = gram + ((static_cast<int64_t>(mat) * splits + sp) * tiles + tile) * kGramTile +
               wave * 512 + lane * 4;
#pragma unroll
  for (int q = 0; q < 2; ++q)
    *reinterpret_cast<float4*>(out + q * 256) = make_float4(v[q][0], v[q][1], v[q][2], v[q][3]);
}

// Blocks of X^T a workgroup of the steps kernel has at most, by row blocks of X:
// one a wave and row block; as many as its LDS holds; and most Gram parts.
constexpr int steps_xb(int mb) { return mb == 1 ? 16 : mb == 2 ? 8 : 4; }
constexpr int steps_staged(int mb) { return mb == 4 ? 2 : 4; }  // 48 KB or less
constexpr int gram_parts(int mb) { return mb <= 2 ? 32 : 16; }

// Row block of the w-th block on or below the diagonal: (0, 0), (1, 0), (1, 1),
// (2, 0), ...
__device__ __forceinline__ int sym_row(int w) { return w >= 6 ? 3 : w >= 3 ? 2 : w >= 1 ? 1 : 0; }

// The matrix of this workgroup and which of the matrix's `groups` workgroups it
// is; false past the last. runs > 0: a grid of one dimension in eight runs, one
// an XCD (workgroup b runs on XCD b % 8), so that a matrix's workgroups share
// the L2 that has what all of them read (8 x 128 x 512 75.8 -> 63.6 us, 8 x 32 x
// 4096 65 -> 48). Otherwise blockIdx is (group, matrix): where a matrix has one
// workgroup, or its Gram parts come from another kernel's order (50 x 972 x 36
// 102 us, in runs 106).
struct Group {
  int mat, index, groups;
};
__device__ __forceinline__ bool find_group(int n, int runs, Group& g) {
  if (runs == 0) {
    g = {static_cast<int>(blockIdx.y), static_cast<int>(blockIdx.x), static_cast<int>(gridDim.x)};
    return true;
  }
  const int total = n * runs, per = (total + kXcds - 1) / kXcds;
  const int u = static_cast<int>(blockIdx.x) % kXcds * per + static_cast<int>(blockIdx.x) / kXcds;
  g = {u / runs, u % runs, runs};
  return u < total;
}
int runs_of(int groups) { return groups > 1 ? groups : 0; }
dim3 group_grid(int n, int groups) {
  return groups > 1 ? dim3((n * groups + kXcds - 1) / kXcds * kXcds) : dim3(1, n);
}

// Block (ib, jb) in part sp of `parts` of a matrix's Gram product, as
// orth_gram_kernel lays it out (register group 2 h + q of block b in wave 2 b + h
// of its tile).
template <int MB>
__device__ __forceinline__ int64_t gram_at(int mat, int sp, int parts, int ib, int jb, int lane) {
  const int tile = ib / 2 * (ib / 2 + 1) / 2 + jb / 2, b = 2 * (ib & 1) + (jb & 1);
  return ((static_cast<int64_t>(mat) * parts + sp) * (MB > 2 ? 3 : 1) + tile) * kGramTile +
         b * 1024 + lane * 4;
}

// Block (ib, jb) of the Gram product of xs, an operand of MB row blocks and KS
// slices in LDS of which the first `slices` count, to g (gram_at).
template <int MB>
__device__ __forceinline__ void gram_part(const uint16_t* xs, int KS, int slices, int ib, int jb,
                                          int lane, float* __restrict__ g) {
  f32x16 acc;
#pragma unroll
  for (int r = 0; r < 16; ++r) acc[r] = 0.f;
#pragma unroll 2
  for (int ks = 0; ks < slices; ++ks) {
    auto at = [&](int rb, int part) {
      return *reinterpret_cast<const f16x8*>(xs + ((rb * KS + ks) * 2 + part) * 512 + lane * 8);
    };
    const f16x8 ah = at(ib, 0), al = at(ib, 1), bh = at(jb, 0), bl = at(jb, 1);
    acc = __builtin_amdgcn_mfma_f32_32x32x16_f16(al, bh, acc, 0, 0, 0);
    acc = __builtin_amdgcn_mfma_f32_32x32x16_f16(ah, bl, acc, 0, 0, 0);
    acc = __builtin_amdgcn_mfma_f32_32x32x16_f16(ah, bh, acc, 0, 0, 0);
  }
#pragma unroll
  for (int q = 0; q < 4; ++q)
    *reinterpret_cast<float4*>(g + q * 256) =
        make_float4(acc[4 * q], acc[4 * q + 1], acc[4 * q + 2], acc[4 * q + 3]);
}

// orth_split_kernel where the steps kernel gives the later Gram products: one
// workgroup has XB blocks of X's depth and all of its rows, writes X^T and
// gives its part of the first Gram product. X itself is not written. A launch
// less (4 x 64 x 512 42.6 -> 38.8 us, 512 x 64 x 64 68 -> 60; 8 x 128 x 512
// 75.2 -> 75.9, as many parts to add up as later). Bound by the latency of its
// loads and of the launch.
template <int V, int MB, bool TALL>
__global__ __launch_bounds__(1024) void orth_split_gram_kernel(
    Mats g, Mats mom, float mu, int nesterov, int rows, int cols, float eps,
    const double* __restrict__ part, int nparts, uint16_t* __restrict__ xt_planes,
    int64_t plane_stride, int rk, int n, int runs, float* __restrict__ gram) {
  constexpr int XB = steps_staged(MB), KS = 2 * XB;
  constexpr int TR = TALL ? 32 * XB : 32 * MB, TC = TALL ? 32 * MB : 32 * XB;  // of U
  __shared__ float tile[TR][TC + 1];
  __shared__ __attribute__((aligned(16))) uint16_t xs[MB * KS * 1024];
  __shared__ double red[16];
  Group me;
  if (!find_group(n, runs, me)) return;
  const int mat = me.mat, tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int x0 = me.index * XB, nb = min(XB, rk - x0);
  const int r0 = TALL ? 32 * x0 : 0, c0 = TALL ? 0 : 32 * x0;
  constexpr int NL = TR * TC / (1024 * V);
  static_assert(TR * TC % (1024 * V) == 0, "whole rounds");
  float u[NL][V];
#pragma unroll
  for (int i = 0; i < NL; ++i) {
    const int x = (tid + 1024 * i) * V, r = r0 + x / TC, c = c0 + x % TC;
#pragma unroll
    for (int k = 0; k < V; ++k) u[i][k] = 0.f;
    if (r < rows && c < cols) {
      load_v<V>(g, mat * g.stride + r * g.ld + c, u[i]);
      if (mom.data != nullptr) {
        float m[V];
        load_v<V>(mom, mat * mom.stride + r * mom.ld + c, m);
#pragma unroll
        for (int k = 0; k < V; ++k) u[i][k] = nesterov ? fmaf(mu, m[k], u[i][k]) : m[k];
      }
    }
  }
  double s = 0.0;
  for (int i = tid; i < nparts; i += 1024) s += part[static_cast<int64_t>(mat) * nparts + i];
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) s += __shfl_xor(s, off, 64);
  if (lane == 0) red[wave] = s;
  __syncthreads();
  s = 0.0;
#pragma unroll
  for (int w = 0; w < 16; ++w) s += red[w];
  const double inv = static_cast<double>(kScaleX) / (sqrt(s) + eps);
#pragma unroll
  for (int i = 0; i < NL; ++i) {
    const int x = (tid + 1024 * i) * V;
#pragma unroll
    for (int k = 0; k < V; ++k) tile[x / TC][x % TC + k] = static_cast<float>(u[i][k] * inv);
  }
  __syncthreads();
  auto x_at = [&](int i, int k) { return TALL ? tile[k][i] : tile[i][k]; };
  auto fragment = [&](uint16_t* out, auto value) {
    union {
      uint16_t h[8];
      uint4 v;
    } hi, lo;
#pragma unroll
    for (int j = 0; j < 8; ++j) split(value(8 * (lane >> 5) + j), hi.h[j], lo.h[j]);
    uint4* p = reinterpret_cast<uint4*>(out + lane * 8);
    p[0] = hi.v;
    p[64] = lo.v;
  };
  uint16_t* xt = xt_planes + mat * plane_stride + static_cast<int64_t>(x0) * (2 * MB) * 1024;
  for (int f = wave; f < MB * KS; f += 16) {  // X: row block f / KS
    const int i = 32 * (f / KS) + (lane & 31), k0 = 16 * (f % KS);
    fragment(xs + f * 1024, [&](int j) { return x_at(i, k0 + j); });
  }
  for (int f = wave; f < nb * 2 * MB; f += 16) {  // X^T: row block f / (2 MB)
    const int k = 32 * (f / (2 * MB)) + (lane & 31), i0 = 16 * (f % (2 * MB));
    fragment(xt + f * 1024, [&](int j) { return x_at(i0 + j, k); });
  }
  __syncthreads();
  const int ib = sym_row(wave), jb = wave - ib * (ib + 1) / 2;
  if (wave < MB * (MB + 1) / 2)
    gram_part<MB>(xs, KS, 2 * nb, ib, jb, lane,
                  gram + gram_at<MB>(mat, me.index, me.groups, ib, jb, lane));
}

// The rest of a segment in one launch. Every workgroup adds up the Gram
// product's parts, holds A and P of its matrix in LDS (MB 32-row blocks, at
// most 64 KB each), takes the segment's steps (1 or 2) there, and multiplies
// its share of X. The steps are repeated by every workgroup of a matrix: they
// take a few microseconds, a launch each would take more. A wave has one 32 x
// 32 block: of the m x m products those on and below the diagonal (10 of 16
// waves for MB = 4, at most 3 on a SIMD).
// kLoop: groups of XB blocks of X^T, g = index, index + groups, ...
// kStaged: one group of xbw blocks a workgroup, copied into LDS during the steps;
//   while the card has a CU for each (8 x 128 x 512 91 -> 81 us; 200 x 128 x 512,
//   as a loop of staged groups, 203 -> 220).
// kGram: staged, and the workgroup's blocks of the new X, still in LDS, give
//   its part of the next segment's Gram product: no launch for it, no X in
//   memory (8 x 128 x 512 81 -> 75 us, 32 x 128 x 256 94 -> 77). As many blocks
//   a workgroup as LDS holds, since every workgroup adds up all parts of its
//   matrix (8 x 128 x 512 as 8 parts 75 us, as 16 84), and up to gram_parts()
//   parts (16 parts of 16 x 128 x 1024 115 -> 94 us, of 4 x 128 x 1024 81 -> 83,
//   32 of 1 x 128 x 2048 72 -> 88; 30 of 4 x 64 x 3840 83 -> 67, 63 of 2 x 32 x
//   8000 75 -> 83). While a CU for each workgroup is there, or one
//   workgroup is all of a matrix (512 x 64 x 64 80 -> 67 us; 60 x 128 x 512, 480
//   workgroups, 133 -> 190: the steps are repeated in each).
// SWAP: the result's rows are those of Q (kOut of a wide matrix).
// Where a launch's time goes (copies without each part in turn), MB = 4, kGram,
// one step, eight Gram parts (8 x 128 x 512): 11.4 us, of it the launch 3.2,
// copying X^T 0.2, the Gram parts 2.1, the step's product 2.8, Q X with its stores
// 2.0, the next Gram part 1.2. Two steps, four parts (8 x 256 x 128): 18.7 us, of
// it 3.2, 0.1, 0.9, the five products 12.0, 1.7 and 0.8. Each part is a chain of a
// few dependent loads or products; none is bound by a rate.
enum XGroups { kLoop = 0, kStaged = 1, kGram = 2 };
template <int MB, int EPI, bool SWAP, int MODE>
__global__ __launch_bounds__(1024) void orth_steps_kernel(Product p, Out o, int steps, int rk,
                                                          int xbw, int n, int runs, const float* __restrict__ gram,
                                                          int splits,
                                                          float* __restrict__ next_gram) {
  constexpr bool STAGED = MODE != kLoop;
  static_assert(MODE != kGram || (EPI == kOperand && !SWAP), "the next segment's operand");
  constexpr int KS = 2 * MB, MP = MB == 3 ? 4 : MB, XB = steps_xb(MB);
  constexpr int kOp = MB * KS * 1024;  // values of an operand
  __shared__ __attribute__((aligned(1024))) uint16_t bufs[2][kOp];
  __shared__ __attribute__((aligned(1024))) uint16_t
      xs[STAGED ? steps_staged(MB) * KS * 1024 : 8];
  uint16_t *ba = bufs[0], *bp = bufs[1];
  Group me;
  if (!find_group(n, runs, me)) return;
  const int mat = me.mat, lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int half = lane >> 5, l32 = lane & 31;
  auto frag = [&](const uint16_t* op, int rb, int ks, int part) {
    return *reinterpret_cast<const f16x8*>(op + ((rb * KS + ks) * 2 + part) * 512 + lane * 8);
  };
  f32x16 acc;
  // acc += (hi + lo of a) (hi + lo of b)
  auto mma = [&](const f16x8& ah, const f16x8& al, const f16x8& bh, const f16x8& bl) {
    acc = __builtin_amdgcn_mfma_f32_32x32x16_f16(al, bh, acc, 0, 0, 0);
    acc = __builtin_amdgcn_mfma_f32_32x32x16_f16(ah, bl, acc, 0, 0, 0);
    acc = __builtin_amdgcn_mfma_f32_32x32x16_f16(ah, bh, acc, 0, 0, 0);
  };
  auto zero = [&]() {
#pragma unroll
    for (int r = 0; r < 16; ++r) acc[r] = 0.f;
  };
  // A block of X^T.
  f16x8 x[KS][2];
  auto load_x = [&](int xb) {
    const uint16_t* src = p.a + mat * p.sa + static_cast<int64_t>(xb) * (KS * 1024) + lane * 8;
#pragma unroll
    for (int ks = 0; ks < KS; ++ks)
#pragma unroll
      for (int q = 0; q < 2; ++q)
        x[ks][q] = *reinterpret_cast<const f16x8*>(src + (ks * 2 + q) * 512);
  };
  // Block (ib, jb) of the m x m results.
  const int ib = sym_row(wave), jb = wave - ib * (ib + 1) / 2;
  const bool mine = wave < MB * (MB + 1) / 2;
  auto product = [&](const uint16_t* a, const uint16_t* b) {
    zero();
    if (!mine) return;
#pragma unroll 4
    for (int ks = 0; ks < KS; ++ks)
      mma(frag(a, ib, ks, 0), frag(a, ib, ks, 1), frag(b, jb, ks, 0), frag(b, jb, ks, 1));
  };
  // Values of register group q, rows jb and depth ib of the operand's layout.
  auto place = [&](int q) {
    return ((jb * KS + 2 * ib + (q >> 1)) * 2) * 512 + (l32 + 32 * (q & 1)) * 8 + 4 * half;
  };
  auto polynomial = [&](const uint16_t* a) {  // acc <- a I + b A + c A^2, as kScaleP holds it
    if (!mine) return;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const _Float16* h = reinterpret_cast<const _Float16*>(a + place(q));
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        const float av = static_cast<float>(h[s]) + static_cast<float>(h[512 + s]);
        float v = fmaf(kB * kScaleP / kScaleA, av,
                       acc[4 * q + s] * (kC * kScaleP / (kScaleA * kScaleA)));
        if (ib == jb && 8 * q + 4 * half + s == l32) v += kA * kScaleP;
        acc[4 * q + s] = v;
      }
    }
  };
  auto store = [&](uint16_t* op, float alpha) {  // and the mirror image
    if (!mine) return;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      float v[4];
#pragma unroll
      for (int s = 0; s < 4; ++s) v[s] = acc[4 * q + s] * alpha;
      Parts w = split4(v);
      store_parts(op + place(q), 0, 0, w);
      if (ib != jb) {
        w.hi = transpose4(w.hi, lane & 3);
        w.lo = transpose4(w.lo, lane & 3);
        const int j0 = 4 * (l32 >> 2), row = 8 * q + 4 * half + (lane & 3);
        store_parts(op + ((ib * KS + 2 * jb + (j0 >> 4)) * 2) * 512, row + 32 * ((j0 >> 3) & 1),
                    j0 & 7, w);
      }
    }
  };
  constexpr int TILES = MB > 2 ? 3 : 1;
  const int nb = STAGED ? min(xbw, rk - me.index * xbw) : 0;
  {  // A, from register group 2 h + q of block b in wave 2 b + h of its tile
    const float* g = gram + gram_at<MB>(mat, 0, splits, ib, jb, lane);
    zero();
    if (mine) {
#pragma unroll 4
      for (int sp = 0; sp < splits; ++sp, g += TILES * kGramTile) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const float4 f = *reinterpret_cast<const float4*>(g + q * 256);
          acc[4 * q] += f.x;
          acc[4 * q + 1] += f.y;
          acc[4 * q + 2] += f.z;
          acc[4 * q + 3] += f.w;
        }
      }
    }
    if constexpr (STAGED) {  // X^T on its way into LDS, 1 KB a copy
      const int x0 = me.index * xbw;
      const __amdgpu_buffer_rsrc_t rsrc = __builtin_amdgcn_make_buffer_rsrc(
          (void*)(p.a + mat * p.sa + static_cast<int64_t>(x0) * (KS * 1024)), 0, nb * KS * 2048,
          0x00020000);
      const unsigned lds_x = (unsigned)(uintptr_t)(lds_u8*)xs;
      for (int c = wave; c < nb * KS * 2; c += 16)
        dma16(rsrc, lane * 16, c * 1024, lds_x + c * 1024);
    }
    store(ba, kScaleA / (kScaleX * kScaleX));
    __syncthreads();
  }
  // P = f(A, A^2); with two steps then U = A P and A_2 = U P, each over its
  // first factor, P_2 over A_2, and Q = P_2 P over P. One copy of the code:
  // it runs once a launch, so its size is time (fetching instructions).
#pragma unroll 1
  for (int ph = 0; ph < (steps == 2 ? 5 : 1); ++ph) {
    const bool poly = ph == 0 || ph == 3;
    product(ba, poly ? ba : bp);
    if (poly) polynomial(ba);
    __syncthreads();
    store(ph == 0 || ph == 4 ? bp : ba, poly ? 1.f : 1.f / kScaleP);
    __syncthreads();
  }

  if constexpr (STAGED) {
    __builtin_amdgcn_s_waitcnt(kVm0Lgkm0);  // this wave's copies; after the barrier all
    __syncthreads();
  }
  const int qb = wave % MP, per = STAGED ? xbw : XB;
  int xb = me.index * per + wave / MP;
  const bool busy = qb < MB && wave / MP < per && xb < rk;
  if (MODE != kGram && !busy) return;
  auto times_q = [&]() {  // acc <- the block of X^T times Q
    zero();
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      __builtin_amdgcn_sched_barrier(0);  // not all of Q's fragments at once
      const f16x8 qh = frag(bp, qb, ks, 0), ql = frag(bp, qb, ks, 1);
      const f16x8 xh = STAGED ? frag(xs, wave / MP, ks, 0) : x[ks][0];
      const f16x8 xl = STAGED ? frag(xs, wave / MP, ks, 1) : x[ks][1];
      if constexpr (SWAP)
        mma(qh, ql, xh, xl);
      else
        mma(xh, xl, qh, ql);
    }
  };
  if constexpr (MODE != kGram) {
#pragma unroll 1
    for (; xb < rk; xb += STAGED ? rk : me.groups * XB) {
      if constexpr (!STAGED) load_x(xb);
      times_q();
      float v[4][4];
#pragma unroll
      for (int r = 0; r < 16; ++r) v[r / 4][r % 4] = acc[r];
      store_block<EPI, 4>(p, o, mat, SWAP ? MB : rk, SWAP ? rk : MB, SWAP ? qb : xb,
                          SWAP ? xb : qb, 0, v, lane);
    }
  } else {
    if (busy) times_q();
    __syncthreads();  // xs has been read: now the blocks of X, depth 32 xbw
    if (busy) {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        float v[4];
#pragma unroll
        for (int s = 0; s < 4; ++s) v[s] = acc[4 * q + s] * p.alpha;
        Parts w = split4(v);
        store_parts(xs + (qb * 2 * xbw + 2 * (wave / MP) + (q >> 1)) * 1024, l32 + 32 * (q & 1),
                    4 * half, w);
        w.hi = transpose4(w.hi, lane & 3);
        w.lo = transpose4(w.lo, lane & 3);
        const int j0 = 4 * (l32 >> 2), row = 8 * q + 4 * half + (lane & 3);
        store_parts(p.out_n + mat * p.so +
                        (static_cast<int64_t>(xb) * KS + 2 * qb + (j0 >> 4)) * 1024,
                    row + 32 * ((j0 >> 3) & 1), j0 & 7, w);
      }
    }
    __syncthreads();
    if (mine)
      gram_part<MB>(xs, 2 * xbw, 2 * nb, ib, jb, lane,
                    next_gram + gram_at<MB>(mat, me.index, me.groups, ib, jb, lane));
  }
}

int ceil32(int v) { return (v + 31) / 32; }

// Workspace, in values (16 bits) per matrix: X and two X^T (or the other way
// round for tall matrices); five m x m operands, or, for short sides up to
// 128, the Gram product's parts; then the norm's partials.
struct Space {
  int64_t x, mm;  // values of one X operand, of one m x m operand
  int tiles, splits;  // short sides up to 128: Gram tiles, parts along the depth
  int gram_xbw;   // blocks of X^T a workgroup that gives the Gram parts too (no X then), or 0
  int64_t gram;   // floats of the Gram parts; with gram_xbw there are two such
  int64_t part;   // partial sums per matrix
  size_t bytes;
};
int norm_parts(int n, int64_t values) {
  // Few values: short chunks, whose time is that of a few loads.
  const int64_t chunk = n * values > (int64_t(1) << 23) ? 8192 : 2048;
  return static_cast<int>(std::min<int64_t>(1024, (values + chunk - 1) / chunk));
}
Space space(int n, int rows, int cols) {
  Space s{};
  const int64_t m = ceil32(std::min(rows, cols)), k = ceil32(std::max(rows, cols));
  s.x = m * 2 * k * 1024;
  if (m <= 4) {
    s.tiles = m > 2 ? 3 : 1;
    const int mb = static_cast<int>(m), xbw = steps_staged(mb);
    const int64_t own = (k + xbw - 1) / xbw;
    if (own <= gram_parts(mb) && (own == 1 || own * n <= 256)) {
      s.gram_xbw = xbw;
      s.splits = static_cast<int>(own);
    } else {
      // A workgroup a CU, at least 16 slices each (two a wave).
      const int64_t most = std::min<int64_t>(16, std::max<int64_t>(1, 2 * k / 16));
      s.splits = static_cast<int>(std::max<int64_t>(
          1, std::min<int64_t>(most, 256 / (static_cast<int64_t>(std::max(n, 1)) * s.tiles))));
    }
    s.gram = static_cast<int64_t>(s.tiles) * s.splits * kGramTile;
  } else {
    s.mm = m * 2 * m * 1024;
  }
  s.part = norm_parts(n, static_cast<int64_t>(rows) * cols);
  s.bytes = static_cast<size_t>(n) * (((s.gram_xbw ? 2 : 3) * s.x + 5 * s.mm) * 2 +
                                      (s.gram_xbw ? 2 : 1) * s.gram * 4 + s.part * 8);
  return s;
}

// Most steps of the first segment and of the later ones. Relative Frobenius
// error of fp32 results against 64 bits (gradients of 1.5 m tokens; plain
// torch fp32 / single steps / 2 + 2 + 1 / 3 + 2, in 1e-6):
//   8 x 128 x 512    1.7 / 0.9 / 2.0 /  -      4 x 512 x 512     2.1 / 0.9 /  -  /  -
//   8 x 128 x 128    1.3 / 1.0 / 2.8 /  -      4 x 1024 x 1024   2.7 / 2.3 / 3.4 / 7.7
//   2 x 1024 x 4096  3.5 / 2.6 / 1.9 / 5.3     1 x 2048 x 2048   3.5 / 2.9 / 3.4 / 9.4
// A bf16 result rounds by 1.7e-3, so it takes the fewest operations (pairs up
// to m = 128, where a launch holds two steps). An fp32 result keeps plain
// fp32's accuracy: single steps, and pairs from m = 1024 on. In a Muon step
// with fp32 weights the update is a small part of the weight, and with it the
// error: pairs.
struct Segments {
  int first, later;
};
Segments segment_rule(bool bf16_out, bool muon, int m) {
  if (bf16_out) return {m <= 128 ? 2 : 3, 2};
  return muon || m >= 1024 ? Segments{2, 2} : Segments{1, 1};
}

// Groups of four columns are aligned to their size.
int aligned4(const moe_matrices& m) {
  const uintptr_t size = m.dtype == MOE_BF16 ? 8 : 16;
  return reinterpret_cast<uintptr_t>(m.data) % size == 0 && m.ld % 4 == 0 && m.stride % 4 == 0;
}

template <int EPI>
int64_t tile_count(int B, int n, int ra, int rb) {
  const int64_t ta = (ra + B - 1) / B, tb = (rb + B - 1) / B;
  return n * (EPI == kSym ? ta * (ta + 1) / 2 : ta * tb);
}

// Tile shapes: 64 x 64 with the depth split over the waves, 128 x 128 (two
// workgroups a CU; eight waves each: 16 x 500 x 1500 395 us, with four 405),
// 256 x 256 (one). Measured, whole calls (small / 128 / 256): 2 x 1024^2 (72
// tiles of 128) 384 / 455 / - us; 2048^2 (136) 1052 / 913 / -; 4096 x 14336
// (528) 9998 / 8003 / 7640; 32 x 1024^2 (1152) - / 2552 / 2660; 256 x 64 x 256
// (256, a quarter of each used) 134 / 157 / -. So: small tiles up to half a
// 128-tile a CU and where 128-tiles would compute twice their area; of the others
// whichever take less by their rounds, one of 256-tiles counting as 1.9 of
// 128-tiles at depths up to 1024, as 1.7 beyond (4096 x 14336, X <- Q X: 4 rounds
// 1.21 ms, 7 rounds 1.28). Symmetric products of 513 to 640 128-tiles, two rounds
// against one of 256-tiles, whole calls (128 / 256): 16 x 1024^2 1363 / 1331 us,
// 28 x 768^2 1150 / 1098, 58 x 512^2 917 / 850, 175 x 256^2 590 / 510, 40 x 640^2
// 1048 / 1050, 19 x 896^2 1229 / 1253, 29 x 700^2 1031 / 1061.
template <int EPI>
hipError_t launch_product(Product p0, Product* p1, const Out& o, int n, int ra, int rb, int KS,
                          int& flip, hipStream_t s) {
  auto grid = [&](int B) {
    const int64_t t = (tile_count<EPI>(B, n, ra, rb) + kXcds - 1) / kXcds * kXcds;
    return dim3(static_cast<unsigned>(t), p1 ? 2 : 1);
  };
  p0.flip = flip;
  flip ^= 1;
  if (p1) p1->flip = p0.flip;
  const Product& q = p1 ? *p1 : p0;
  const int64_t t64 = tile_count<EPI>(2, n, ra, rb), t128 = tile_count<EPI>(4, n, ra, rb);
  const int64_t t256 = tile_count<EPI>(8, n, ra, rb);
  if (t128 <= kSmallTiles || t64 <= 2 * t128) {
    if (t64 * (p1 ? 2 : 1) <= 256)
      orth_product_small_kernel<EPI, 8><<<grid(2), 512, 0, s>>>(p0, q, o, n, ra, rb, KS);
    else
      orth_product_small_kernel<EPI, 4><<<grid(2), 256, 0, s>>>(p0, q, o, n, ra, rb, KS);
  } else if ((KS <= 64 ? 19 : 17) * ((t256 + 255) / 256) > 10 * ((t128 + 511) / 512))
    orth_product_kernel<EPI, 2, 1, 2, 4><<<grid(4), 512, 0, s>>>(p0, q, o, n, ra, rb, KS);
  else
    orth_product_kernel<EPI, 2, 4, 4, 2><<<grid(8), 512, 0, s>>>(p0, q, o, n, ra, rb, KS);
  return hipGetLastError();
}

// f with the number of row blocks (1 to 4) as a type.
template <typename F>
void with_blocks(int rm, F f) {
  switch (rm) {
    case 1: f(std::integral_constant<int, 1>{}); break;
    case 2: f(std::integral_constant<int, 2>{}); break;
    case 3: f(std::integral_constant<int, 3>{}); break;
    default: f(std::integral_constant<int, 4>{}); break;
  }
}

// p.a: X^T; gram: `splits` parts. next_gram (NULL: not wanted): the next
// segment's parts, of gram_xbw blocks each.
template <int EPI, bool SWAP>
hipError_t launch_steps(const Product& p, const Out& o, int steps, int n, int rm, int rk,
                        const float* gram, int splits, int gram_xbw, float* next_gram,
                        hipStream_t s) {
  with_blocks(rm, [&](auto mb) {
    constexpr int MB = decltype(mb)::value;
    if constexpr (EPI == kOperand) {
      if (next_gram != nullptr) {
        const int groups = (rk + gram_xbw - 1) / gram_xbw;
        orth_steps_kernel<MB, EPI, SWAP, kGram>
            <<<group_grid(n, groups), 1024, 0, s>>>(p, o, steps, rk, gram_xbw, n,
                                                    runs_of(groups), gram, splits, next_gram);
        return;
      }
    }
    // As few blocks of X^T a workgroup as leave a CU for each.
    int xbw = 1;
    auto groups_of = [&](int per) { return (rk + per - 1) / per; };
    auto fits = [&](int per) { return static_cast<int64_t>(groups_of(per)) * n <= 256; };
    while (xbw < steps_staged(MB) && !fits(xbw)) xbw *= 2;
    if (fits(xbw)) {
      orth_steps_kernel<MB, EPI, SWAP, kStaged>
          <<<group_grid(n, groups_of(xbw)), 1024, 0, s>>>(
              p, o, steps, rk, xbw, n, runs_of(groups_of(xbw)), gram, splits, nullptr);
    } else {
      const int groups = std::min(groups_of(steps_xb(MB)), std::max(1, 256 / n));
      orth_steps_kernel<MB, EPI, SWAP, kLoop>
          <<<dim3(groups, n), 1024, 0, s>>>(p, o, steps, rk, 0, n, 0, gram, splits, nullptr);
    }
  });
  return hipGetLastError();
}

}  // namespace

size_t orth_ws_bytes(int n, int rows, int cols) { return space(n, rows, cols).bytes; }

int64_t orth_tiles(int n, int rows, int cols) {
  const int64_t m = (std::min(rows, cols) + 63) / 64, k = (std::max(rows, cols) + 63) / 64;
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
  uint16_t *X = sp.gram_xbw ? nullptr : take(sp.x), *XT = take(sp.x), *XT2 = take(sp.x);
  uint16_t *A = take(sp.mm), *U = take(sp.mm), *P = take(sp.mm), *Q = take(sp.mm),
           *Q2 = take(sp.mm);
  float* gram = reinterpret_cast<float*>(take(2 * sp.gram));
  float* next_gram = sp.gram_xbw ? reinterpret_cast<float*>(take(2 * sp.gram)) : nullptr;
  double* part = reinterpret_cast<double*>(base);

  const Mats gm{g.data, g.ld, g.stride, g.dtype == MOE_BF16};
  const Mats wm{w.data, w.ld, w.stride, w.dtype == MOE_BF16};
  const Mats mm = mom ? Mats{mom->data, mom->ld, mom->stride, 0} : Mats{nullptr, 0, 0, 0};
  const int nparts = static_cast<int>(sp.part);
  const int64_t values = static_cast<int64_t>(rows) * cols;
  const int64_t chunk = ((values + nparts - 1) / nparts + 3) / 4 * 4;
  const bool vec4 = cols % 4 == 0 && aligned4(g) && (mom == nullptr || aligned4(*mom));
  const int tr = (rows + 63) / 64, tc = (cols + 63) / 64;
  auto run = [&](auto norm, auto split) {
    norm<<<dim3(nparts, n), 256, 0, s>>>(gm, mm, d.mu, d.nesterov, rows, cols, chunk, part);
    split<<<dim3(tr * tc, n), 256, 0, s>>>(gm, mm, d.mu, d.nesterov, rows, cols, d.eps, part,
                                           nparts, tall ? XT : X, tall ? X : XT, sp.x, tc);
  };
  auto run_gram = [&](auto vec, auto mb) {
    constexpr int V = decltype(vec)::value, MB = decltype(mb)::value;
    orth_norm_kernel<V>
        <<<dim3(nparts, n), 256, 0, s>>>(gm, mm, d.mu, d.nesterov, rows, cols, chunk, part);
    auto split = tall ? orth_split_gram_kernel<V, MB, true> : orth_split_gram_kernel<V, MB, false>;
    split<<<group_grid(n, sp.splits), 1024, 0, s>>>(gm, mm, d.mu, d.nesterov, rows, cols, d.eps,
                                                    part, nparts, XT, sp.x, rk, n, runs_of(sp.splits),
                                                    gram);
  };
  if (sp.gram_xbw) {
    with_blocks(rm, [&](auto mb) {
      if (vec4)
        run_gram(std::integral_constant<int, 4>{}, mb);
      else
        run_gram(std::integral_constant<int, 1>{}, mb);
    });
  } else if (vec4) {
    run(orth_norm_kernel<4>, orth_split_kernel<4>);
  } else {
    run(orth_norm_kernel<1>, orth_split_kernel<1>);
  }
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;

  const Out none{};
  const Out out{wm, rows, cols, mom ? 1.f - d.lr * d.weight_decay : 0.f,
                mom ? -d.lr * d.scale : 1.f, mom != nullptr, aligned4(w)};
  // Every other product takes its tiles in the opposite order: what the last
  // one wrote at its end is still in the 256 MB cache.
  int flip = 0;
  // Symmetric m x m product: out = so (a b / (sa sb) + beta aux + gamma I).
  auto sym_args = [&](const uint16_t* a, const uint16_t* b, float sa, float sb, uint16_t* out,
                      float so, float alpha) {
    return Product{a, b, sp.mm, sp.mm, out, out, sp.mm, nullptr, alpha * so / (sa * sb), 0.f, 0.f};
  };
  auto sym = [&](const Product& p) {
    return launch_product<kSym>(p, nullptr, none, n, rm, rm, 2 * rm, flip, s);
  };
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
    if (rm <= 4) {
      if (next_gram == nullptr)
        orth_gram_kernel<<<dim3(sp.tiles * sp.splits, n), 512, 0, s>>>(X, sp.x, rm, 2 * rk,
                                                                       sp.tiles, sp.splits, gram);
      Product x{XT, nullptr, sp.x, 0, X, XT2, sp.x, nullptr, 1.f / kScaleP, 0.f, 0.f};
      if (left > 0) {
        e = launch_steps<kOperand, false>(x, none, L, n, rm, rk, gram, sp.splits, sp.gram_xbw,
                                          next_gram, s);
        std::swap(XT, XT2);
        if (next_gram != nullptr) std::swap(gram, next_gram);
      } else {
        x.alpha = 1.f / (kScaleP * kScaleX);
        e = tall ? launch_steps<kOut, false>(x, out, L, n, rm, rk, gram, sp.splits, 0, nullptr, s)
                 : launch_steps<kOut, true>(x, out, L, n, rm, rk, gram, sp.splits, 0, nullptr, s);
      }
      if (e != hipSuccess) return e;
      continue;
    }
    Product gram_p{X, X, sp.x, sp.x, A, A, sp.mm, nullptr, kScaleA / (kScaleX * kScaleX), 0.f, 0.f};
    e = launch_product<kSym>(gram_p, nullptr, none, n, rm, rm, 2 * rk, flip, s);
    if (e != hipSuccess) return e;
    uint16_t *q = Q, *q2 = Q2;
    if ((e = poly(q)) != hipSuccess) return e;
    const uint16_t* pl = q;  // the last P
    for (int i = 1; i < L; ++i) {
      // U = A P (with the product of the P so far, from the second step on),
      // A <- U P, the next P.
      Product u = sym_args(A, pl, kScaleA, kScaleP, U, kScaleA, 1.f);
      Product qq = sym_args(pl, q, kScaleP, kScaleP, q2, kScaleP, 1.f);
      // Both in one launch while that is one round of workgroups (4096 x 4096,
      // 136 + 136 tiles of 256: 540 us together, 488 one after the other).
      const bool pair = tile_count<kSym>(8, n, rm, rm) <= 128;
      e = launch_product<kSym>(u, i > 1 && pair ? &qq : nullptr, none, n, rm, rm, 2 * rm, flip, s);
      if (e == hipSuccess && i > 1 && !pair) e = sym(qq);
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
    // X <- Q X. An operand for the next segment takes either orientation; the
    // caller's matrix has its rows at i and its columns at j.
    Product x{XT, q, sp.x, sp.mm, X, XT2, sp.x, nullptr, 1.f / kScaleP, 0.f, 0.f};
    if (left > 0) {
      e = launch_product<kOperand>(x, nullptr, none, n, rk, rm, 2 * rm, flip, s);
      std::swap(XT, XT2);
    } else {
      x.alpha = 1.f / (kScaleP * kScaleX);
      if (!tall) {
        std::swap(x.a, x.b);
        std::swap(x.sa, x.sb);
      }
      const int ra = tall ? rk : rm, rb = tall ? rm : rk;
      e = launch_product<kOut>(x, nullptr, out, n, ra, rb, 2 * rm, flip, s);
    }
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace moe

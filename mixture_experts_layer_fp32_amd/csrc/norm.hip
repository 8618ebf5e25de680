// Layer norm forward and backward (include/moe_norm.h).
//
//   h = (x - mean) rstd,  y = h gamma + beta
//   dx = rstd (g - mean(g) - h mean(g h)) + dres,  g = dy gamma
//   dgamma = sum_rows dy h,  dbeta = sum_rows dy
//
// Both passes are bound by memory: a few operations per value. A row belongs
// to a group of G threads (one wave, or one workgroup of G threads), 16 values
// a thread, that hold it in registers, so x (and dy) are read once; gamma and
// beta, and in the backward the column sums, stay in registers over all rows
// of the group. Measured (a copy of 1 GiB moves 5.1 TB/s): forward 8192 x 4096
// bf16 25.4 us, 5.3 TB/s (part of x is still cached); backward with the residual
// 16384 x 2048 bf16 62 us, 4.3 TB/s, 4096 x 7168 fp32 91 us, 5.1 TB/s. What it
// took: the row's two sums across the lanes in registers and one barrier a row
// (44 -> 34 us forward), non-temporal stores (34 -> 32; backward 64 -> 57), the
// hardware's bf16 conversion (32 -> 27), the waves' means joined without a
// division each (4096 x 7168 fp32 43 -> 38). Tried and slower: two rows in flight
// ahead, non-temporal loads of bf16 rows, fewer or one row per workgroup. Rows
// above 8192 values (16 waves, nothing read ahead) and above 16384 (x from the
// caches a second and third time) are further off: 3000 x 10000 bf16 48 us, 2.5
// TB/s, 2000 x 20000 bf16 50 us, 3.2, 1000 x 40000 fp32 87 us, 3.7; their
// backward with the residual 104, 98 and 178 us.
#include <algorithm>

#include "moe_internal.h"

namespace moe {
namespace {

// Vectors of 16 bytes that need only their element's alignment: rows of odd
// widths start anywhere, and the hardware loads such vectors whole.
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef u32x4 u32x4_a2 __attribute__((aligned(2)));
typedef u32x4 u32x4_a4 __attribute__((aligned(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

template <typename T>
struct Vec;
template <>
struct Vec<float> {
  static constexpr int N = 4;
  typedef u32x4_a4 raw_a;
  static __device__ __forceinline__ void unpack(const u32x4& r, float (&f)[N]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = __uint_as_float(r[i]);
  }
  static __device__ __forceinline__ u32x4 pack(const float (&f)[N]) {
    return u32x4{__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                 __float_as_uint(f[3])};
  }
  static __device__ __forceinline__ void store1(float* p, float v) { *p = v; }
};
template <>
struct Vec<uint16_t> {  // bf16
  static constexpr int N = 8;
  typedef u32x4_a2 raw_a;
  static __device__ __forceinline__ void unpack(const u32x4& r, float (&f)[N]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(r[i] << 16);
      f[2 * i + 1] = __uint_as_float(r[i] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ u32x4 pack(const float (&f)[N]) {
    // v_cvt_pk_bf16_f32: two values an instruction, to nearest even, NaN kept.
    u32x4 r;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      r[i] = __builtin_bit_cast(
          uint32_t, __builtin_convertvector(f32x2{f[2 * i], f[2 * i + 1]}, bf16x2));
    return r;
  }
  static __device__ __forceinline__ void store1(uint16_t* p, float v) { *p = f32_to_bf16(v); }
};

// Values [v N, v N + N) of a row of D values, those past D as zeros.
template <typename T>
__device__ __forceinline__ u32x4 load_vec(const T* row, int v, int nfull, int D) {
  constexpr int N = Vec<T>::N;
  u32x4 r = {0, 0, 0, 0};
  if (v < nfull) {
    r = *reinterpret_cast<const typename Vec<T>::raw_a*>(row + static_cast<int64_t>(v) * N);
  } else if (v == nfull) {
    for (int e = 0; e < D - nfull * N; ++e) {
      if constexpr (sizeof(T) == 4)
        r[e] = __float_as_uint(row[nfull * N + e]);
      else
        r[e / 2] |= static_cast<uint32_t>(row[nfull * N + e]) << (16 * (e & 1));
    }
  }
  return r;
}
template <typename T>
__device__ __forceinline__ void store_vec(T* row, int v, int nfull, int D,
                                          const float (&f)[Vec<T>::N]) {
  constexpr int N = Vec<T>::N;
  if (v < nfull) {
    __builtin_nontemporal_store(Vec<T>::pack(f), reinterpret_cast<typename Vec<T>::raw_a*>(row + static_cast<int64_t>(v) * N));
  } else if (v == nfull) {
#pragma unroll
    for (int e = 0; e < N; ++e)
      if (e < D - nfull * N) Vec<T>::store1(row + nfull * N + e, f[e]);
  }
}
// N fp32 parameters of vector v, `pad` without any (zeros past D).
template <int N>
__device__ __forceinline__ void load_param(const float* p, int v, int D, float pad,
                                           float (&f)[N]) {
#pragma unroll
  for (int i = 0; i < N / 4; ++i) {
    float q[4] = {pad, pad, pad, pad};
    if (p != nullptr) Vec<float>::unpack(load_vec(p, v * (N / 4) + i, D / 4, D), q);
#pragma unroll
    for (int e = 0; e < 4; ++e) f[4 * i + e] = q[e];
  }
}

// Sum over the wave, in every lane: two quad permutes and two mirrors leave
// each row of 16 lanes with its sum, four lane reads add the rows. (Shuffles
// through LDS cost about 100 cycles each of a chain of six.)
template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
  return __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), CTRL, 0xF, 0xF, false));
}
template <int CTRL>
__device__ __forceinline__ double dpp(double v) {
  return __hiloint2double(__builtin_amdgcn_mov_dpp(__double2hiint(v), CTRL, 0xF, 0xF, false),
                          __builtin_amdgcn_mov_dpp(__double2loint(v), CTRL, 0xF, 0xF, false));
}
__device__ __forceinline__ float lane_value(float v, int l) {
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), l));
}
__device__ __forceinline__ double lane_value(double v, int l) {
  return __hiloint2double(__builtin_amdgcn_readlane(__double2hiint(v), l),
                          __builtin_amdgcn_readlane(__double2loint(v), l));
}
template <typename S>
__device__ __forceinline__ S wave_sum(S v) {
  v += dpp<0xB1>(v);   // quad_perm 1 0 3 2
  v += dpp<0x4E>(v);   // quad_perm 2 3 0 1
  v += dpp<0x141>(v);  // row_half_mirror
  v += dpp<0x140>(v);  // row_mirror
  return (lane_value(v, 0) + lane_value(v, 16)) + (lane_value(v, 32) + lane_value(v, 48));
}

// A buffer for what a group's waves tell each other. Calls alternate `slot`,
// so one barrier a call is enough: a wave that writes a slot again has passed
// the barrier of the call in between, and with it every read of the slot's
// last use.
template <int G>
struct Exchange {
  double s[2][G / 64];
  float f[2][3][G / 64];
};

// Sum of a vector's values: of four in fp32, of the fours in fp64 (eight bf16
// values of 2^125 leave fp32's range; of either type values below 2^126 do not).
template <int N>
__device__ __forceinline__ double vec_sum(const float (&f)[N]) {
  double s = (f[0] + f[2]) + (f[1] + f[3]);
#pragma unroll
  for (int e = 4; e < N; e += 4) s += (f[e] + f[e + 2]) + (f[e + 1] + f[e + 3]);
  return s;
}

// mean and 1 / sqrt(variance + eps) of the group's values f (places that hold
// none are zeros; cnt of the thread's, n_wave of the wave's are values). Each
// wave takes its own mean and centred sum of squares; the waves' are joined
// by M2 = sum_w (M2_w + n_w (mean_w - mean)^2). The sums of values are added
// across threads in fp64, so that a mean near zero keeps its digits.
template <int G, int NV, int N>
__device__ __forceinline__ void row_stats(const float (&f)[NV][N], const int (&cnt)[NV],
                                          float n_wave, int D, float eps, Exchange<G>& ex,
                                          int& slot, float& mean, float& rstd) {
  double s = vec_sum<N>(f[0]);
#pragma unroll
  for (int i = 1; i < NV; ++i) s += vec_sum<N>(f[i]);
  s = wave_sum(s);
  const float mw = n_wave > 0.f ? static_cast<float>(s / n_wave) : 0.f;
  float m2 = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int e = 0; e < N; ++e)
      if (e < cnt[i]) m2 = fmaf(f[i][e] - mw, f[i][e] - mw, m2);
  m2 = wave_sum(m2);
  if constexpr (G > 64) {
    constexpr int W = G / 64;
    if ((threadIdx.x & 63) == 0) {
      ex.s[slot][threadIdx.x >> 6] = s;
      ex.f[slot][0][threadIdx.x >> 6] = m2;
      ex.f[slot][1][threadIdx.x >> 6] = n_wave;
      ex.f[slot][2][threadIdx.x >> 6] = mw;
    }
    __syncthreads();
    s = 0.0;
#pragma unroll
    for (int w = 0; w < W; ++w) s += ex.s[slot][w];
    mean = static_cast<float>(s / D);
    m2 = 0.f;
#pragma unroll
    for (int w = 0; w < W; ++w) {
      const float nw = ex.f[slot][1][w];
      const float d = nw > 0.f ? ex.f[slot][2][w] - mean : 0.f;
      m2 += fmaf(nw * d, d, ex.f[slot][0][w]);
    }
    slot ^= 1;
  } else {
    mean = mw;
  }
  rstd = 1.f / sqrtf(m2 / static_cast<float>(D) + eps);
}

// Sums of two values over the group's G threads, in every thread.
template <int G>
__device__ __forceinline__ void group_sum(float (&s)[2], Exchange<G>& ex, int& slot) {
  s[0] = wave_sum(s[0]);
  s[1] = wave_sum(s[1]);
  if constexpr (G > 64) {
    constexpr int W = G / 64;
    if ((threadIdx.x & 63) == 0) {
      ex.f[slot][0][threadIdx.x >> 6] = s[0];
      ex.f[slot][1][threadIdx.x >> 6] = s[1];
    }
    __syncthreads();
    s[0] = s[1] = 0.f;
#pragma unroll
    for (int w = 0; w < W; ++w) {
      s[0] += ex.f[slot][0][w];
      s[1] += ex.f[slot][1][w];
    }
    slot ^= 1;
  }
}

// The same of one value in fp64 (G > 64).
template <int G>
__device__ __forceinline__ double group_sum(double s, Exchange<G>& ex, int& slot) {
  s = wave_sum(s);
  if ((threadIdx.x & 63) == 0) ex.s[slot][threadIdx.x >> 6] = s;
  __syncthreads();
  s = 0.0;
#pragma unroll
  for (int w = 0; w < G / 64; ++w) s += ex.s[slot][w];
  slot ^= 1;
  return s;
}

constexpr int wg_of(int G) { return G == 64 ? 256 : G; }

// ---- forward: the row in registers -----------------------------------------
template <typename T, int G, int NV>
__global__ __launch_bounds__(wg_of(G)) void norm_fwd_kernel(
    const T* __restrict__ x, const float* __restrict__ gamma, const float* __restrict__ beta,
    float eps, T* __restrict__ y, float* __restrict__ mean_out, float* __restrict__ rstd_out,
    int64_t rows, int D) {
  constexpr int N = Vec<T>::N, WG = wg_of(G), R = WG / G;
  __shared__ Exchange<G> ex;
  int slot = 0;
  const int t = threadIdx.x % G, nfull = D / N;
  const int64_t step = static_cast<int64_t>(gridDim.x) * R;
  int64_t r = static_cast<int64_t>(blockIdx.x) * R + threadIdx.x / G;
  // The next row is in flight while one is computed (G = 1024: the registers
  // that 16 waves leave a thread do not hold it).
  constexpr bool kAhead = G < 1024;
  u32x4 next[NV];
  auto fetch = [&](int64_t q) {
#pragma unroll
    for (int i = 0; i < NV; ++i) next[i] = load_vec(x + q * D, t + i * G, nfull, D);
  };
  if (kAhead && r < rows) fetch(r);
  float gm[NV][N], bt[NV][N], n_wave = 0.f;
  int cnt[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    load_param<N>(gamma, t + i * G, D, 1.f, gm[i]);
    load_param<N>(beta, t + i * G, D, 0.f, bt[i]);
    cnt[i] = min(max(D - (t + i * G) * N, 0), N);
    n_wave += static_cast<float>(cnt[i]);
  }
  n_wave = wave_sum(n_wave);
  for (; r < rows; r += step) {
    float f[NV][N];
    if (!kAhead) fetch(r);
#pragma unroll
    for (int i = 0; i < NV; ++i) Vec<T>::unpack(next[i], f[i]);
    if (kAhead && r + step < rows) fetch(r + step);
    float mean, rstd;
    row_stats<G, NV, N>(f, cnt, n_wave, D, eps, ex, slot, mean, rstd);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
#pragma unroll
      for (int e = 0; e < N; ++e) f[i][e] = fmaf((f[i][e] - mean) * rstd, gm[i][e], bt[i][e]);
      store_vec(y + r * D, t + i * G, nfull, D, f[i]);
    }
    if (t == 0) {
      if (mean_out != nullptr) mean_out[r] = mean;
      if (rstd_out != nullptr) rstd_out[r] = rstd;
    }
  }
}

// ---- forward: rows wider than the registers hold ---------------------------
// One workgroup a row; the second and third reads of x come from the caches. A
// thread adds up to 256 values: from vector to vector in fp64, as across threads
// (in fp32 the y of a constant row of 262144 values 1000.1 was 0.6 instead of 0;
// the pass is bound by memory either way).
template <typename T>
__global__ __launch_bounds__(1024) void norm_fwd_wide_kernel(
    const T* __restrict__ x, const float* __restrict__ gamma, const float* __restrict__ beta,
    float eps, T* __restrict__ y, float* __restrict__ mean_out, float* __restrict__ rstd_out,
    int64_t rows, int D) {
  constexpr int N = Vec<T>::N, G = 1024;
  __shared__ Exchange<G> ex;
  int slot = 0;
  const int t = threadIdx.x, nfull = D / N, nvec = (D + N - 1) / N;
  const float fd = static_cast<float>(D);
  for (int64_t r = blockIdx.x; r < rows; r += gridDim.x) {
    const T* xr = x + r * D;
    float f[N], s[2] = {0.f, 0.f};
    double sum = 0.0;
    for (int v = t; v < nvec; v += G) {
      Vec<T>::unpack(load_vec(xr, v, nfull, D), f);
      sum += vec_sum<N>(f);
    }
    const float mean = static_cast<float>(group_sum<G>(sum, ex, slot) / D);
    for (int v = t; v < nvec; v += G) {
      Vec<T>::unpack(load_vec(xr, v, nfull, D), f);
#pragma unroll
      for (int e = 0; e < N; ++e)
        if (v * N + e < D) s[0] = fmaf(f[e] - mean, f[e] - mean, s[0]);
    }
    group_sum<G>(s, ex, slot);
    const float rstd = 1.f / sqrtf(s[0] / fd + eps);
    for (int v = t; v < nvec; v += G) {
      Vec<T>::unpack(load_vec(xr, v, nfull, D), f);
      float gm[N], bt[N];
      load_param<N>(gamma, v, D, 1.f, gm);
      load_param<N>(beta, v, D, 0.f, bt);
#pragma unroll
      for (int e = 0; e < N; ++e) f[e] = fmaf((f[e] - mean) * rstd, gm[e], bt[e]);
      store_vec(y + r * D, v, nfull, D, f);
    }
    if (t == 0) {
      if (mean_out != nullptr) mean_out[r] = mean;
      if (rstd_out != nullptr) rstd_out[r] = rstd;
    }
  }
}

// ---- backward: the row in registers ----------------------------------------
// PARAMS: this workgroup's sums of dy h and dy over its rows go to row
// blockIdx.x of part_g and part_b [gridDim.x][D] (NULL: not wanted); a single
// workgroup writes dgamma and dbeta themselves.
template <typename T, int G, int NV, bool PARAMS>
__global__ __launch_bounds__(wg_of(G)) void norm_bwd_kernel(
    const T* __restrict__ x, const T* __restrict__ dy, const float* __restrict__ gamma,
    const float* __restrict__ mean_in, const float* __restrict__ rstd_in,
    const T* __restrict__ dres, T* __restrict__ dx, float* __restrict__ part_g,
    float* __restrict__ part_b, int64_t rows, int D) {
  constexpr int N = Vec<T>::N, WG = wg_of(G), R = WG / G;
  // red: with several groups a workgroup, the column sums of the others.
  __shared__ Exchange<G> ex;
  __shared__ float red[R > 1 && PARAMS ? (R - 1) * 64 * NV * N : 1];
  int slot = 0;
  const int t = threadIdx.x % G, grp = threadIdx.x / G, nfull = D / N;
  float gm[NV][N], dg[NV][N], db[NV][N];
  int cnt[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    load_param<N>(gamma, t + i * G, D, 1.f, gm[i]);
    cnt[i] = min(max(D - (t + i * G) * N, 0), N);
#pragma unroll
    for (int e = 0; e < N; ++e) dg[i][e] = db[i][e] = 0.f;
  }
  const float fd = static_cast<float>(D);
  const int64_t step = static_cast<int64_t>(gridDim.x) * R;
  int64_t r = static_cast<int64_t>(blockIdx.x) * R + grp;
  u32x4 nx[NV], nd[NV];
  float nm = 0.f, nr = 0.f;
  auto fetch = [&](int64_t q) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      nx[i] = load_vec(x + q * D, t + i * G, nfull, D);
      nd[i] = load_vec(dy + q * D, t + i * G, nfull, D);
    }
    nm = mean_in[q];
    nr = rstd_in[q];
  };
  constexpr bool kAhead = G < 1024;  // as in the forward
  if (kAhead && r < rows) fetch(r);
  for (; r < rows; r += step) {
    float h[NV][N], d[NV][N], s[2] = {0.f, 0.f};
    if (!kAhead) fetch(r);
    const float mean = nm, rstd = nr;
    u32x4 res[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      Vec<T>::unpack(nx[i], h[i]);
      Vec<T>::unpack(nd[i], d[i]);
      res[i] = dres != nullptr ? load_vec(dres + r * D, t + i * G, nfull, D) : u32x4{0, 0, 0, 0};
    }
    if (kAhead && r + step < rows) fetch(r + step);
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int e = 0; e < N; ++e) {
        // Places past D hold d = 0, and h = 0: -mean rstd may be infinite where
        // (x - mean) rstd is not, in rows of nearly equal values above 1e36.
        // (Up to 3 % at ragged widths; a branch around it, or x = mean there,
        // cost as much or more.)
        h[i][e] = e < cnt[i] ? (h[i][e] - mean) * rstd : 0.f;
        if (PARAMS) {
          dg[i][e] = fmaf(d[i][e], h[i][e], dg[i][e]);
          db[i][e] += d[i][e];
        }
        d[i][e] *= gm[i][e];
        s[0] += d[i][e];
        s[1] = fmaf(d[i][e], h[i][e], s[1]);
      }
    group_sum<G>(s, ex, slot);
    const float c0 = s[0] / fd, c1 = s[1] / fd;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float o[N];
      Vec<T>::unpack(res[i], o);
#pragma unroll
      for (int e = 0; e < N; ++e) o[e] = fmaf(rstd, d[i][e] - c0 - h[i][e] * c1, o[e]);
      store_vec(dx + r * D, t + i * G, nfull, D, o);
    }
  }
  if constexpr (PARAMS) {
    // dgamma then dbeta: the other groups' sums through LDS to group 0.
    auto flush = [&](float(&a)[NV][N], float* o) {
      if (o == nullptr) return;
      o += static_cast<int64_t>(blockIdx.x) * D;
      if constexpr (R > 1) {
        __syncthreads();
        if (grp > 0) {
#pragma unroll
          for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int e = 0; e < N; ++e) red[((grp - 1) * NV * N + i * N + e) * 64 + t] = a[i][e];
        }
        __syncthreads();
        if (grp > 0) return;
#pragma unroll
        for (int q = 0; q < R - 1; ++q)
#pragma unroll
          for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int e = 0; e < N; ++e) a[i][e] += red[(q * NV * N + i * N + e) * 64 + t];
      }
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int e = 0; e < N; ++e) {
          const int c = (t + i * G) * N + e;
          if (c < D) o[c] = a[i][e];
        }
    };
    flush(dg, part_g);
    flush(db, part_b);
  }
}

// ---- backward: wide rows ---------------------------------------------------
template <typename T>
__global__ __launch_bounds__(1024) void norm_bwd_wide_kernel(
    const T* __restrict__ x, const T* __restrict__ dy, const float* __restrict__ gamma,
    const float* __restrict__ mean_in, const float* __restrict__ rstd_in,
    const T* __restrict__ dres, T* __restrict__ dx, int64_t rows, int D) {
  constexpr int N = Vec<T>::N, G = 1024;
  __shared__ Exchange<G> ex;
  int slot = 0;
  const int t = threadIdx.x, nfull = D / N, nvec = (D + N - 1) / N;
  const float fd = static_cast<float>(D);
  for (int64_t r = blockIdx.x; r < rows; r += gridDim.x) {
    const float mean = mean_in[r], rstd = rstd_in[r];
    const bool far = isinf(mean * rstd);
    float h[N], d[N], gm[N], s[2] = {0.f, 0.f};
    for (int v = t; v < nvec; v += G) {
      Vec<T>::unpack(load_vec(x + r * D, v, nfull, D), h);
      Vec<T>::unpack(load_vec(dy + r * D, v, nfull, D), d);
      load_param<N>(gamma, v, D, 1.f, gm);
      if (far && v == nfull) {  // h = 0 past D, as in the registers' kernel
#pragma unroll
        for (int e = 0; e < N; ++e)
          if (v * N + e >= D) h[e] = mean;
      }
#pragma unroll
      for (int e = 0; e < N; ++e) {
        s[0] = fmaf(d[e], gm[e], s[0]);
        s[1] = fmaf(d[e] * gm[e], (h[e] - mean) * rstd, s[1]);
      }
    }
    group_sum<G>(s, ex, slot);
    const float c0 = s[0] / fd, c1 = s[1] / fd;
    for (int v = t; v < nvec; v += G) {
      float o[N];
      Vec<T>::unpack(load_vec(x + r * D, v, nfull, D), h);
      Vec<T>::unpack(load_vec(dy + r * D, v, nfull, D), d);
      load_param<N>(gamma, v, D, 1.f, gm);
      const u32x4 res = dres != nullptr ? load_vec(dres + r * D, v, nfull, D) : u32x4{0, 0, 0, 0};
      Vec<T>::unpack(res, o);
#pragma unroll
      for (int e = 0; e < N; ++e)
        o[e] = fmaf(rstd, d[e] * gm[e] - c0 - (h[e] - mean) * rstd * c1, o[e]);
      store_vec(dx + r * D, v, nfull, D, o);
    }
  }
}
// Column sums of rows [blockIdx.y chunk, ...): one thread a column.
template <typename T>
__global__ __launch_bounds__(256) void norm_param_kernel(const T* __restrict__ x,
                                                         const T* __restrict__ dy,
                                                         const float* __restrict__ mean_in,
                                                         const float* __restrict__ rstd_in,
                                                         float* __restrict__ part_g,
                                                         float* __restrict__ part_b, int64_t rows,
                                                         int D, int64_t chunk) {
  const int c = blockIdx.x * 256 + threadIdx.x;
  if (c >= D) return;
  const int64_t r1 = min(rows, (blockIdx.y + 1) * chunk);
  float dg = 0.f, db = 0.f;
  for (int64_t r = blockIdx.y * chunk; r < r1; ++r) {
    const float d = load_act(dy + r * D + c);
    dg = fmaf(d, (load_act(x + r * D + c) - mean_in[r]) * rstd_in[r], dg);
    db += d;
  }
  if (part_g != nullptr) part_g[static_cast<int64_t>(blockIdx.y) * D + c] = dg;
  if (part_b != nullptr) part_b[static_cast<int64_t>(blockIdx.y) * D + c] = db;
}

// dgamma (blockIdx.y 0) and dbeta (1): 32 columns a workgroup, the P partial
// rows shared out over 32 half waves, each adding its own in row order, then
// the half waves in order. P == 0 writes zeros.
constexpr int kFinishCols = 32, kFinishRows = 32;
__global__ __launch_bounds__(kFinishCols * kFinishRows) void norm_finish_kernel(
    const float* __restrict__ part, int P, int D, float* __restrict__ dgamma,
    float* __restrict__ dbeta) {
  __shared__ float red[kFinishRows][kFinishCols];
  float* out = blockIdx.y == 0 ? dgamma : dbeta;
  if (out == nullptr) return;
  const int t = threadIdx.x % kFinishCols, w = threadIdx.x / kFinishCols;
  const int c = blockIdx.x * kFinishCols + t;
  const float* p = part + static_cast<int64_t>(blockIdx.y) * P * D;
  float s = 0.f;
  if (c < D) {
#pragma unroll 8
    for (int q = w; q < P; q += kFinishRows) s += p[static_cast<int64_t>(q) * D + c];
  }
  red[w][t] = s;
  __syncthreads();
  if (w == 0 && c < D) {
#pragma unroll
    for (int q = 1; q < kFinishRows; ++q) s += red[q][t];
    out[c] = s;
  }
}

constexpr int kRegVals = 16;          // values of a row per thread
constexpr int kMaxRegWidth = 16384;   // 1024 threads
constexpr int kCus = 256;

// Threads a row: the fewest of 64, 128, ... 1024 that hold D in kRegVals each.
int group_of(int D) {
  int g = 64;
  while (g * kRegVals < D) g *= 2;
  return g;
}
int64_t groups_per_wg(int g) { return wg_of(g) / g; }

// Workgroups of the backward's row pass, and so partial rows.
int64_t bwd_parts(int64_t rows, int D) {
  if (rows == 0) return 0;
  if (D > kMaxRegWidth) return std::min<int64_t>(rows, 64);
  const int g = group_of(D);
  const int64_t wgs = (rows + groups_per_wg(g) - 1) / groups_per_wg(g);
  return std::min<int64_t>(wgs, 2 * kCus * 256 / wg_of(g));
}

template <typename T, int G>
void fwd_g(const void* x, const float* gamma, const float* beta, float eps, void* y, float* mean,
           float* rstd, int64_t rows, int D, hipStream_t s) {
  constexpr int NV = kRegVals / Vec<T>::N, R = wg_of(G) / G;
  const int64_t wgs = (rows + R - 1) / R;
  const int grid = static_cast<int>(std::min<int64_t>(wgs, 8 * kCus * 256 / wg_of(G)));
  norm_fwd_kernel<T, G, NV><<<grid, wg_of(G), 0, s>>>(
      static_cast<const T*>(x), gamma, beta, eps, static_cast<T*>(y), mean, rstd, rows, D);
}

template <typename T>
hipError_t fwd_t(int64_t rows, int D, const void* x, const float* gamma, const float* beta,
                 float eps, void* y, float* mean, float* rstd, hipStream_t s) {
  if (D > kMaxRegWidth) {
    norm_fwd_wide_kernel<T><<<static_cast<int>(std::min<int64_t>(rows, 2 * kCus)), 1024, 0, s>>>(
        static_cast<const T*>(x), gamma, beta, eps, static_cast<T*>(y), mean, rstd, rows, D);
    return hipGetLastError();
  }
  switch (group_of(D)) {
    case 64: fwd_g<T, 64>(x, gamma, beta, eps, y, mean, rstd, rows, D, s); break;
    case 128: fwd_g<T, 128>(x, gamma, beta, eps, y, mean, rstd, rows, D, s); break;
    case 256: fwd_g<T, 256>(x, gamma, beta, eps, y, mean, rstd, rows, D, s); break;
    case 512: fwd_g<T, 512>(x, gamma, beta, eps, y, mean, rstd, rows, D, s); break;
    default: fwd_g<T, 1024>(x, gamma, beta, eps, y, mean, rstd, rows, D, s); break;
  }
  return hipGetLastError();
}

template <typename T, int G>
void bwd_g(const void* x, const void* dy, const float* gamma, const float* mean,
           const float* rstd, const void* dres, void* dx, float* part_g, float* part_b,
           int64_t rows, int D, hipStream_t s) {
  constexpr int NV = kRegVals / Vec<T>::N;
  const int grid = static_cast<int>(bwd_parts(rows, D));
  const T *xt = static_cast<const T*>(x), *dyt = static_cast<const T*>(dy),
          *rt = static_cast<const T*>(dres);
  T* dxt = static_cast<T*>(dx);
  if (part_g != nullptr || part_b != nullptr)
    norm_bwd_kernel<T, G, NV, true>
        <<<grid, wg_of(G), 0, s>>>(xt, dyt, gamma, mean, rstd, rt, dxt, part_g, part_b, rows, D);
  else
    norm_bwd_kernel<T, G, NV, false><<<grid, wg_of(G), 0, s>>>(xt, dyt, gamma, mean, rstd, rt, dxt,
                                                               nullptr, nullptr, rows, D);
}

template <typename T>
void bwd_t(int64_t rows, int D, const void* x, const void* dy, const float* gamma,
           const float* mean, const float* rstd, const void* dres, void* dx, float* part_g,
           float* part_b, hipStream_t s) {
  if (D > kMaxRegWidth) {
    const T *xt = static_cast<const T*>(x), *dyt = static_cast<const T*>(dy);
    norm_bwd_wide_kernel<T><<<static_cast<int>(std::min<int64_t>(rows, 2 * kCus)), 1024, 0, s>>>(
        xt, dyt, gamma, mean, rstd, static_cast<const T*>(dres), static_cast<T*>(dx), rows, D);
    if (part_g != nullptr || part_b != nullptr) {
      const int64_t P = bwd_parts(rows, D);
      norm_param_kernel<T><<<dim3((D + 255) / 256, static_cast<unsigned>(P)), 256, 0, s>>>(
          xt, dyt, mean, rstd, part_g, part_b, rows, D, (rows + P - 1) / P);
    }
    return;
  }
  switch (group_of(D)) {
    case 64: bwd_g<T, 64>(x, dy, gamma, mean, rstd, dres, dx, part_g, part_b, rows, D, s); break;
    case 128: bwd_g<T, 128>(x, dy, gamma, mean, rstd, dres, dx, part_g, part_b, rows, D, s); break;
    case 256: bwd_g<T, 256>(x, dy, gamma, mean, rstd, dres, dx, part_g, part_b, rows, D, s); break;
    case 512: bwd_g<T, 512>(x, dy, gamma, mean, rstd, dres, dx, part_g, part_b, rows, D, s); break;
    default: bwd_g<T, 1024>(x, dy, gamma, mean, rstd, dres, dx, part_g, part_b, rows, D, s); break;
  }
}

}  // namespace

size_t norm_bwd_part_floats(int64_t rows, int D) {
  return 2 * static_cast<size_t>(bwd_parts(rows, D)) * D;
}

hipError_t launch_norm(bool bf16, int64_t rows, int D, const void* x, const float* gamma,
                       const float* beta, float eps, void* y, float* mean, float* rstd,
                       hipStream_t s) {
  return bf16 ? fwd_t<uint16_t>(rows, D, x, gamma, beta, eps, y, mean, rstd, s)
              : fwd_t<float>(rows, D, x, gamma, beta, eps, y, mean, rstd, s);
}

hipError_t launch_norm_bwd(bool bf16, int64_t rows, int D, const void* x, const void* dy,
                           const float* gamma, const float* mean, const float* rstd,
                           const void* dres, void* dx, float* dgamma, float* dbeta, float* part,
                           hipStream_t s) {
  const bool params = dgamma != nullptr || dbeta != nullptr;
  const int64_t P = bwd_parts(rows, D);
  if (rows > 0) {
    // One part: the sums are the gradients themselves.
    float* pg = P == 1 ? dgamma : params ? part : nullptr;
    float* pb = P == 1 ? dbeta : params ? part + P * D : nullptr;
    if (bf16)
      bwd_t<uint16_t>(rows, D, x, dy, gamma, mean, rstd, dres, dx, pg, pb, s);
    else
      bwd_t<float>(rows, D, x, dy, gamma, mean, rstd, dres, dx, pg, pb, s);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || P == 1) return e;
  }
  if (!params) return hipSuccess;
  norm_finish_kernel<<<dim3((D + kFinishCols - 1) / kFinishCols, 2), kFinishCols * kFinishRows, 0,
                       s>>>(
      part, static_cast<int>(P), D, dgamma, dbeta);
  return hipGetLastError();
}

}  // namespace moe

// Layer norm forward and backward (include/moe_norm.h).
//
//   h = (x - mean) rstd,  y = h gamma + beta
//   dx = rstd (g - mean(g) - h mean(g h)) + dres,  g = dy gamma
//   dgamma = sum_rows dy h,  dbeta = sum_rows dy
//
// Both passes are bound by memory: a few operations per value. A row belongs
// to a group of G threads (one wave, or one workgroup of G threads) that hold
// it in registers, so x (and dy) are read once; gamma and beta, and in the
// backward the column sums, stay in registers over all rows of the group.
#include <algorithm>

#include "moe_internal.h"

namespace moe {
namespace {

// Vectors of 16 bytes that need only their element's alignment: rows of odd
// widths start anywhere, and the hardware loads such vectors whole.
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef u32x4 u32x4_a2 __attribute__((aligned(2)));
typedef u32x4 u32x4_a4 __attribute__((aligned(4)));

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
    u32x4 r;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      r[i] = f32_to_bf16(f[2 * i]) | (static_cast<uint32_t>(f32_to_bf16(f[2 * i + 1])) << 16);
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
    *reinterpret_cast<typename Vec<T>::raw_a*>(row + static_cast<int64_t>(v) * N) =
        Vec<T>::pack(f);
  } else if (v == nfull) {
#pragma unroll
    for (int e = 0; e < N; ++e)
      if (e < D - nfull * N) Vec<T>::store1(row + nfull * N + e, f[e]);
  }
}
// N fp32 parameters of vector v, `pad` where there are none.
template <int N>
__device__ __forceinline__ void load_param(const float* p, int v, int D, float pad,
                                           float (&f)[N]) {
#pragma unroll
  for (int e = 0; e < N; ++e) f[e] = p != nullptr && v * N + e < D ? p[v * N + e] : pad;
}

// Sums of NS values over the group's G threads, in every thread. red holds
// 2 x NS x (G / 64) floats; calls alternate `slot`, so one barrier each is
// enough: a thread that writes a slot again has passed the barrier of the
// call in between, and with it every read of the slot's last use.
template <int G, int NS>
__device__ __forceinline__ void group_sum(float (&s)[NS], float* red, int& slot) {
#pragma unroll
  for (int i = 0; i < NS; ++i)
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) s[i] += __shfl_xor(s[i], off, 64);
  if constexpr (G > 64) {
    constexpr int W = G / 64;
    float* r = red + slot * NS * W;
    if ((threadIdx.x & 63) == 0) {
#pragma unroll
      for (int i = 0; i < NS; ++i) r[i * W + (threadIdx.x >> 6)] = s[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NS; ++i) {
      s[i] = 0.f;
#pragma unroll
      for (int w = 0; w < W; ++w) s[i] += r[i * W + w];
    }
    slot ^= 1;
  }
}

constexpr int wg_of(int G) { return G == 64 ? 256 : G; }

// ---- forward: the row in registers -----------------------------------------
template <typename T, int G, int NV>
__global__ __launch_bounds__(wg_of(G)) void norm_fwd_kernel(
    const T* __restrict__ x, const float* __restrict__ gamma, const float* __restrict__ beta,
    float eps, T* __restrict__ y, float* __restrict__ mean_out, float* __restrict__ rstd_out,
    int64_t rows, int D) {
  constexpr int N = Vec<T>::N, WG = wg_of(G), R = WG / G;
  __shared__ float red[2 * (G / 64)];
  int slot = 0;
  const int t = threadIdx.x % G, nfull = D / N;
  float gm[NV][N], bt[NV][N];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    load_param<N>(gamma, t + i * G, D, 1.f, gm[i]);
    load_param<N>(beta, t + i * G, D, 0.f, bt[i]);
  }
  const float fd = static_cast<float>(D);
  const int64_t step = static_cast<int64_t>(gridDim.x) * R;
  int64_t r = static_cast<int64_t>(blockIdx.x) * R + threadIdx.x / G;
  u32x4 next[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i)
    next[i] = r < rows ? load_vec(x + r * D, t + i * G, nfull, D) : u32x4{0, 0, 0, 0};
  for (; r < rows; r += step) {
    float f[NV][N];
#pragma unroll
    for (int i = 0; i < NV; ++i) Vec<T>::unpack(next[i], f[i]);
    if (r + step < rows) {
#pragma unroll
      for (int i = 0; i < NV; ++i) next[i] = load_vec(x + (r + step) * D, t + i * G, nfull, D);
    }
    float s[1] = {0.f};
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int e = 0; e < N; ++e) s[0] += f[i][e];
    group_sum<G, 1>(s, red, slot);
    const float mean = s[0] / fd;  // (a constant row's mean is exact where its sum is)
    s[0] = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int e = 0; e < N; ++e) {
        f[i][e] -= mean;
        if ((t + i * G) * N + e < D) s[0] = fmaf(f[i][e], f[i][e], s[0]);
      }
    group_sum<G, 1>(s, red, slot);
    const float rstd = 1.f / sqrtf(s[0] / fd + eps);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
#pragma unroll
      for (int e = 0; e < N; ++e) f[i][e] = fmaf(f[i][e] * rstd, gm[i][e], bt[i][e]);
      store_vec(y + r * D, t + i * G, nfull, D, f[i]);
    }
    if (t == 0) {
      if (mean_out != nullptr) mean_out[r] = mean;
      if (rstd_out != nullptr) rstd_out[r] = rstd;
    }
  }
}

// ---- forward: rows wider than the registers hold ---------------------------
// One workgroup a row; the second and third reads of x come from the caches.
template <typename T>
__global__ __launch_bounds__(1024) void norm_fwd_wide_kernel(
    const T* __restrict__ x, const float* __restrict__ gamma, const float* __restrict__ beta,
    float eps, T* __restrict__ y, float* __restrict__ mean_out, float* __restrict__ rstd_out,
    int64_t rows, int D) {
  constexpr int N = Vec<T>::N, G = 1024;
  __shared__ float red[2 * (G / 64)];
  int slot = 0;
  const int t = threadIdx.x, nfull = D / N, nvec = (D + N - 1) / N;
  const float fd = static_cast<float>(D);
  for (int64_t r = blockIdx.x; r < rows; r += gridDim.x) {
    const T* xr = x + r * D;
    float f[N], s[1] = {0.f};
    for (int v = t; v < nvec; v += G) {
      Vec<T>::unpack(load_vec(xr, v, nfull, D), f);
#pragma unroll
      for (int e = 0; e < N; ++e) s[0] += f[e];
    }
    group_sum<G, 1>(s, red, slot);
    const float mean = s[0] / fd;  // (a constant row's mean is exact where its sum is)
    s[0] = 0.f;
    for (int v = t; v < nvec; v += G) {
      Vec<T>::unpack(load_vec(xr, v, nfull, D), f);
#pragma unroll
      for (int e = 0; e < N; ++e)
        if (v * N + e < D) s[0] = fmaf(f[e] - mean, f[e] - mean, s[0]);
    }
    group_sum<G, 1>(s, red, slot);
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
// PARAMS: this workgroup's sums of dy h and dy over its rows go to
// part[2][gridDim.x][D].
template <typename T, int G, int NV, bool PARAMS>
__global__ __launch_bounds__(wg_of(G)) void norm_bwd_kernel(
    const T* __restrict__ x, const T* __restrict__ dy, const float* __restrict__ gamma,
    const float* __restrict__ mean_in, const float* __restrict__ rstd_in,
    const T* __restrict__ dres, T* __restrict__ dx, float* __restrict__ part, int64_t rows,
    int D) {
  constexpr int N = Vec<T>::N, WG = wg_of(G), R = WG / G;
  // Sums of the row's two means; with several groups a workgroup, the column
  // sums of the others at the end.
  __shared__ float red[R > 1 && PARAMS ? (R - 1) * 64 * NV * N : 4 * (G / 64)];
  int slot = 0;
  const int t = threadIdx.x % G, grp = threadIdx.x / G, nfull = D / N;
  float gm[NV][N], dg[NV][N], db[NV][N];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    load_param<N>(gamma, t + i * G, D, 1.f, gm[i]);
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
  if (r < rows) fetch(r);
  for (; r < rows; r += step) {
    float h[NV][N], d[NV][N], s[2] = {0.f, 0.f};
    const float mean = nm, rstd = nr;
    u32x4 res[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      Vec<T>::unpack(nx[i], h[i]);
      Vec<T>::unpack(nd[i], d[i]);
      res[i] = dres != nullptr ? load_vec(dres + r * D, t + i * G, nfull, D) : u32x4{0, 0, 0, 0};
    }
    if (r + step < rows) fetch(r + step);
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int e = 0; e < N; ++e) {
        h[i][e] = (h[i][e] - mean) * rstd;
        if (PARAMS) {
          dg[i][e] = fmaf(d[i][e], h[i][e], dg[i][e]);
          db[i][e] += d[i][e];
        }
        d[i][e] *= gm[i][e];
        // Places past D hold d = 0 and a finite h unless the row's own
        // statistics are not finite, and then the whole row is NaN anyway.
        s[0] += d[i][e];
        s[1] = fmaf(d[i][e], h[i][e], s[1]);
      }
    group_sum<G, 2>(s, red, slot);
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
    float* out = part + static_cast<int64_t>(blockIdx.x) * D;
    auto flush = [&](float(&a)[NV][N], float* o) {
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
    flush(dg, out);
    flush(db, out + static_cast<int64_t>(gridDim.x) * D);
  }
}

// ---- backward: wide rows ---------------------------------------------------
template <typename T>
__global__ __launch_bounds__(1024) void norm_bwd_wide_kernel(
    const T* __restrict__ x, const T* __restrict__ dy, const float* __restrict__ gamma,
    const float* __restrict__ mean_in, const float* __restrict__ rstd_in,
    const T* __restrict__ dres, T* __restrict__ dx, int64_t rows, int D) {
  constexpr int N = Vec<T>::N, G = 1024;
  __shared__ float red[4 * (G / 64)];
  int slot = 0;
  const int t = threadIdx.x, nfull = D / N, nvec = (D + N - 1) / N;
  const float fd = static_cast<float>(D);
  for (int64_t r = blockIdx.x; r < rows; r += gridDim.x) {
    const float mean = mean_in[r], rstd = rstd_in[r];
    float h[N], d[N], gm[N], s[2] = {0.f, 0.f};
    for (int v = t; v < nvec; v += G) {
      Vec<T>::unpack(load_vec(x + r * D, v, nfull, D), h);
      Vec<T>::unpack(load_vec(dy + r * D, v, nfull, D), d);
      load_param<N>(gamma, v, D, 1.f, gm);
#pragma unroll
      for (int e = 0; e < N; ++e) {
        s[0] = fmaf(d[e], gm[e], s[0]);
        s[1] = fmaf(d[e] * gm[e], (h[e] - mean) * rstd, s[1]);
      }
    }
    group_sum<G, 2>(s, red, slot);
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
                                                         float* __restrict__ part, int64_t rows,
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
  part[static_cast<int64_t>(blockIdx.y) * D + c] = dg;
  part[(static_cast<int64_t>(gridDim.y) + blockIdx.y) * D + c] = db;
}

// dgamma (blockIdx.y 0) and dbeta (1): the P partial rows added in row order
// per wave, then the waves in order. P == 0 writes zeros.
constexpr int kFinishWaves = 16;
__global__ __launch_bounds__(64 * kFinishWaves) void norm_finish_kernel(
    const float* __restrict__ part, int P, int D, float* __restrict__ dgamma,
    float* __restrict__ dbeta) {
  __shared__ float red[kFinishWaves][64];
  float* out = blockIdx.y == 0 ? dgamma : dbeta;
  if (out == nullptr) return;
  const int c = blockIdx.x * 64 + (threadIdx.x & 63), w = threadIdx.x >> 6;
  const float* p = part + static_cast<int64_t>(blockIdx.y) * P * D;
  float s = 0.f;
  if (c < D) {
#pragma unroll 8
    for (int q = w; q < P; q += kFinishWaves) s += p[static_cast<int64_t>(q) * D + c];
  }
  red[w][threadIdx.x & 63] = s;
  __syncthreads();
  if (w == 0 && c < D) {
#pragma unroll
    for (int q = 1; q < kFinishWaves; ++q) s += red[q][threadIdx.x];
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
           const float* rstd, const void* dres, void* dx, float* part, int64_t rows, int D,
           hipStream_t s) {
  constexpr int NV = kRegVals / Vec<T>::N;
  const int grid = static_cast<int>(bwd_parts(rows, D));
  const T *xt = static_cast<const T*>(x), *dyt = static_cast<const T*>(dy),
          *rt = static_cast<const T*>(dres);
  T* dxt = static_cast<T*>(dx);
  if (part != nullptr)
    norm_bwd_kernel<T, G, NV, true>
        <<<grid, wg_of(G), 0, s>>>(xt, dyt, gamma, mean, rstd, rt, dxt, part, rows, D);
  else
    norm_bwd_kernel<T, G, NV, false>
        <<<grid, wg_of(G), 0, s>>>(xt, dyt, gamma, mean, rstd, rt, dxt, nullptr, rows, D);
}

template <typename T>
void bwd_t(int64_t rows, int D, const void* x, const void* dy, const float* gamma,
           const float* mean, const float* rstd, const void* dres, void* dx, float* part,
           hipStream_t s) {
  if (D > kMaxRegWidth) {
    const T *xt = static_cast<const T*>(x), *dyt = static_cast<const T*>(dy);
    norm_bwd_wide_kernel<T><<<static_cast<int>(std::min<int64_t>(rows, 2 * kCus)), 1024, 0, s>>>(
        xt, dyt, gamma, mean, rstd, static_cast<const T*>(dres), static_cast<T*>(dx), rows, D);
    if (part != nullptr) {
      const int64_t P = bwd_parts(rows, D);
      norm_param_kernel<T><<<dim3((D + 255) / 256, static_cast<unsigned>(P)), 256, 0, s>>>(
          xt, dyt, mean, rstd, part, rows, D, (rows + P - 1) / P);
    }
    return;
  }
  switch (group_of(D)) {
    case 64: bwd_g<T, 64>(x, dy, gamma, mean, rstd, dres, dx, part, rows, D, s); break;
    case 128: bwd_g<T, 128>(x, dy, gamma, mean, rstd, dres, dx, part, rows, D, s); break;
    case 256: bwd_g<T, 256>(x, dy, gamma, mean, rstd, dres, dx, part, rows, D, s); break;
    case 512: bwd_g<T, 512>(x, dy, gamma, mean, rstd, dres, dx, part, rows, D, s); break;
    default: bwd_g<T, 1024>(x, dy, gamma, mean, rstd, dres, dx, part, rows, D, s); break;
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
  if (rows > 0) {
    if (bf16)
      bwd_t<uint16_t>(rows, D, x, dy, gamma, mean, rstd, dres, dx, params ? part : nullptr, s);
    else
      bwd_t<float>(rows, D, x, dy, gamma, mean, rstd, dres, dx, params ? part : nullptr, s);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (!params) return hipSuccess;
  norm_finish_kernel<<<dim3((D + 63) / 64, 2), 64 * kFinishWaves, 0, s>>>(
      part, static_cast<int>(bwd_parts(rows, D)), D, dgamma, dbeta);
  return hipGetLastError();
}

}  // namespace moe

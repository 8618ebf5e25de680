// Balance loss of the router: counts, probability sums, loss; its gradient;
// the router's backward from dense logit gradients (formulas in
// moe_balance.h).
//
// Forward and backward are bound by reading the logits (and writing their
// gradients) once: a token's E logits sit in the registers of L lanes
// (L = 8 .. 64, the power of two that covers E, 64 beyond), lane l holding
// experts l, l + L, ...; maximum and sum are exchanged between the L lanes.
// The forward sums p over a workgroup's tokens in registers, then over its
// lane groups in LDS, writes one partial of E values, and a second launch
// adds the partials in fp64 (one workgroup needs no second launch).
#include <algorithm>
#include <type_traits>

#include "moe_internal.h"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxParts = 256;   // workgroups of the forward

__device__ __forceinline__ float load_logit(const float* p) { return *p; }
__device__ __forceinline__ float load_logit(const uint16_t* p) { return bf16_to_f32(*p); }
__device__ __forceinline__ float load_logit(const _Float16* p) { return static_cast<float>(*p); }

template <int L>
__device__ __forceinline__ float group_max(float v) {
#pragma unroll
  for (int off = L / 2; off > 0; off >>= 1) v = fmaxf(v, __shfl_xor(v, off, L));
  return v;
}
template <int L>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int off = L / 2; off > 0; off >>= 1) v += __shfl_xor(v, off, L);
  return v;
}

// p of one token: e[i] = exp(z - max) on return, the factor 1 / sum returned.
// A row of -inf alone gives p = 0.
template <typename T, int L, int NI>
__device__ __forceinline__ float softmax_row(const T* __restrict__ z, int E, int l,
                                             float (&e)[NI]) {
  float m = -INFINITY;
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    e[i] = l + L * i < E ? load_logit(z + l + L * i) : -INFINITY;
    m = fmaxf(m, e[i]);
  }
  m = group_max<L>(m);
  if (m == -INFINITY) m = 0.f;  // (fmaxf drops NaN; exp(NaN) brings it back)
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    e[i] = expf(e[i] - m);
    s += e[i];
  }
  s = group_sum<L>(s);
  return s == 0.f ? 0.f : 1.f / s;
}

// ws: prob[parts][E] fp32, count[parts][E], tokens[parts] (with one part the
// results are written at once).
__device__ __forceinline__ void write_loss(int E, int k, float coef, const int32_t* counts,
                                           int32_t n, const double* prob, int32_t* tokens,
                                           float* loss, double* s_red) {
  double v = 0.0;
  for (int e = threadIdx.x; e < E; e += blockDim.x) v += prob[e] * counts[e];
  s_red[threadIdx.x] = v;
  __syncthreads();
  for (int w = static_cast<int>(blockDim.x) / 2; w > 0; w >>= 1) {
    if (static_cast<int>(threadIdx.x) < w) s_red[threadIdx.x] += s_red[threadIdx.x + w];
    __syncthreads();
  }
  if (threadIdx.x == 0) {
    const double N = n;
    *tokens = n;
    *loss = n > 0 ? static_cast<float>(coef * (static_cast<double>(E) / (k * N * N)) * s_red[0])
                  : 0.f;
  }
}

template <typename T, int L, int NI>
__global__ __launch_bounds__(kThreads) void balance_part_kernel(
    int Tn, int E, int k, const T* __restrict__ logits, const int32_t* __restrict__ topk,
    const uint8_t* __restrict__ mask, float coef, int parts, float* __restrict__ p_prob,
    int32_t* __restrict__ p_count, int32_t* __restrict__ p_tok, int32_t* __restrict__ counts,
    int32_t* __restrict__ tokens, float* __restrict__ prob_sum, float* __restrict__ loss) {
  constexpr int G = kThreads / L;   // tokens at a time
  constexpr int EC = L * NI;
  __shared__ float s_prob[kThreads * NI];        // [G][EC]
  __shared__ int32_t s_count[EC];
  __shared__ int32_t s_tok;
  __shared__ double s_d[EC + kThreads];
  const int tid = threadIdx.x, l = tid % L, g = tid / L;
  for (int e = tid; e < EC; e += kThreads) s_count[e] = 0;
  if (tid == 0) s_tok = 0;
  __syncthreads();
  const int64_t t0 = static_cast<int64_t>(Tn) * blockIdx.x / parts;
  const int64_t t1 = static_cast<int64_t>(Tn) * (blockIdx.x + 1) / parts;
  float acc[NI] = {};
  int tok = 0;
  for (int64_t t = t0 + g; t < t1; t += G) {
    if (mask && mask[t] == 0) continue;  // (uniform in the token's lanes)
    float e[NI];
    const float r = softmax_row<T, L, NI>(logits + t * E, E, l, e);
#pragma unroll
    for (int i = 0; i < NI; ++i) acc[i] += e[i] * r;
    tok += l == 0;
  }
  for (int64_t q = t0 * k + tid; q < t1 * k; q += kThreads) {
    const int e = topk[q];
    if (e >= 0 && e < E && !(mask && mask[q / k] == 0)) atomicAdd(&s_count[e], 1);
  }
  if (tok) atomicAdd(&s_tok, tok);
#pragma unroll
  for (int i = 0; i < NI; ++i) s_prob[g * EC + l + L * i] = acc[i];
  __syncthreads();
  for (int e = tid; e < E; e += kThreads) {
    float v = 0.f;
    for (int j = 0; j < G; ++j) v += s_prob[j * EC + e];
    if (parts == 1) {
      counts[e] = s_count[e];
      prob_sum[e] = v;
      s_d[e] = v;
    } else {
      p_prob[static_cast<int64_t>(blockIdx.x) * E + e] = v;
      p_count[static_cast<int64_t>(blockIdx.x) * E + e] = s_count[e];
    }
  }
  if (parts > 1) {
    if (tid == 0) p_tok[blockIdx.x] = s_tok;
    return;
  }
  __syncthreads();
  write_loss(E, k, coef, s_count, s_tok, s_d, tokens, loss, s_d + EC);
}

// One workgroup of 1024 threads: the partials of an expert are summed by
// 1024 / EP threads (EP: E rounded up to a power of two), each taking every
// so-manieth part in order, then joined in order.
__global__ __launch_bounds__(1024) void balance_finish_kernel(
    int E, int k, float coef, int parts, int EP, const float* __restrict__ p_prob,
    const int32_t* __restrict__ p_count, const int32_t* __restrict__ p_tok,
    int32_t* __restrict__ counts, int32_t* __restrict__ tokens, float* __restrict__ prob_sum,
    float* __restrict__ loss) {
  __shared__ double s_prob[1024];
  __shared__ int32_t s_count[1024];
  __shared__ double s_red[1024];
  __shared__ int32_t s_tok;
  const int tid = threadIdx.x, e = tid % EP, j = tid / EP, J = 1024 / EP;
  if (tid == 0) s_tok = 0;
  double v = 0.0;
  int c = 0;
  if (e < E)
    for (int p = j; p < parts; p += J) {
      v += p_prob[static_cast<int64_t>(p) * E + e];
      c += p_count[static_cast<int64_t>(p) * E + e];
    }
  s_red[tid] = v;
  s_count[tid] = c;
  __syncthreads();
  if (tid < parts) atomicAdd(&s_tok, p_tok[tid]);
  if (j == 0) {
    for (int i = 1; i < J; ++i) {
      v += s_red[i * EP + e];
      c += s_count[i * EP + e];
    }
    if (e < E) {
      counts[e] = c;
      prob_sum[e] = static_cast<float>(v);
      s_prob[e] = v;
    }
  }
  __syncthreads();
  if (j == 0 && e < E) s_count[e] = c;
  __syncthreads();
  write_loss(E, k, coef, s_count, s_tok, s_prob, tokens, loss, s_red);
}

__global__ void balance_empty_kernel(int E, int32_t* counts, int32_t* tokens, float* prob_sum,
                                     float* loss) {
  for (int e = threadIdx.x; e < E; e += blockDim.x) {
    counts[e] = 0;
    prob_sum[e] = 0.f;
  }
  if (threadIdx.x == 0) {
    *tokens = 0;
    *loss = 0.f;
  }
}

template <typename T, int L, int NI>
__global__ __launch_bounds__(kThreads) void balance_bwd_kernel(
    int Tn, int E, int k, const T* __restrict__ logits, const int32_t* __restrict__ topk,
    const uint8_t* __restrict__ mask, float coef, const int32_t* __restrict__ counts,
    const int32_t* __restrict__ tokens, const float* __restrict__ dloss,
    const float* __restrict__ dlogit, float* __restrict__ dlogits) {
  constexpr int G = kThreads / L;
  const int tid = threadIdx.x, l = tid % L;
  const double N = *tokens;
  // coef E / (k N^2) c: the gradient of the loss for p
  const double scale = N > 0.0 ? static_cast<double>(coef) * E / (k * N * N) *
                                     (dloss ? static_cast<double>(*dloss) : 1.0)
                               : 0.0;
  float f[NI];
#pragma unroll
  for (int i = 0; i < NI; ++i)
    f[i] = l + L * i < E ? static_cast<float>(scale * counts[l + L * i]) : 0.f;
  const int64_t step = static_cast<int64_t>(gridDim.x) * G;
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * G + tid / L; t < Tn; t += step) {
    float d[NI] = {};
    if (!(mask && mask[t] == 0)) {
      float e[NI];
      const float r = softmax_row<T, L, NI>(logits + t * E, E, l, e);
      float dot = 0.f;
#pragma unroll
      for (int i = 0; i < NI; ++i) dot += e[i] * f[i];
      dot = group_sum<L>(dot) * r;
#pragma unroll
      for (int i = 0; i < NI; ++i) d[i] = e[i] * r * (f[i] - dot);
    }
    if (dlogit) {
      for (int j = 0; j < k; ++j) {
        const int x = topk[t * k + j];
        const float v = dlogit[t * k + j];
#pragma unroll
        for (int i = 0; i < NI; ++i)
          if (x == l + L * i) d[i] += v;
      }
    }
#pragma unroll
    for (int i = 0; i < NI; ++i)
      if (l + L * i < E) dlogits[t * E + l + L * i] = d[i];
  }
}

// ---------------------------------------------------------------------------
// Dense router backward on v_mfma_f32_32x32x2_f32.
//   dx [T, D] = dz [T, E] W [E, D]    (contraction over experts)
//   dW [E, D] = dz^T [E, T] x [T, D]  (contraction over tokens, in parts)
// C [M, N] = sum_k A(k, m) B(k, n), a 64 x 64 tile per workgroup of four
// waves (one 32 x 32 block each), K in steps of 16 through LDS.
// ---------------------------------------------------------------------------
typedef float f32x16 __attribute__((ext_vector_type(16)));
constexpr int TM = 64, TN = 64, TK = 16, kLdsPitch = 68;

// A_KM: A is [K][M] in memory (dz for dW), else [M][K] (dz for dx).
template <typename TB, bool A_KM>
__global__ __launch_bounds__(kThreads) void router_dense_kernel(
    const float* __restrict__ A, const TB* __restrict__ B, float* __restrict__ C, int64_t M,
    int N, int64_t K, int parts, int accumulate) {
  __shared__ float sa[TK * kLdsPitch], sb[TK * kLdsPitch];
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
  const int nt = (N + TN - 1) / TN;
  const int64_t m0 = static_cast<int64_t>(blockIdx.x / nt) * TM;
  const int n0 = static_cast<int>(blockIdx.x % nt) * TN;
  const int64_t k0 = K * blockIdx.y / parts, k1 = K * (blockIdx.y + 1) / parts;
  C += static_cast<int64_t>(blockIdx.y) * M * N;
  const int wm = 32 * (wave >> 1), wn = 32 * (wave & 1);
  f32x16 acc;
#pragma unroll
  for (int r = 0; r < 16; ++r) acc[r] = 0.f;
  for (int64_t kb = k0; kb < k1; kb += TK) {
#pragma unroll
    for (int i = 0; i < TK * TM / kThreads; ++i) {
      const int q = tid + kThreads * i;
      const int kk = A_KM ? q / TM : q % TK, m = A_KM ? q % TM : q / TK;
      const bool ok = kb + kk < k1 && m0 + m < M;
      sa[kk * kLdsPitch + m] =
          ok ? A[A_KM ? (kb + kk) * M + m0 + m : (m0 + m) * K + kb + kk] : 0.f;
      const int bk = q / TN, n = q % TN;
      const bool okb = kb + bk < k1 && n0 + n < N;
      sb[bk * kLdsPitch + n] = okb ? load_act(B + (kb + bk) * N + n0 + n) : 0.f;
    }
    __syncthreads();
#pragma unroll
    for (int kk = 0; kk < TK; kk += 2) {
      const int ks = kk + (lane >> 5);
      acc = __builtin_amdgcn_mfma_f32_32x32x2f32(sa[ks * kLdsPitch + wm + (lane & 31)],
                                                 sb[ks * kLdsPitch + wn + (lane & 31)], acc, 0, 0,
                                                 0);
    }
    __syncthreads();
  }
#pragma unroll
  for (int r = 0; r < 16; ++r) {
    const int64_t m = m0 + wm + 8 * (r / 4) + 4 * (lane >> 5) + r % 4;
    const int n = n0 + wn + (lane & 31);
    if (m < M && n < N) {
      float* c = C + m * N + n;
      *c = accumulate ? *c + acc[r] : acc[r];
    }
  }
}

__global__ __launch_bounds__(kThreads) void router_dense_sum_kernel(const float4* __restrict__ part,
                                                                    float4* __restrict__ out,
                                                                    int64_t n4, int parts) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  if (i >= n4) return;
  float4 v = part[i];
  for (int p = 1; p < parts; ++p) {
    const float4 w = part[p * n4 + i];
    v.x += w.x;
    v.y += w.y;
    v.z += w.z;
    v.w += w.w;
  }
  out[i] = v;
}

// Workgroups of the forward: some 8 K logits each, at most kMaxParts.
int balance_parts(int T, int E) {
  const int64_t n = (static_cast<int64_t>(T) * E + 8191) / 8192;
  return static_cast<int>(std::min<int64_t>(std::max<int64_t>(n, 1), kMaxParts));
}

// Parts of the tokens in dW: enough workgroups for the chip, at least 256
// tokens each.
int dense_parts(int T, int E, int D) {
  const int64_t tiles = static_cast<int64_t>((E + TM - 1) / TM) * ((D + TN - 1) / TN);
  const int64_t want = (1024 + tiles - 1) / tiles;
  return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(want, (T + 255) / 256)));
}

// f(lanes per token, registers per lane) for E experts.
template <typename F>
hipError_t for_experts(int E, F f) {
  if (E <= 8) return f(std::integral_constant<int, 8>{}, std::integral_constant<int, 1>{});
  if (E <= 16) return f(std::integral_constant<int, 16>{}, std::integral_constant<int, 1>{});
  if (E <= 32) return f(std::integral_constant<int, 32>{}, std::integral_constant<int, 1>{});
  if (E <= 64) return f(std::integral_constant<int, 64>{}, std::integral_constant<int, 1>{});
  if (E <= 128) return f(std::integral_constant<int, 64>{}, std::integral_constant<int, 2>{});
  if (E <= 256) return f(std::integral_constant<int, 64>{}, std::integral_constant<int, 4>{});
  if (E <= 512) return f(std::integral_constant<int, 64>{}, std::integral_constant<int, 8>{});
  return f(std::integral_constant<int, 64>{}, std::integral_constant<int, 16>{});
}

template <typename T>
hipError_t balance_loss(int Tn, int E, int k, const T* logits, const int32_t* topk,
                        const uint8_t* mask, float coef, int32_t* counts, int32_t* tokens,
                        float* prob_sum, float* loss, void* ws, hipStream_t s) {
  const int parts = balance_parts(Tn, E);
  float* p_prob = static_cast<float*>(ws);
  int32_t* p_count = reinterpret_cast<int32_t*>(p_prob + static_cast<int64_t>(parts) * E);
  int32_t* p_tok = p_count + static_cast<int64_t>(parts) * E;
  hipError_t e = for_experts(E, [&](auto L, auto NI) {
    balance_part_kernel<T, decltype(L)::value, decltype(NI)::value>
        <<<parts, kThreads, 0, s>>>(Tn, E, k, logits, topk, mask, coef, parts, p_prob, p_count,
                                    p_tok, counts, tokens, prob_sum, loss);
    return hipGetLastError();
  });
  if (e == hipSuccess && parts > 1) {
    int EP = 1;
    while (EP < E) EP *= 2;
    balance_finish_kernel<<<1, 1024, 0, s>>>(E, k, coef, parts, EP, p_prob, p_count, p_tok,
                                             counts, tokens, prob_sum, loss);
    e = hipGetLastError();
  }
  return e;
}

template <typename T>
hipError_t balance_bwd(int Tn, int E, int k, const T* logits, const int32_t* topk,
                       const uint8_t* mask, float coef, const int32_t* counts,
                       const int32_t* tokens, const float* dloss, const float* dlogit,
                       float* dlogits, hipStream_t s) {
  return for_experts(E, [&](auto L, auto NI) {
    constexpr int G = kThreads / decltype(L)::value;
    const int64_t grid = std::min<int64_t>((static_cast<int64_t>(Tn) + G - 1) / G, 2048);
    balance_bwd_kernel<T, decltype(L)::value, decltype(NI)::value>
        <<<static_cast<unsigned>(grid), kThreads, 0, s>>>(Tn, E, k, logits, topk, mask, coef,
                                                          counts, tokens, dloss, dlogit, dlogits);
    return hipGetLastError();
  });
}

template <typename TX>
hipError_t dense_bwd(int T, int E, int D, const float* dlogits, const TX* x, const float* w,
                     int accumulate, float* dx, float* dw, float* ws, hipStream_t s) {
  hipError_t e = hipSuccess;
  const int nt = (D + TN - 1) / TN;
  if (dx != nullptr && T > 0) {
    const int64_t mt = (static_cast<int64_t>(T) + TM - 1) / TM;
    router_dense_kernel<float, false><<<static_cast<unsigned>(mt * nt), kThreads, 0, s>>>(
        dlogits, w, dx, T, D, E, 1, accumulate);
    e = hipGetLastError();
  }
  if (e == hipSuccess && dw != nullptr) {
    const int parts = T > 0 ? dense_parts(T, E, D) : 1;
    const int64_t mt = (E + TM - 1) / TM;
    const dim3 grid(static_cast<unsigned>(mt * nt), static_cast<unsigned>(parts));
    router_dense_kernel<TX, true><<<grid, kThreads, 0, s>>>(dlogits, x, parts > 1 ? ws : dw, E, D,
                                                            T, parts, 0);
    e = hipGetLastError();
    if (e == hipSuccess && parts > 1) {
      const int64_t n4 = static_cast<int64_t>(E) * D / 4;
      router_dense_sum_kernel<<<static_cast<unsigned>((n4 + kThreads - 1) / kThreads), kThreads, 0,
                                s>>>(reinterpret_cast<const float4*>(ws),
                                     reinterpret_cast<float4*>(dw), n4, parts);
      e = hipGetLastError();
    }
  }
  return e;
}

}  // namespace

size_t balance_ws_bytes(int T, int E) {
  const size_t parts = static_cast<size_t>(balance_parts(T, E));
  return parts * E * 8 + parts * 4;
}

hipError_t launch_balance_loss(int dtype, int T, int E, int k, const void* logits,
                               const int32_t* topk, const uint8_t* mask, float coef,
                               int32_t* counts, int32_t* tokens, float* prob_sum, float* loss,
                               void* ws, hipStream_t s) {
  if (T == 0) {
    balance_empty_kernel<<<1, 256, 0, s>>>(E, counts, tokens, prob_sum, loss);
    return hipGetLastError();
  }
  if (dtype == MOE_F32)
    return balance_loss(T, E, k, static_cast<const float*>(logits), topk, mask, coef, counts,
                        tokens, prob_sum, loss, ws, s);
  if (dtype == MOE_BF16)
    return balance_loss(T, E, k, static_cast<const uint16_t*>(logits), topk, mask, coef, counts,
                        tokens, prob_sum, loss, ws, s);
  return balance_loss(T, E, k, static_cast<const _Float16*>(logits), topk, mask, coef, counts,
                      tokens, prob_sum, loss, ws, s);
}

hipError_t launch_balance_bwd(int dtype, int T, int E, int k, const void* logits,
                              const int32_t* topk, const uint8_t* mask, float coef,
                              const int32_t* counts, const int32_t* tokens, const float* dloss,
                              const float* dlogit, float* dlogits, hipStream_t s) {
  if (T == 0) return hipSuccess;
  if (dtype == MOE_F32)
    return balance_bwd(T, E, k, static_cast<const float*>(logits), topk, mask, coef, counts,
                       tokens, dloss, dlogit, dlogits, s);
  if (dtype == MOE_BF16)
    return balance_bwd(T, E, k, static_cast<const uint16_t*>(logits), topk, mask, coef, counts,
                       tokens, dloss, dlogit, dlogits, s);
  return balance_bwd(T, E, k, static_cast<const _Float16*>(logits), topk, mask, coef, counts,
                     tokens, dloss, dlogit, dlogits, s);
}

size_t router_dense_ws_floats(int T, int E, int D) {
  const int parts = T > 0 ? dense_parts(T, E, D) : 1;
  return parts > 1 ? static_cast<size_t>(parts) * E * D : 0;
}

hipError_t launch_router_dense_bwd(bool bf16, int T, int E, int D, const float* dlogits,
                                   const void* x, const float* w, int accumulate, float* dx,
                                   float* dw, float* ws, hipStream_t s) {
  if (bf16)
    return dense_bwd(T, E, D, dlogits, static_cast<const uint16_t*>(x), w, accumulate, dx, dw, ws,
                     s);
  return dense_bwd(T, E, D, dlogits, static_cast<const float*>(x), w, accumulate, dx, dw, ws, s);
}

}  // namespace moe

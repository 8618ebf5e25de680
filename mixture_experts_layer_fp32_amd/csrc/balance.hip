// Balance loss of the router: counts, probability sums, loss; its gradient;
// the router's backward from dense logit gradients (formulas in
// moe_balance.h).
//
// Forward and backward read the logits (and write their gradients) once: a
// token's E logits sit in the registers of L lanes, lane l holding experts l,
// l + L, ... (NI of them): few lanes a token (L = 4 .. 64, up to 8 logits each)
// keep several tokens in a wave and the exchanges of maximum and sum short. The forward sums p over a workgroup's tokens in
// registers, then over its lane groups in LDS, writes one partial of E values,
// and a second launch adds the partials in fp64 (one workgroup needs no second
// launch). 16384 x 128 fp32 logits, k = 8: 10.4 + 5.9 us forward, 9.6 backward in
// a trace with two sets of inputs (12.1 and 7.5 us a call over one set), where
// the 8.4 MB to read take 1.7 us (the gradient's 16.8 MB 3.3): kMaxParts
// workgroups leave half of the CUs without work, and the second launch, one
// workgroup, reads 128 parts. (More parts, and a join without a launch of its
// own, have not been measured.)
#include <algorithm>
#include <type_traits>

#include "moe_internal.h"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kLossThreads = 512;
constexpr int kMaxParts = 128;   // workgroups of the forward

__device__ __forceinline__ float load_logit(const float* p) { return *p; }
__device__ __forceinline__ float load_logit(const uint16_t* p) { return bf16_to_f32(*p); }
__device__ __forceinline__ float load_logit(const _Float16* p) { return static_cast<float>(*p); }

// Exchanges between the L lanes of a token: inside 16 lanes by DPP, beyond by
// shuffles.
template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
  return __builtin_bit_cast(
      float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), CTRL, 0xF, 0xF, false));
}
template <int L, typename F>
__device__ __forceinline__ float group_reduce(float v, F f) {
  if (L > 1) v = f(v, dpp<0xB1>(v));    // lane ^ 1
  if (L > 2) v = f(v, dpp<0x4E>(v));    // lane ^ 2
  if (L > 4) v = f(v, dpp<0x141>(v));   // 7 - lane in groups of 8
  if (L > 8) v = f(v, dpp<0x140>(v));   // 15 - lane in groups of 16
  if (L > 16) v = f(v, __shfl_xor(v, 16, 64));
  if (L > 32) v = f(v, __shfl_xor(v, 32, 64));
  return v;
}
template <int L>
__device__ __forceinline__ float group_max(float v) {
  return group_reduce<L>(v, [](float a, float b) { return fmaxf(a, b); });
}
template <int L>
__device__ __forceinline__ float group_sum(float v) {
  return group_reduce<L>(v, [](float a, float b) { return a + b; });
}

// A token's logits (-inf past E), loaded without branches.
template <typename T, int L, int NI>
__device__ __forceinline__ void load_row(const T* __restrict__ z, int E, int l, float (&e)[NI]) {
#pragma unroll
  for (int i = 0; i < NI; ++i) e[i] = load_logit(z + min(l + L * i, E - 1));
#pragma unroll
  for (int i = 0; i < NI; ++i) e[i] = l + L * i < E ? e[i] : -INFINITY;
}
// p of one token: its logits in e, exp(z - max) on return, the factor 1 / sum
// returned. A row of -inf alone gives p = 0.
template <int L, int NI>
__device__ __forceinline__ float softmax_row(float (&e)[NI]) {
  float m = -INFINITY;
#pragma unroll
  for (int i = 0; i < NI; ++i) m = fmaxf(m, e[i]);
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

// The loss from the sums: v, each thread's share of sum c P, is added over the
// workgroup (waves by shuffles, then in order).
__device__ __forceinline__ void write_loss(int E, int k, float coef, double v, int32_t n,
                                           int32_t* tokens, float* loss, double* s_red) {
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) v += __shfl_xor(v, off, 64);
  if ((threadIdx.x & 63) == 0) s_red[threadIdx.x >> 6] = v;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < static_cast<int>(blockDim.x) / 64; ++w) v += s_red[w];
    const double N = n;
    *tokens = n;
    *loss = n > 0 ? static_cast<float>(coef * (static_cast<double>(E) / (k * N * N)) * v) : 0.f;
  }
}

// With more than one part, each writes p_prob[part][E] fp32, p_count[part][E]
// and p_tok[part] (the workspace, in this order).
template <typename T, int L, int NI>
__global__ __launch_bounds__(kLossThreads) void balance_part_kernel(
    int Tn, int E, int k, const T* __restrict__ logits, const int32_t* __restrict__ topk,
    const uint8_t* __restrict__ mask, float coef, int parts, float* __restrict__ p_prob,
    int32_t* __restrict__ p_count, int32_t* __restrict__ p_tok, int32_t* __restrict__ counts,
    int32_t* __restrict__ tokens, float* __restrict__ prob_sum, float* __restrict__ loss) {
  constexpr int G = kLossThreads / L;   // tokens at a time
  constexpr int EC = L * NI;
  __shared__ float s_prob[kLossThreads * NI];    // [G][EC]
  __shared__ int32_t s_count[EC];
  __shared__ int32_t s_tok;
  __shared__ double s_red[kLossThreads / 64];
  const int tid = threadIdx.x, l = tid % L, g = tid / L;
  for (int e = tid; e < EC; e += kLossThreads) s_count[e] = 0;
  if (tid == 0) s_tok = 0;
  __syncthreads();
  const int64_t t0 = static_cast<int64_t>(Tn) * blockIdx.x / parts;
  const int64_t t1 = static_cast<int64_t>(Tn) * (blockIdx.x + 1) / parts;
  float acc[NI] = {};
  int tok = 0;
  // The first slots of this thread, read before the tokens' logits are waited
  // for.
  constexpr int kSlots = 4;
  const int64_t q0 = t0 * k + tid, q1 = t1 * k;
  int slot[kSlots];
#pragma unroll
  for (int i = 0; i < kSlots; ++i) slot[i] = topk[min(q0 + i * kLossThreads, q1 - 1)];
  // Two tokens at a time (fewer registers: one), logits and mask in flight
  // together; a token that does not count is read and left out.
  constexpr int U = NI <= 8 ? 2 : 1;
  for (int64_t t = t0 + g; t < t1; t += U * G) {
    float e[U][NI];
    bool on[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t tu = min(t + u * G, t1 - 1);
      load_row<T, L, NI>(logits + tu * E, E, l, e[u]);
      on[u] = t + u * G < t1 && !(mask && mask[tu] == 0);
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (on[u]) {  // (uniform in the token's lanes)
        const float r = softmax_row<L, NI>(e[u]);
#pragma unroll
        for (int i = 0; i < NI; ++i) acc[i] += e[u][i] * r;
        tok += l == 0;
      }
  }
  auto count = [&](int64_t q, int e) {
    // (a part has fewer than 2^31 slots)
    if (e >= 0 && e < E && !(mask && mask[t0 + static_cast<uint32_t>(q - t0 * k) / k] == 0))
      atomicAdd(&s_count[e], 1);
  };
#pragma unroll
  for (int i = 0; i < kSlots; ++i)
    if (q0 + i * kLossThreads < q1) count(q0 + i * kLossThreads, slot[i]);
  for (int64_t q = q0 + kSlots * kLossThreads; q < q1; q += kLossThreads) count(q, topk[q]);
  if (tok) atomicAdd(&s_tok, tok);
#pragma unroll
  for (int i = 0; i < NI; ++i) s_prob[g * EC + l + L * i] = acc[i];
  __syncthreads();
  // Sum over the G lane groups: two halves until one is left.
  for (int w = G / 2; w > 0; w >>= 1) {
    for (int q = tid; q < w * EC; q += kLossThreads) s_prob[q] += s_prob[q + w * EC];
    __syncthreads();
  }
  double cp = 0.0;
  for (int e = tid; e < E; e += kLossThreads) {
    const float v = s_prob[e];
    if (parts == 1) {
      counts[e] = s_count[e];
      prob_sum[e] = v;
      cp += static_cast<double>(v) * s_count[e];
    } else {
      p_prob[static_cast<int64_t>(blockIdx.x) * E + e] = v;
      p_count[static_cast<int64_t>(blockIdx.x) * E + e] = s_count[e];
    }
  }
  if (parts > 1) {
    if (tid == 0) p_tok[blockIdx.x] = s_tok;
    return;
  }
  write_loss(E, k, coef, cp, s_tok, tokens, loss, s_red);
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
  __shared__ double s_red[16];
  const int tid = threadIdx.x, e = tid % EP, j = tid / EP, J = 1024 / EP;
  // Tokens: every wave adds the parts' numbers up for itself.
  int n = 0;
  for (int p = tid & 63; p < parts; p += 64) n += p_tok[p];
  double v = 0.0;
  int c = 0;
  if (e < E) {
    for (int p0 = j; p0 < parts; p0 += 16 * J) {  // sixteen parts' loads in flight
      float f[16];
      int m[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int p = min(p0 + i * J, parts - 1);
        f[i] = p_prob[static_cast<int64_t>(p) * E + e];
        m[i] = p_count[static_cast<int64_t>(p) * E + e];
      }
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (p0 + i * J < parts) {
          v += f[i];
          c += m[i];
        }
    }
  }
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) n += __shfl_xor(n, off, 64);
  s_prob[tid] = v;
  s_count[tid] = c;
  __syncthreads();
  double cp = 0.0;
  if (j == 0) {
    for (int i = 1; i < J; ++i) {
      v += s_prob[i * EP + e];
      c += s_count[i * EP + e];
    }
    if (e < E) {
      counts[e] = c;
      prob_sum[e] = static_cast<float>(v);
      cp = v * c;
    }
  }
  write_loss(E, k, coef, cp, n, tokens, loss, s_red);
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
  constexpr int kSlots = 8;
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
    float d[NI] = {}, e[NI];
    load_row<T, L, NI>(logits + t * E, E, l, e);
    // The first slots, in flight with the logits.
    int x[kSlots];
    float v[kSlots];
    if (dlogit) {
#pragma unroll
      for (int j = 0; j < kSlots; ++j) {
        x[j] = topk[t * k + min(j, k - 1)];
        v[j] = dlogit[t * k + min(j, k - 1)];
      }
    }
    if (!(mask && mask[t] == 0)) {
      const float r = softmax_row<L, NI>(e);
      float dot = 0.f;
#pragma unroll
      for (int i = 0; i < NI; ++i) dot += e[i] * f[i];
      dot = group_sum<L>(dot) * r;
#pragma unroll
      for (int i = 0; i < NI; ++i) d[i] = e[i] * r * (f[i] - dot);
    }
    if (dlogit) {
      auto add = [&](int xj, float vj) {
#pragma unroll
        for (int i = 0; i < NI; ++i)
          if (xj == l + L * i) d[i] += vj;
      };
#pragma unroll
      for (int j = 0; j < kSlots; ++j)
        if (j < k) add(x[j], v[j]);
      for (int j = kSlots; j < k; ++j) add(topk[t * k + j], dlogit[t * k + j]);
    }
    if (E == L * NI) {
#pragma unroll
      for (int i = 0; i < NI; ++i) dlogits[t * E + l + L * i] = d[i];
    } else {
#pragma unroll
      for (int i = 0; i < NI; ++i)
        if (l + L * i < E) dlogits[t * E + l + L * i] = d[i];
    }
  }
}

// ---------------------------------------------------------------------------
// Dense router backward
//   dx [T, D] = dz [T, E] W [E, D]    (contraction over experts)
//   dW [E, D] = dz^T [E, T] x [T, D]  (contraction over tokens, in parts)
// with fp32 precision on the bf16 matrix cores: an fp32 value is the exact sum
// of three bf16 values (its 24 significant bits cut into 8 each), a product of
// two is nine bf16 products, of which those below 2^-24 of it (lo mid, mid lo
// and lo lo) are left out; x in bf16 needs three. That is six (three)
// instructions at 16 times the rate of the fp32 one. (Infinities come out as
// NaN.)
// ---------------------------------------------------------------------------
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef unsigned u32x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
typedef __attribute__((address_space(3))) unsigned char lds_u8;

// The three parts of two values, packed (a in the low half).
__device__ __forceinline__ void split2(float a, float b, uint32_t& hi, uint32_t& mid,
                                       uint32_t& lo) {
  const uint32_t a1 = __float_as_uint(a), b1 = __float_as_uint(b);
  const float ar = a - __uint_as_float(a1 & 0xffff0000u);
  const float br = b - __uint_as_float(b1 & 0xffff0000u);
  const uint32_t a2 = __float_as_uint(ar), b2 = __float_as_uint(br);
  const uint32_t a3 = __float_as_uint(ar - __uint_as_float(a2 & 0xffff0000u));
  const uint32_t b3 = __float_as_uint(br - __uint_as_float(b2 & 0xffff0000u));
  hi = __builtin_amdgcn_perm(b1, a1, 0x07060302);
  mid = __builtin_amdgcn_perm(b2, a2, 0x07060302);
  lo = __builtin_amdgcn_perm(b3, a3, 0x07060302);
}
__device__ __forceinline__ void split8(const float (&f)[8], uint4 (&p)[3]) {
  uint32_t w[3][4];
#pragma unroll
  for (int i = 0; i < 4; ++i) split2(f[2 * i], f[2 * i + 1], w[0][i], w[1][i], w[2][i]);
#pragma unroll
  for (int q = 0; q < 3; ++q) p[q] = make_uint4(w[q][0], w[q][1], w[q][2], w[q][3]);
}
__device__ __forceinline__ f32x16 mma32(const uint4& a, const uint4& b, const f32x16& c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a),
                                                 __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}
// c += a b from the parts, smallest products first.
__device__ __forceinline__ f32x16 mma_parts(const uint4 (&a)[3], const uint4 (&b)[3], f32x16 c) {
  c = mma32(a[2], b[0], c);
  c = mma32(a[0], b[2], c);
  c = mma32(a[1], b[1], c);
  c = mma32(a[1], b[0], c);
  c = mma32(a[0], b[1], c);
  return mma32(a[0], b[0], c);
}

// dx of up to KC experts: a workgroup takes MT tokens and a range of columns. Its
// dz is split into LDS ([part][KC / 64][MT tokens][64], 16-byte chunk c of token
// r at c ^ (r & 7) ^ ((r >> 3) & 1)); every wave takes blocks
// of 32 columns, reads W from memory in the fragments' own order (a lane 8
// experts of one column) one block ahead and splits it in registers: W is
// read once per workgroup, mostly from L2, and needs no workspace. Eight waves
// over 128 tokens for up to 128 experts (with four over 64 tokens, two
// workgroups a CU, W is read and split twice as often: 63 us for T = 16384,
// E = 128, D = 2048, against 54 to 57; its products alone would take 41 at the
// rate of a large bf16 product), four over 64 tokens beyond (LDS).
constexpr unsigned kOutOfRange = 0x80000000u;  // past W (at most 2^30 bytes), and so is a chunk's
template <int KC, int MT, int THREADS>
__global__ __launch_bounds__(THREADS, 1) void router_dx_kernel(
    const float* __restrict__ dz, const float* __restrict__ W, float* __restrict__ dx, int T,
    int E, int D, int cols, int col_tiles, int accumulate) {
  constexpr int NM = MT / 32, NW = THREADS / 64, NK = KC / 16;
  constexpr int kPlane = MT * (KC < 64 ? 64 : KC) * 2;  // (rows of 64 at least)
  __shared__ __attribute__((aligned(16))) unsigned char smem[3 * kPlane];
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
  const int64_t t0 = static_cast<int64_t>(blockIdx.x / col_tiles) * MT;
  const int c_begin = static_cast<int>(blockIdx.x % col_tiles) * cols;
  const int c_end = min(c_begin + cols, D);
  const int half = lane >> 5, l31 = lane & 31;
  // dz's rows of this workgroup; tokens past T read zeros.
  const __amdgpu_buffer_rsrc_t z_rsrc = __builtin_amdgcn_make_buffer_rsrc(
      (void*)(dz + t0 * E), 0, static_cast<int>(min(static_cast<int64_t>(MT), T - t0)) * E * 4,
      0x00020000);
  for (int q = tid; q < MT * (KC / 8); q += THREADS) {
    const int r = q / (KC / 8), c = q % (KC / 8);
    // (experts past E: the next token's values, replaced by zeros)
    const int at = (r * E + 8 * c) * 4;
    const f32x4 lo = __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(z_rsrc, at, 0, 0));
    const f32x4 hi = __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(z_rsrc, at + 16, 0, 0));
    float f[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = 8 * c + j < E ? (j < 4 ? lo[j & 3] : hi[j & 3]) : 0.f;
    uint4 p[3];
    split8(f, p);
    const int o = (c >> 3) * (MT * 128) + r * 128 +
                  (((c & 7) ^ (r & 7) ^ ((r >> 3) & 1)) << 4);
#pragma unroll
    for (int i = 0; i < 3; ++i) *reinterpret_cast<uint4*>(smem + i * kPlane + o) = p[i];
  }
  __syncthreads();
  // W's rows past E lie past the resource and read zeros.
  const __amdgpu_buffer_rsrc_t w_rsrc = __builtin_amdgcn_make_buffer_rsrc(
      (void*)W, 0, E * D * 4, 0x00020000);
  // dx's rows of this workgroup (rows past T: neither read nor written).
  const __amdgpu_buffer_rsrc_t d_rsrc = __builtin_amdgcn_make_buffer_rsrc(
      dx + t0 * D, 0, static_cast<int>(min(static_cast<int64_t>(MT), T - t0)) * D * 4,
      0x00020000);
  float wf[NK][8];
  auto fetch = [&](int ks, int c0) {
    unsigned voff = c0 < c_end ? ((16 * ks + 8 * half) * D + c0 + l31) * 4 : kOutOfRange;
    asm volatile("" : "+v"(voff));  // (kept in one register, not one per row and step)
#pragma unroll
    for (int j = 0; j < 8; ++j)
      wf[ks][j] = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(
                                                w_rsrc, static_cast<int>(voff + j * D * 4), 0, 0));
  };
#pragma unroll
  for (int ks = 0; ks < NK; ++ks) fetch(ks, c_begin + 32 * wave);
  for (int c0 = c_begin + 32 * wave; c0 < c_end; c0 += 32 * NW) {
    f32x16 acc[NM];
#pragma unroll
    for (int m = 0; m < NM; ++m)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[m][r] = 0.f;
#pragma unroll
    for (int ks = 0; ks < NK; ++ks) {
      uint4 b[3];
      split8(wf[ks], b);
      fetch(ks, c0 + 32 * NW);
      constexpr int kA[6] = {2, 0, 1, 1, 0, 0}, kB[6] = {0, 2, 1, 0, 1, 0};
#pragma unroll
      for (int m0 = 0; m0 < NM; m0 += 2) {
        uint4 a[2][3];
#pragma unroll
        for (int m = 0; m < 2; ++m) {
          const int r = 32 * (m0 + m) + l31, c = 2 * ks + half;
          const int o = (c >> 3) * (MT * 128) + r * 128 +
                        (((c & 7) ^ (r & 7) ^ ((r >> 3) & 1)) << 4);
#pragma unroll
          for (int i = 0; i < 3; ++i)
            a[m][i] = *reinterpret_cast<const uint4*>(smem + i * kPlane + o);
        }
#pragma unroll
        for (int i = 0; i < 6; ++i)
#pragma unroll
          for (int m = 0; m < 2; ++m) acc[m0 + m] = mma32(a[m][kA[i]], b[kB[i]], acc[m0 + m]);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    int at = 0;
#pragma unroll
    for (int m = 0; m < NM; ++m)
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        if (r % 4 == 0) {
          at = ((32 * m + 8 * (r / 4) + 4 * half) * D + c0 + l31) * 4;
          asm volatile("" : "+v"(at));
        }
        const int o = at + (r % 4) * D * 4;
        float v = acc[m][r];
        if (accumulate)
          v += __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(d_rsrc, o, 0, 0));
        __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(v), d_rsrc, o, 0, 0);
      }
  }
}

// dx for more experts than LDS holds: waves over 64 tokens, 32 columns each,
// whose sums stay in registers over all experts: dz comes in chunks of 128
// experts, split into one of two LDS slots while the other is used, W a chunk
// ahead as above. (With a pass over dx for each 256 experts, added up in
// memory: T = 16384, E = 512, D = 2048 324 us against 212, 4096 x 384 x 7168 280
// against 145.)
constexpr int kManyMT = 64, kManyKC = 128;
template <int THREADS>
__global__ __launch_bounds__(THREADS, 1) void router_dx_many_kernel(
    const float* __restrict__ dz, const float* __restrict__ W, float* __restrict__ dx, int T,
    int E, int D, int col_tiles, int accumulate) {
  constexpr int MT = kManyMT, KC = kManyKC, NM = MT / 32, NK = KC / 16;
  constexpr int kPlane = MT * KC * 2, kItems = MT * (KC / 8) / THREADS;
  __shared__ __attribute__((aligned(16))) unsigned char smem[2 * 3 * kPlane];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int64_t t0 = static_cast<int64_t>(blockIdx.x / col_tiles) * MT;
  const int col = static_cast<int>(blockIdx.x % col_tiles) * (THREADS / 2) + 32 * wave + (lane & 31);
  const int half = lane >> 5, l31 = lane & 31;
  const int rows = static_cast<int>(min(static_cast<int64_t>(MT), T - t0));
  const __amdgpu_buffer_rsrc_t z_rsrc =
      __builtin_amdgcn_make_buffer_rsrc((void*)(dz + t0 * E), 0, rows * E * 4, 0x00020000);
  const __amdgpu_buffer_rsrc_t d_rsrc =
      __builtin_amdgcn_make_buffer_rsrc(dx + t0 * D, 0, rows * D * 4, 0x00020000);
  const __amdgpu_buffer_rsrc_t w_rsrc =
      __builtin_amdgcn_make_buffer_rsrc((void*)W, 0, E * D * 4, 0x00020000);
  float z[kItems][8];
  auto load = [&](int e0) {
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
      const int q = tid + THREADS * i, r = q / (KC / 8), e = e0 + 8 * (q % (KC / 8));
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const f32x4 v = __builtin_bit_cast(
            f32x4, __builtin_amdgcn_raw_buffer_load_b128(z_rsrc, (r * E + e) * 4 + 16 * h, 0, 0));
#pragma unroll
        for (int j = 0; j < 4; ++j) z[i][4 * h + j] = e + 4 * h + j < E ? v[j] : 0.f;
      }
    }
  };
  auto put = [&](int slot) {
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
      const int q = tid + THREADS * i, r = q / (KC / 8), c = q % (KC / 8);
      uint4 p[3];
      split8(z[i], p);
      const int o = (c >> 3) * (MT * 128) + r * 128 +
                    (((c & 7) ^ (r & 7) ^ ((r >> 3) & 1)) << 4);
#pragma unroll
      for (int j = 0; j < 3; ++j)
        *reinterpret_cast<uint4*>(smem + (3 * slot + j) * kPlane + o) = p[j];
    }
  };
  float wf[NK][8];
  auto fetch = [&](int ks, int e0) {
    unsigned voff = col < D ? ((e0 + 16 * ks + 8 * half) * D + col) * 4 : kOutOfRange;
    asm volatile("" : "+v"(voff));
#pragma unroll
    for (int j = 0; j < 8; ++j)  // (rows past E: zeros)
      wf[ks][j] = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(
                                                w_rsrc, static_cast<int>(voff + j * D * 4), 0, 0));
  };
  f32x16 acc[NM];
#pragma unroll
  for (int m = 0; m < NM; ++m)
#pragma unroll
    for (int r = 0; r < 16; ++r) acc[m][r] = 0.f;
  load(0);
#pragma unroll
  for (int ks = 0; ks < NK; ++ks) fetch(ks, 0);
  put(0);
  int slot = 0;
  for (int e0 = 0; e0 < E; e0 += KC, slot ^= 1) {
    __syncthreads();
    const bool more = e0 + KC < E;
    if (more) load(e0 + KC);
#pragma unroll
    for (int ks = 0; ks < NK; ++ks) {
      uint4 b[3], a[NM][3];
      split8(wf[ks], b);
      fetch(ks, e0 + KC);  // (past E behind the last chunk)
#pragma unroll
      for (int m = 0; m < NM; ++m) {
        const int r = 32 * m + l31, c = 2 * ks + half;
        const int o = (c >> 3) * (MT * 128) + r * 128 +
                      (((c & 7) ^ (r & 7) ^ ((r >> 3) & 1)) << 4);
#pragma unroll
        for (int i = 0; i < 3; ++i)
          a[m][i] = *reinterpret_cast<const uint4*>(smem + (3 * slot + i) * kPlane + o);
      }
      constexpr int kA[6] = {2, 0, 1, 1, 0, 0}, kB[6] = {0, 2, 1, 0, 1, 0};
#pragma unroll
      for (int i = 0; i < 6; ++i)
#pragma unroll
        for (int m = 0; m < NM; ++m) acc[m] = mma32(a[m][kA[i]], b[kB[i]], acc[m]);
      __builtin_amdgcn_sched_barrier(0);
    }
    if (more) put(slot ^ 1);
  }
#pragma unroll
  for (int m = 0; m < NM; ++m)
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      const int at = col < D ? ((32 * m + 8 * (r / 4) + 4 * half + r % 4) * D + col) * 4
                             : static_cast<int>(kOutOfRange);
      float v = acc[m][r];
      if (accumulate)
        v += __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(d_rsrc, at, 0, 0));
      __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(v), d_rsrc, at, 0, 0);
    }
}

// dW: a workgroup takes up to ME experts, 128 columns and a part of the
// tokens, in steps of 32 tokens: dz and x go through registers (the next
// step's loads run beside this step's products) into LDS rows [token][...],
// dz in its parts, and are read transposed. ME = 128: a 2 x 2 layout of waves
// of 64 experts x 64 columns, each part its own 256-byte rows; ME = 32: every
// wave all experts x 32 columns, the parts side by side in one row.
// T = 16384, E = 128, D = 2048, bf16 x: 36 to 40 us (its products 21 at the rate
// of a large bf16 product; 32 parts of dW are written) and 7 to add the parts
// up; fp32 x 60.
template <typename TX, int ME>
struct DwShape {
  static constexpr bool kF32 = sizeof(TX) == 4;
  static constexpr int BQ = 128, BK = 32, ROW = 256;
  static constexpr int NPB = kF32 ? 3 : 1;                  // parts of x
  static constexpr int NRA = ME == 128 ? 3 : 1;             // row blocks of dz
  static constexpr int MP = ME == 128 ? 2 : 1, MQ = ME == 128 ? 2 : 1;
  static constexpr int SLOT = (NRA + NPB) * BK * ROW;
  static constexpr int SLOTS = kF32 && ME == 128 ? 1 : 2;   // two workgroups a CU
};
__device__ __forceinline__ int t_off(int k, int col) {
  return k * 256 + (((col >> 3) ^ ((k & 3) << 2)) << 4) + ((col & 7) << 1);
}

template <typename TX, int ME>
__global__ __launch_bounds__(kThreads, 2) void router_dw_kernel(
    const float* __restrict__ dz, const TX* __restrict__ x, float* __restrict__ C, int T, int E,
    int D, int parts) {
  using S = DwShape<TX, ME>;
  __shared__ __attribute__((aligned(1024))) unsigned char smem[S::SLOTS * S::SLOT];
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
  const int nt = (D + S::BQ - 1) / S::BQ;
  const int m0 = static_cast<int>(blockIdx.x / nt) * ME, n0 = static_cast<int>(blockIdx.x % nt) * S::BQ;
  const int64_t k0 = static_cast<int64_t>(T) * blockIdx.y / parts;
  const int64_t k1 = static_cast<int64_t>(T) * (blockIdx.y + 1) / parts;
  C += static_cast<int64_t>(blockIdx.y) * E * D;
  // dz: thread -> token tid / 8, ME / 8 adjacent experts; x: token tid / 16
  // (and + 16), 8 adjacent columns.
  constexpr int NE = ME / 8;
  struct Step {
    float z[NE], x[S::kF32 ? 16 : 1];
    uint4 u[2];
  };
  const int zt = tid >> 3, ze = (tid & 7) * NE, xt = tid >> 4, xc = (tid & 15) * 8;
  // (Tokens past the part read zeros; experts past E and columns past D read
  // what follows in memory: their sums are not stored.)
  auto fetch = [&](int64_t kb, Step& st) {
    const int n = static_cast<int>(min(static_cast<int64_t>(S::BK), k1 - kb));
    const __amdgpu_buffer_rsrc_t zr = __builtin_amdgcn_make_buffer_rsrc(
        (void*)(dz + kb * E), 0, n * E * 4, 0x00020000);
    const __amdgpu_buffer_rsrc_t xr = __builtin_amdgcn_make_buffer_rsrc(
        (void*)(x + kb * D), 0, n * D * static_cast<int>(sizeof(TX)), 0x00020000);
    const int z_at = (zt * E + m0 + ze) * 4;
#pragma unroll
    for (int j = 0; j < NE; j += 4) {
      const f32x4 v = __builtin_bit_cast(
          f32x4, __builtin_amdgcn_raw_buffer_load_b128(zr, z_at + 4 * j, 0, 0));
#pragma unroll
      for (int i = 0; i < 4; ++i) st.z[j + i] = v[i];
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int x_at = ((xt + 16 * i) * D + n0 + xc) * static_cast<int>(sizeof(TX));
      const u32x4 lo = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(xr, x_at, 0, 0));
      if constexpr (S::kF32) {
        const u32x4 hi = __builtin_bit_cast(
            u32x4, __builtin_amdgcn_raw_buffer_load_b128(xr, x_at + 16, 0, 0));
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          st.x[8 * i + j] = __uint_as_float(lo[j]);
          st.x[8 * i + 4 + j] = __uint_as_float(hi[j]);
        }
      } else {
        st.u[i] = make_uint4(lo[0], lo[1], lo[2], lo[3]);
      }
    }
  };
  auto put = [&](int slot, const Step& st) {
    const auto& fz = st.z;
    const auto& fx = st.x;
    const auto& ux = st.u;
    unsigned char* base = smem + slot * S::SLOT;
    if constexpr (ME == 128) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float f[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = fz[8 * h + j];
        uint4 p[3];
        split8(f, p);
#pragma unroll
        for (int i = 0; i < 3; ++i)
          *reinterpret_cast<uint4*>(base + i * S::BK * S::ROW + t_off(zt, ze + 8 * h)) = p[i];
      }
    } else {
      uint32_t w[3][2];
#pragma unroll
      for (int j = 0; j < 2; ++j) split2(fz[2 * j], fz[2 * j + 1], w[0][j], w[1][j], w[2][j]);
#pragma unroll
      for (int i = 0; i < 3; ++i)
        *reinterpret_cast<uint2*>(base + t_off(zt, 32 * i + ze)) = make_uint2(w[i][0], w[i][1]);
    }
    base += S::NRA * S::BK * S::ROW;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int o = t_off(xt + 16 * i, xc);
      if constexpr (S::kF32) {
        float f[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = fx[8 * i + j];
        uint4 p[3];
        split8(f, p);
#pragma unroll
        for (int q = 0; q < 3; ++q)
          *reinterpret_cast<uint4*>(base + q * S::BK * S::ROW + o) = p[q];
      } else {
        *reinterpret_cast<uint4*>(base + o) = ux[i];
      }
    }
  };
  // Transposed fragment of the 32 columns from col of 16 rows (tokens): lane l
  // gets tokens 8 (l / 32) .. + 7 of column col + l % 32.
  const int grp = lane >> 4, j16 = lane & 15;
  auto frag = [&](const unsigned char* rows, int col) {
    const lds_u8* p = (const lds_u8*)rows + t_off(8 * (grp >> 1) + (j16 >> 2),
                                                  col + 16 * (grp & 1) + 4 * (j16 & 3));
    const uint2 lo = __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)p));
    const uint2 hi = __builtin_bit_cast(
        uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(p + 4 * S::ROW)));
    return make_uint4(lo.x, lo.y, hi.x, hi.y);
  };
  const int wm = ME == 128 ? 64 * (wave >> 1) : 0;
  const int wn = ME == 128 ? 64 * (wave & 1) : 32 * wave;
  f32x16 acc[S::MP][S::MQ];
#pragma unroll
  for (int i = 0; i < S::MP; ++i)
#pragma unroll
    for (int j = 0; j < S::MQ; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;
  // Steps are fetched two ahead: step i's registers are free once it is in LDS.
  const int64_t steps = (k1 - k0 + S::BK - 1) / S::BK;
  Step st[2];
  if (steps > 0) fetch(k0, st[0]);
  if (steps > 1) fetch(k0 + S::BK, st[1]);
  if (steps > 0) put(0, st[0]);
  if (steps > 2) fetch(k0 + 2 * S::BK, st[0]);
  auto products = [&](int slot) {
    const unsigned char* za = smem + slot * S::SLOT;
    const unsigned char* xb = za + S::NRA * S::BK * S::ROW;
#pragma unroll
    for (int kk = 0; kk < S::BK; kk += 16) {
      uint4 fa[S::MP][3], fb[S::MQ][S::NPB];
#pragma unroll
      for (int i = 0; i < S::MP; ++i)
#pragma unroll
        for (int q = 0; q < 3; ++q)
          fa[i][q] = ME == 128 ? frag(za + q * S::BK * S::ROW + kk * S::ROW, wm + 32 * i)
                               : frag(za + kk * S::ROW, 32 * q);
#pragma unroll
      for (int j = 0; j < S::MQ; ++j)
#pragma unroll
        for (int q = 0; q < S::NPB; ++q)
          fb[j][q] = frag(xb + q * S::BK * S::ROW + kk * S::ROW, wn + 32 * j);
#pragma unroll
      for (int i = 0; i < S::MP; ++i)
#pragma unroll
        for (int j = 0; j < S::MQ; ++j) {
          if constexpr (S::kF32) {
            acc[i][j] = mma_parts(fa[i], fb[j], acc[i][j]);
          } else {
#pragma unroll
            for (int q = 2; q >= 0; --q) acc[i][j] = mma32(fa[i][q], fb[j][0], acc[i][j]);
          }
        }
    }
  };
  // Step i from slot i % 2, step i + 1 put beside it (or, with one slot, in its
  // place behind a second barrier); nxt holds step i + 1.
  auto step = [&](int64_t i, Step& nxt) {
    __syncthreads();
    products(S::SLOTS == 2 ? static_cast<int>(i & 1) : 0);
    if (i + 1 < steps) {
      if (S::SLOTS == 1) __syncthreads();
      put(S::SLOTS == 2 ? static_cast<int>((i + 1) & 1) : 0, nxt);
      if (i + 3 < steps) fetch(k0 + (i + 3) * S::BK, nxt);
    }
  };
  for (int64_t i = 0; i < steps; i += 2) {
    step(i, st[1]);
    if (i + 1 < steps) step(i + 1, st[0]);
  }
#pragma unroll
  for (int i = 0; i < S::MP; ++i)
#pragma unroll
    for (int j = 0; j < S::MQ; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const int e = m0 + wm + 32 * i + 8 * (r / 4) + 4 * (lane >> 5) + r % 4;
        const int c = n0 + wn + 32 * j + (lane & 31);
        if (e < E && c < D) C[static_cast<int64_t>(e) * D + c] = acc[i][j][r];
      }
}

// The parts of dW added up: 64 float4 of it a workgroup, wave w the parts w,
// w + 4, ... in order with eight loads in flight, then the waves in order.
__global__ __launch_bounds__(kThreads) void router_dense_sum_kernel(const float4* __restrict__ part,
                                                                    float4* __restrict__ out,
                                                                    int64_t n4, int parts) {
  __shared__ float4 s_sum[kThreads];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 64 + lane;
  float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
  auto add = [](float4& a, const float4& b) {
    a.x += b.x;
    a.y += b.y;
    a.z += b.z;
    a.w += b.w;
  };
  if (i < n4)
    for (int p0 = wave; p0 < parts; p0 += 32) {
      float4 w[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) w[j] = part[min(p0 + 4 * j, parts - 1) * n4 + i];
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (p0 + 4 * j < parts) add(v, w[j]);
    }
  s_sum[threadIdx.x] = v;
  __syncthreads();
  if (wave == 0 && i < n4) {
#pragma unroll
    for (int w = 1; w < 4; ++w) add(v, s_sum[64 * w + lane]);
    out[i] = v;
  }
}

// Workgroups of the forward: some 8 K logits each, at most kMaxParts.
int balance_parts(int T, int E) {
  const int64_t n = (static_cast<int64_t>(T) * E + 8191) / 8192;
  return static_cast<int>(std::min<int64_t>(std::max<int64_t>(n, 1), kMaxParts));
}

// Experts of a dW tile, and the parts its tokens are cut into: two workgroups
// for every CU, at least 64 tokens each (two steps). Few tokens stay in one part,
// which needs no launch to add parts up (in parts against in one: 128 tokens, 8
// experts, D = 128, 8.9 : 6.3 us, 256 8.5 : 7.9; 256 x 256 x 4096 18.7 : 11.8, but
// 200 x 64 x 1024 11.5 : 15.1, and 512 x 8 x 128 8.7 : 13.7). Over 64 to 800
// tokens and ten sizes of E x D the two are level near 285 tokens of fp32 x and
// 580 of bf16 x with up to 32 experts, near 115 to 225 with 64 or 128 in few
// tiles, near 740 with 64 tiles or more. (With 64 tiles the rule changes too
// early: 320 x 256 x 7168 26.2 : 14.1.)
int dw_experts(int E) { return E <= 32 ? 32 : 128; }
int dense_parts(int T, int E, int D) {
  const int me = dw_experts(E);
  const int64_t tiles = static_cast<int64_t>((E + me - 1) / me) * ((D + 127) / 128);
  if (T <= 128 || (T <= 256 && (me == 32 || tiles >= 64))) return 1;
  const int64_t want = std::max<int64_t>(1, 512 / tiles);
  return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(want, T / 64)));
}

// f(lanes per token, registers per lane) for E experts.
template <typename F>
hipError_t for_experts(int E, F f) {
  using std::integral_constant;
  if (E <= 8) return f(integral_constant<int, 4>{}, integral_constant<int, 2>{});
  if (E <= 16) return f(integral_constant<int, 4>{}, integral_constant<int, 4>{});
  if (E <= 32) return f(integral_constant<int, 8>{}, integral_constant<int, 4>{});
  if (E <= 64) return f(integral_constant<int, 16>{}, integral_constant<int, 4>{});
  if (E <= 128) return f(integral_constant<int, 16>{}, integral_constant<int, 8>{});
  if (E <= 256) return f(integral_constant<int, 32>{}, integral_constant<int, 8>{});
  if (E <= 512) return f(integral_constant<int, 64>{}, integral_constant<int, 8>{});
  return f(integral_constant<int, 64>{}, integral_constant<int, 16>{});
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
        <<<parts, kLossThreads, 0, s>>>(Tn, E, k, logits, topk, mask, coef, parts, p_prob, p_count,
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
  if (dx != nullptr && T > 0) {
    auto launch = [&](auto kc, auto tokens, auto threads) {
      constexpr int MT = decltype(tokens)::value, NT = decltype(threads)::value;
      const int64_t mt = (static_cast<int64_t>(T) + MT - 1) / MT;
      // Columns of a workgroup: all, or fewer until there are some 2^15 / MT.
      const int64_t want = std::max<int64_t>(1, (1 << 15) / MT / mt);
      const int step = NT / 2;  // 32 columns a wave
      const int cols = static_cast<int>((D + step * want - 1) / (step * want) * step);
      const int ct = (D + cols - 1) / cols;
      router_dx_kernel<decltype(kc)::value, MT, NT><<<static_cast<unsigned>(mt * ct), NT, 0, s>>>(
          dlogits, w, dx, T, E, D, cols, ct, accumulate);
    };
    using std::integral_constant;
    if (E <= 16)
      launch(integral_constant<int, 16>{}, integral_constant<int, 128>{},
             integral_constant<int, 512>{});
    else if (E <= 64)
      launch(integral_constant<int, 64>{}, integral_constant<int, 128>{},
             integral_constant<int, 512>{});
    else if (E <= 128)
      launch(integral_constant<int, 128>{}, integral_constant<int, 128>{},
             integral_constant<int, 512>{});
    else if (E <= 256)
      launch(integral_constant<int, 256>{}, integral_constant<int, 64>{},
             integral_constant<int, 256>{});
    else {
      const int64_t mt = (static_cast<int64_t>(T) + kManyMT - 1) / kManyMT;
      // 256 columns a workgroup, 128 where that leaves CUs idle.
      auto many = [&](auto threads) {
        constexpr int NT = decltype(threads)::value;
        const int ct = (D + NT / 2 - 1) / (NT / 2);
        router_dx_many_kernel<NT><<<static_cast<unsigned>(mt * ct), NT, 0, s>>>(
            dlogits, w, dx, T, E, D, ct, accumulate);
      };
      if (mt * ((D + 255) / 256) >= 256)
        many(integral_constant<int, 512>{});
      else
        many(integral_constant<int, 256>{});
    }
    e = hipGetLastError();
  }
  if (e == hipSuccess && dw != nullptr) {
    const int parts = T > 0 ? dense_parts(T, E, D) : 1, me = dw_experts(E);
    const dim3 grid(static_cast<unsigned>((E + me - 1) / me * ((D + 127) / 128)),
                    static_cast<unsigned>(parts));
    auto* k = me == 32 ? router_dw_kernel<TX, 32> : router_dw_kernel<TX, 128>;
    k<<<grid, kThreads, 0, s>>>(dlogits, x, parts > 1 ? ws : dw, T, E, D, parts);
    e = hipGetLastError();
    if (e == hipSuccess && parts > 1) {
      const int64_t n4 = static_cast<int64_t>(E) * D / 4;
      router_dense_sum_kernel<<<static_cast<unsigned>((n4 + 63) / 64), kThreads, 0, s>>>(
          reinterpret_cast<const float4*>(ws), reinterpret_cast<float4*>(dw), n4, parts);
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

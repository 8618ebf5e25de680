// Grouped expert products in FP8 with block scales (formats in moe_fp8.h), on
// gfx950's 16x16x128 FP8 matrix instruction.
//
//   y[r, c] = sum_b xs[b, r] ws[c / 128, b] sum_{k in block b} xq[r, k] wq[c, k]
// and, gated, h = SiLU(y_gate) y_up.
//
// One matrix instruction sums exactly one block of 128: it starts from zero,
// and its 16 x 16 sums are added to the fp32 accumulators with one FMA each,
// scaled by xs ws. The weights are the instruction's first operand: a lane
// then holds four output columns of one row, so xs is one value per lane and
// row block, ws one scalar per 64 columns, and a scale costs no more than its
// FMA. The FMAs (4 per instruction, 16 cycles of vector issue) run beside the
// matrix core's 32 cycles (a loop of both alone loses 2 % to a loop without
// the FMAs): a wave issues an instruction's FMAs three instructions later, and
// two waves share a SIMD.
#include <algorithm>
#include <type_traits>

#include "ckpt.h"
#include "moe_internal.h"

namespace moe {
namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) unsigned char lds_u8;

constexpr int kXcds = 8;
constexpr int kMaxTableExperts = MOE_MAX_EXPERTS;
constexpr int kOutOfRange = 0x40000000;  // a load offset past every buffer (all < 2^30)

enum OutKind { kOutF32 = 0, kOutF16 = 1, kOutBf16 = 2 };

#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
// 16 (4) bytes a lane global -> LDS at lds_base + 16 (4) * lane; offsets past
// the resource write zeros. Counted by vmcnt. (s_nop: a copy needs one wait
// state behind a write of M0, and five behind the v_readfirstlane that makes a
// resource's register, which nobody adds to assembly; four states more were
// 0.3 to 1.9 % slower, so that these cost about 1 %.)
__device__ __forceinline__ void dma16(__amdgpu_buffer_rsrc_t rsrc, int voff, int soff,
                                      unsigned lds_base) {
  asm volatile("s_mov_b32 m0, %3\n\ts_nop 3\n\tbuffer_load_dwordx4 %0, %1, %2 offen lds"
               :: "v"(voff), "s"(rsrc), "s"(soff), "s"(lds_base) : "memory", "m0");
}
__device__ __forceinline__ void dma4(__amdgpu_buffer_rsrc_t rsrc, int voff, int soff,
                                     unsigned lds_base) {
  asm volatile("s_mov_b32 m0, %3\n\ts_nop 3\n\tbuffer_load_dword %0, %1, %2 offen lds"
               :: "v"(voff), "s"(rsrc), "s"(soff), "s"(lds_base) : "memory", "m0");
}
#pragma clang diagnostic pop

__device__ __forceinline__ uint32_t f16_sat_bits(float f) {
  const float c = f > 65504.f ? 65504.f : (f < -65504.f ? -65504.f : f);
  return __builtin_bit_cast(unsigned short, static_cast<_Float16>(c));
}

// (SiLU first: of a large negative g it is 0, where g u may be infinite.)
__device__ __forceinline__ float silu_mul(float g, float u) {
  return g * __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-1.4426950408889634f * g)) * u;
}

__device__ __forceinline__ f32x4 mma(const i32x8& w, const i32x8& x) {
  const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, x, zero, 0, 0, 0, 0, 0, 0);
}

// LDS rows hold 128 codes; 16-byte chunk c of a row sits at c ^ swz(i), i the
// row's place in its 16-row fragment: the eight rows of every group of lanes
// that a 16-byte read serves together then cover all banks.
__device__ __forceinline__ int swz(int i) { return (i & 7) ^ ((i >> 3) & 1); }
// Fragment b (0 .. 3) of a 64-column group takes, in place i (0 .. 15), column
// of_place(i) + of_frag(b): lane group g of its results holds places 4 g ..
// 4 g + 3. A lane then has 16 bytes of adjacent outputs at a time, the four
// lanes of a row 64: 16-bit outputs 8 g .. 8 g + 7 of each half of the group,
// from two fragments, fp32 ones 4 g .. 4 g + 3 of each quarter. (With 16 adjacent
// columns a lane, stores of 16 bytes 64 apart: fp32 outputs of 32768 rows,
// 2048 -> 7168, 802 us against 687; with fp16 ones, 32 apart, 543 against 539.)
template <int KIND>
struct Cols {
  static constexpr int kRun = KIND == kOutF32 ? 4 : 8;  // adjacent columns of a lane
  // column of place i in fragment 0, and what fragment b adds
  static __device__ __forceinline__ int of_place(int i) {
    return kRun * (i >> 2) + (i & 3);
  }
  static constexpr int of_frag(int b) {
    return KIND == kOutF32 ? 16 * b : 4 * (b & 1) + 32 * (b >> 1);
  }
  // the place of column j
  static __device__ __forceinline__ int place(int j) {
    return KIND == kOutF32 ? j & 15 : (j & 3) | ((j >> 1) & 12);
  }
};

// 16 bytes of adjacent outputs of a row.
template <int KIND>
__device__ __forceinline__ void store_run(void* out, int64_t o, const float (&v)[Cols<KIND>::kRun]) {
  if constexpr (KIND == kOutF32) {
    *reinterpret_cast<float4*>(static_cast<float*>(out) + o) = make_float4(v[0], v[1], v[2], v[3]);
  } else {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      w[i] = KIND == kOutF16
                 ? f16_sat_bits(v[2 * i]) | (f16_sat_bits(v[2 * i + 1]) << 16)
                 : cvt_bf16x2(v[2 * i], v[2 * i + 1]);
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(out) + o) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// Four adjacent outputs of a row.
template <int KIND>
__device__ __forceinline__ void store4(void* out, int64_t o, const f32x4& v) {
  if (KIND == kOutF32)
    *reinterpret_cast<f32x4*>(static_cast<float*>(out) + o) = v;
  else if (KIND == kOutF16)
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(out) + o) =
        make_uint2(f16_sat_bits(v[0]) | (f16_sat_bits(v[1]) << 16),
                   f16_sat_bits(v[2]) | (f16_sat_bits(v[3]) << 16));
  else
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(out) + o) =
        make_uint2(cvt_bf16x2(v[0], v[1]), cvt_bf16x2(v[2], v[3]));
}

// Tiles before each expert (s_pref) and first rows (s_off, clamped to
// cap_rows), by wave 0.
__device__ __forceinline__ void tile_table(const int32_t* __restrict__ offsets, int n_exp,
                                           int64_t cap_rows, int bm, int nt, int lane,
                                           int* s_pref, int* s_off) {
  int base = 0;
  for (int e0 = 0; e0 < n_exp; e0 += 64) {
    const int e = e0 + lane;
    int beg = 0, end = 0;
    if (e < n_exp) {
      if (offsets) {
        beg = offsets[e];
        end = offsets[e + 1];
      } else {
        end = static_cast<int>(cap_rows);
      }
      beg = static_cast<int>(min(max(static_cast<int64_t>(beg), int64_t(0)), cap_rows));
      end = static_cast<int>(
          min(max(static_cast<int64_t>(end), static_cast<int64_t>(beg)), cap_rows));
    }
    const int tiles = (end - beg + bm - 1) / bm * nt;
    int incl = tiles;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
      const int y = __shfl_up(incl, off, 64);
      if (lane >= off) incl += y;
    }
    if (e < n_exp) {
      s_pref[e] = base + incl - tiles;
      s_off[e] = beg;
      if (e == n_exp - 1) {
        s_pref[n_exp] = base + incl;
        s_off[n_exp] = end;
      }
    }
    base += __shfl(incl, 63, 64);
  }
}

// The expert of tile t: the last one whose tiles begin at or before t.
__device__ __forceinline__ int find_expert(const int* s_pref, int n_exp, int t, int lane) {
  int expert = 0;
  for (int e0 = 1; e0 <= n_exp; e0 += 64) {
    const int idx = e0 + lane;
    const bool le = idx <= n_exp && s_pref[idx] <= t;
    expert += __popcll(__ballot(le));
    if (__ballot(idx <= n_exp && !le)) break;
  }
  return __builtin_amdgcn_readfirstlane(expert);
}

// ---------------------------------------------------------------------------
// Large tiles: up to 256 rows x 256 product columns (gated: 128 gate and the
// matching 128 up columns), eight waves, wave (wr, wc) a quarter of the rows
// x 128 columns: 128 accumulators a lane. Both operands of a K step (one
// block of 128) are copied to LDS one step ahead (2 x 64 KB), with the rows'
// 256 scales; the LDS holds no third slot. One workgroup per CU works through
// its share of the tile list, which is dealt to the XCDs in contiguous runs.
// Mixtral-style gate_up (16384 rows, 4096 x 28672): 1.74 to 1.89 ms from card
// to card (their clocks differ), 2.04 to 2.21 PFLOP/s, against 2.66 to 2.77
// that a library's plain FP8 product of 8192^3 reaches and 3.7 of a loop of the
// instruction alone (random operands: the clock falls to 2.0 GHz). A step takes
// 1.9 us, 1.1 of them matrix instructions; a step's first fragments read behind
// the products of the step before (4 % faster to 3 % slower, by shape and card)
// and lines touched two steps ahead (2 to 6 % slower) did not shorten the rest.
// ---------------------------------------------------------------------------
constexpr int kThreads = 512;
constexpr int BM = 256, BN = 256, BK = 128;
constexpr int kTile = BM * BK;           // bytes of one operand's slot
constexpr int kOffW = 2 * kTile, kOffS = 4 * kTile;
constexpr int kLds = kOffS + 2 * BM * 4;

template <bool GATED, int KIND>
__global__ __launch_bounds__(kThreads, 1) void fp8_gemm_kernel(
    const uint8_t* __restrict__ Xq, const float* __restrict__ Xs,
    const int32_t* __restrict__ offsets, int n_experts, int64_t cap_rows,
    const uint8_t* __restrict__ Wq, const float* __restrict__ Ws, void* __restrict__ out, int K,
    int N) {
  constexpr int BN_OUT = GATED ? BN / 2 : BN;
  static_assert(kLds + 2 * (kMaxTableExperts + 1) * 4 <= 160 * 1024, "LDS budget");
  __shared__ __attribute__((aligned(1024))) unsigned char smem[kLds];
  __shared__ int s_tab[2 * (kMaxTableExperts + 1)];
  int* s_pref = s_tab;
  int* s_off = s_tab + kMaxTableExperts + 1;

  const int tid = threadIdx.x;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int n_exp = offsets ? n_experts : 1;
  const int nt = (N + BN_OUT - 1) / BN_OUT;
  const int ncols = GATED ? 2 * N : N;          // weight rows per expert
  const int nk = (K + BK - 1) / BK;             // K steps = scale blocks
  const int nnb = (ncols + 127) / 128;
  const bool k_tail = (K & 64) != 0;            // the last step holds 64 codes a row
  if (wave == 0) tile_table(offsets, n_exp, cap_rows, BM, nt, tid, s_pref, s_off);
  __syncthreads();
  const int R = __builtin_amdgcn_readfirstlane(s_pref[n_exp]);
  const int G8 = static_cast<int>(gridDim.x) / kXcds;
  const int xcd = static_cast<int>(blockIdx.x) % kXcds, slot = static_cast<int>(blockIdx.x) / kXcds;
  const int per = (R + kXcds - 1) / kXcds;
  const int run_end = min((xcd + 1) * per, R);
  int t = xcd * per + slot;
  if (t >= run_end) return;  // (the whole workgroup)
  const unsigned lds0 = (unsigned)(uintptr_t)(lds_u8*)smem;
  const int lane = tid & 63;
  const int wr = wave >> 1, wc = wave & 1;

  struct Tile {
    int expert, row, rows, n0;
  };
  auto decode = [&](int tile) {
    Tile d;
    d.expert = find_expert(s_pref, n_exp, tile, lane);
    const int seg_beg = __builtin_amdgcn_readfirstlane(s_off[d.expert]);
    const int seg_end = __builtin_amdgcn_readfirstlane(s_off[d.expert + 1]);
    const int local = tile - __builtin_amdgcn_readfirstlane(s_pref[d.expert]);
    const int mt = (seg_end - seg_beg + BM - 1) / BM;
    const int nb = local / mt, mb = local - nb * mt;
    d.row = seg_beg + mb * BM;  // full row blocks, then the rest
    d.rows = min(BM, seg_end - d.row);
    d.n0 = nb * BN_OUT;
    return d;
  };
  // Weight scales of the wave's two 64-column groups, 64 steps from kt on, one
  // a lane.
  auto load_ws = [&](const Tile& d, int kt, float (&v)[2]) {
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const int c = GATED ? q * N + d.n0 + 64 * wc : d.n0 + 128 * wc + 64 * q;
      v[q] = Ws[(static_cast<int64_t>(d.expert) * nnb + min(c / 128, nnb - 1)) * nk +
                min(kt + lane, nk - 1)];
    }
  };

  // Copies: wave w takes the 8-row groups w + 8 i of each operand (rows 64 i
  // further on for the next i; gated: up columns from i = 2); lane -> row
  // l / 8, LDS chunk l % 8. Rows past the tile's (weight rows past the
  // expert's) lie past the resources and read zeros, as does the half that a
  // short last block lacks (its offsets are out of range); a gate column past
  // N reads up columns, whose results are not stored.
  const int crow = 8 * wave + (lane >> 3);
  const int xc = (lane & 7) ^ swz(crow & 15), wk = (lane & 7) ^ swz(Cols<KIND>::place(crow));
  const int x_voff = crow * K + 16 * xc, w_voff = crow * K + 16 * wk;
  const int s_voff = 4 * (64 * (wave & 3) + lane);
  auto rsrc = [&](const void* base, int bytes) {
    const uint64_t a = reinterpret_cast<uint64_t>(base);
    const uint64_t lo = static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(static_cast<int>(a)));
    const uint64_t hi = static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(static_cast<int>(a >> 32)));
    return __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void*>(lo | hi << 32), 0,
                                             __builtin_amdgcn_readfirstlane(bytes), 0x00020000);
  };
  // Where the next step to be copied lies: its tile's operands, the step kc.
  struct Copy {
    const uint8_t *x, *w;
    const float* s;
    int x_bytes, w_bytes, s_bytes, kc;
  };
  auto copy_from = [&](const Tile& d, bool any) {
    Copy c;
    c.x = Xq + static_cast<int64_t>(d.row) * K;
    c.w = Wq + (static_cast<int64_t>(d.expert) * ncols + d.n0) * K;
    c.s = Xs + d.row;
    c.x_bytes = any ? d.rows * K : 0;
    c.w_bytes = any ? (ncols - d.n0) * K : 0;
    c.s_bytes = any ? d.rows * 4 : 0;
    c.kc = 0;
    return c;
  };
  auto copy_scales = [&](const Copy& c, int sl) {
    dma4(rsrc(c.s, c.s_bytes), s_voff, 0,
         lds0 + kOffS + sl * BM * 4 + (wave & 3) * 256);
  };
  // Copy i: 0 .. 3 weights, 4 .. 7 activations, into slot sl.
  auto copy = [&](const Copy& c, int i, int sl) {
    const bool cut = k_tail && c.kc == nk - 1;
    if (i < 4)
      dma16(rsrc(c.w, c.w_bytes),
            (cut && wk >= 4 ? kOutOfRange : w_voff + c.kc * BK) +
                (GATED && i >= 2 ? N + 64 * (i - 2) : 64 * i) * K,
            0, lds0 + kOffW + sl * kTile + (wave + 8 * i) * 1024);
    else
      dma16(rsrc(c.x, c.x_bytes),
            (cut && xc >= 4 ? kOutOfRange : x_voff + c.kc * BK) + 64 * (i - 4) * K, 0,
            lds0 + sl * kTile + (wave + 8 * (i - 4)) * 1024);
  };
  auto advance = [&](Copy& c) {
    c.s += cap_rows;
    ++c.kc;
  };

  // A tile's first step is copied during the last one of the tile before it,
  // so that the tiles follow one another without a gap: `first` is the slot of
  // the tile's step 0.
  Tile cur = decode(t);
  int first = 0;
  float ws_next[2];
  load_ws(cur, 0, ws_next);
  Copy c = copy_from(cur, true);
  {
    copy_scales(c, 0);
#pragma unroll
    for (int i = 0; i < 8; ++i) copy(c, i, 0);
    advance(c);
  }
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  while (true) {
    const bool has_next = t + G8 < run_end;
    const Tile next = has_next ? decode(t + G8) : cur;
    float wsv[2] = {ws_next[0], ws_next[1]};
    load_ws(next, 0, ws_next);

    auto run = [&](auto nxb_c) {
      constexpr int NX = decltype(nxb_c)::value;  // 16-row blocks per wave
      const int rowbase = wr * NX * 16;
      f32x4 acc[2][4][NX];
#pragma unroll
      for (int q = 0; q < 2; ++q)
#pragma unroll
        for (int b = 0; b < 4; ++b)
#pragma unroll
          for (int x = 0; x < NX; ++x) acc[q][b][x] = f32x4{0.f, 0.f, 0.f, 0.f};
      // LDS addresses of fragments: row (l % 16), chunks 2 (l / 16) and + 1
      // (the lanes that are served together then meet no bank twice; with
      // chunks l / 16 and 4 + l / 16 half of the LDS cycles were conflicts).
      int x_addr[2], w_addr[2];
      const int i16 = lane & 15, g = lane >> 4;
      {
        const int wrow = (GATED ? 64 * wc : 128 * wc) + Cols<KIND>::of_place(i16);
#pragma unroll
        for (int p = 0; p < 2; ++p) {
          x_addr[p] = (rowbase + i16) * 128 + (((2 * g + p) ^ swz(i16)) << 4);
          w_addr[p] = kOffW + wrow * 128 + (((2 * g + p) ^ swz(i16)) << 4);
        }
      }
      auto frag = [&](int base, const int(&a)[2]) {
        const int4 lo = *reinterpret_cast<const int4*>(smem + base + a[0]);
        const int4 hi = *reinterpret_cast<const int4*>(smem + base + a[1]);
        return i32x8{lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
      };
      for (int kt = 0; kt < nk; ++kt) {
        if (kt > 0 && (kt & 63) == 0) load_ws(cur, kt, wsv);
        // Every wave's copies of this step are done (each has waited for its
        // own), and every wave has read what the next copies overwrite.
        asm volatile("s_barrier" ::: "memory");
        const int slot_k = (first + kt) & 1, sl = slot_k * kTile;
        if (kt + 1 == nk) c = copy_from(next, has_next);
        i32x8 xf[NX], wf[2];
        float s[2][NX];
#pragma unroll
        for (int x = 0; x < NX; ++x) xf[x] = frag(sl + x * 16 * 128, x_addr);
        wf[0] = frag(sl, w_addr);
#pragma unroll
        for (int x = 0; x < NX; ++x) {
          const float sx = *reinterpret_cast<const float*>(
              smem + kOffS + slot_k * BM * 4 + (rowbase + 16 * x + i16) * 4);
#pragma unroll
          for (int q = 0; q < 2; ++q)
            s[q][x] = sx * __builtin_bit_cast(float, __builtin_amdgcn_readlane(
                                                         __builtin_bit_cast(int, wsv[q]), kt & 63));
        }
        copy_scales(c, slot_k ^ 1);
        constexpr int LAG = 3, M = 8 * NX;
        f32x4 part[LAG + 1];
#pragma unroll
        for (int m = 0; m < M + LAG; ++m) {
          if (m < M) {
            const int f = m / NX, x = m % NX;
            if (x == 0) {
              if (f + 1 < 8) {
                const int q = (f + 1) >> 2, b = (f + 1) & 3;
                wf[(f + 1) & 1] =
                    frag(sl + (q * (GATED ? 128 : 64) + Cols<KIND>::of_frag(b)) * 128, w_addr);
              }
              // The next step's copies early in this one, two at a time (all at
              // once hold up the reads; spread over the step they come late:
              // 5 to 20 % slower either way).
              if (f < 4) {
                copy(c, 2 * f, slot_k ^ 1);
                copy(c, 2 * f + 1, slot_k ^ 1);
              }
            }
            part[m % (LAG + 1)] = mma(wf[f & 1], xf[x]);
          }
          if (m >= LAG) {
            const int o = m - LAG, f = o / NX, x = o % NX;
#pragma unroll
            for (int r = 0; r < 4; ++r)
              acc[f >> 2][f & 3][x][r] = __builtin_fmaf(part[o % (LAG + 1)][r], s[f >> 2][x],
                                                        acc[f >> 2][f & 3][x][r]);
          }
          __builtin_amdgcn_sched_barrier(0);
        }
        advance(c);
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
      }
      // ---- epilogue: row l % 16 of each row block, columns as in Cols ----
#pragma unroll
      for (int x = 0; x < NX; ++x) {
        const int r = rowbase + 16 * x + i16;
        if (r < cur.rows) {
          const int64_t o = static_cast<int64_t>(cur.row + r) * N;
          constexpr int RUN = Cols<KIND>::kRun;
#pragma unroll
          for (int q = 0; q < (GATED ? 1 : 2); ++q) {
            const int c = cur.n0 + (GATED ? 64 : 128) * wc + 64 * q + RUN * g;
#pragma unroll
            for (int b = 0; b < 4; b += RUN / 4) {
              float v[RUN];
#pragma unroll
              for (int i = 0; i < RUN; ++i)
                v[i] = GATED ? silu_mul(acc[0][b + (i >> 2)][x][i & 3], acc[1][b + (i >> 2)][x][i & 3])
                             : acc[q][b + (i >> 2)][x][i & 3];
              if (c < N) store_run<KIND>(out, o + c + Cols<KIND>::of_frag(b), v);
            }
          }
        }
      }
    };
    const int nblk = (cur.rows + 15) / 16;
    switch ((nblk + 3) / 4) {
      case 4: run(std::integral_constant<int, 4>{}); break;
      case 3: run(std::integral_constant<int, 3>{}); break;
      case 2: run(std::integral_constant<int, 2>{}); break;
      default: run(std::integral_constant<int, 1>{}); break;
    }
    if (!has_next) break;
    first = (first + nk) & 1;
    cur = next;
    t += G8;
  }
}

// ---------------------------------------------------------------------------
// Few rows an expert (decoding): the time is that of reading the weights of
// the experts that are hit. A tile is up to 32 rows x 128 product columns
// (gated: 64 gate columns and the matching 64 up columns); the four waves of a
// workgroup cut K (wave w takes blocks w, w + 4, ...), load the weight and
// activation fragments straight into registers, a whole block (16 KB of
// weights) ahead of its use and without a barrier, and add their sums in LDS.
// Two workgroups a CU keep 128 KB in flight there. One new token on eight
// experts (7168 x 4096 codes each, 235 MB): 46 us, 5.1 TB/s, what a copy
// reaches; 78 us with the large tiles.
// ---------------------------------------------------------------------------
constexpr int kSmallThreads = 256, kWaves = kSmallThreads / 64;
constexpr int SM = 32, SN = 128;

template <bool GATED, int KIND>
__global__ __launch_bounds__(kSmallThreads, 2) void fp8_small_kernel(
    const uint8_t* __restrict__ Xq, const float* __restrict__ Xs,
    const int32_t* __restrict__ offsets, int n_experts, int64_t cap_rows,
    const uint8_t* __restrict__ Wq, const float* __restrict__ Ws, void* __restrict__ out, int K,
    int N) {
  constexpr int SN_OUT = GATED ? SN / 2 : SN;
  __shared__ f32x4 red[kWaves * 8 * (SM / 16) * 64];
  __shared__ int s_tab[2 * (kMaxTableExperts + 1)];
  int* s_pref = s_tab;
  int* s_off = s_tab + kMaxTableExperts + 1;
  const int tid = threadIdx.x;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
  const int n_exp = offsets ? n_experts : 1;
  const int nt = (N + SN_OUT - 1) / SN_OUT;
  const int ncols = GATED ? 2 * N : N;
  const int nk = (K + BK - 1) / BK;
  const int nnb = (ncols + 127) / 128;
  const bool k_tail = (K & 64) != 0;
  if (wave == 0) tile_table(offsets, n_exp, cap_rows, SM, nt, tid, s_pref, s_off);
  __syncthreads();
  const int R = __builtin_amdgcn_readfirstlane(s_pref[n_exp]);
  const int G8 = static_cast<int>(gridDim.x) / kXcds;
  const int xcd = static_cast<int>(blockIdx.x) % kXcds, slot = static_cast<int>(blockIdx.x) / kXcds;
  const int per = (R + kXcds - 1) / kXcds;
  const int run_end = min((xcd + 1) * per, R);
  for (int t = xcd * per + slot; t < run_end; t += G8) {
    const int expert = find_expert(s_pref, n_exp, t, lane);
    const int seg_beg = __builtin_amdgcn_readfirstlane(s_off[expert]);
    const int seg_end = __builtin_amdgcn_readfirstlane(s_off[expert + 1]);
    const int local = t - __builtin_amdgcn_readfirstlane(s_pref[expert]);
    const int cnt = seg_end - seg_beg;
    const int mt = (cnt + SM - 1) / SM;
    const int chunk = (cnt + mt - 1) / mt;
    const int nb = local / mt, mb = local - nb * mt;
    const int row_begin = seg_beg + mb * chunk;
    const int rows = min(chunk, seg_end - row_begin);  // <= SM
    if (rows <= 0) continue;  // (uniform)
    const int n0 = nb * SN_OUT;
    // Rows past the tile's lie past the resource and read zeros.
    const __amdgpu_buffer_rsrc_t x_rsrc = __builtin_amdgcn_make_buffer_rsrc(
        (void*)(Xq + static_cast<int64_t>(row_begin) * K), 0, rows * K, 0x00020000);
    const __amdgpu_buffer_rsrc_t w_rsrc = __builtin_amdgcn_make_buffer_rsrc(
        (void*)(Wq + static_cast<int64_t>(expert) * ncols * K), 0, ncols * K, 0x00020000);
    // First weight row of the two 64-column groups (a second group past N
    // repeats the first and is not stored), and their scales.
    int col[2];
    const float* ws_row[2];
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      col[q] = GATED ? q * N + n0 : n0 + (n0 + 64 * q < N ? 64 * q : 0);
      ws_row[q] = Ws + (static_cast<int64_t>(expert) * nnb + col[q] / 128) * nk;
    }
    auto run = [&](auto nx_c) {
      constexpr int NX = decltype(nx_c)::value;  // 16-row blocks
      const int i = lane & 15, g = lane >> 4;
      // A lane reads chunks g and 4 + g of a block of its row (the latter lie
      // beyond the end of a last block of 64).
      const int w_lane = (16 * (i >> 2) + (i & 3)) * K + 16 * g;
      const int x_lane = i * K + 16 * g;
      f32x4 acc[8][NX];
#pragma unroll
      for (int f = 0; f < 8; ++f)
#pragma unroll
        for (int x = 0; x < NX; ++x) acc[f][x] = f32x4{0.f, 0.f, 0.f, 0.f};
      i32x8 wf[8], xf[2][NX];
      float sx[2][NX], wsv[2] = {0.f, 0.f};
      auto load = [&](__amdgpu_buffer_rsrc_t r, int voff, int soff, bool cut) {
        const i32x4 lo =
            __builtin_bit_cast(i32x4, __builtin_amdgcn_raw_buffer_load_b128(r, voff, soff, 0));
        const i32x4 hi = __builtin_bit_cast(
            i32x4,
            __builtin_amdgcn_raw_buffer_load_b128(r, cut ? kOutOfRange : voff + 64, soff, 0));
        return i32x8{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
      };
      auto load_w = [&](int f, int kt) {
        wf[f] = load(w_rsrc, w_lane, (col[f >> 2] + 4 * (f & 3)) * K + kt * BK,
                     k_tail && kt == nk - 1);
      };
      auto load_x = [&](int b, int kt) {
#pragma unroll
        for (int x = 0; x < NX; ++x) {
          xf[b][x] = load(x_rsrc, x_lane + 16 * x * K, kt * BK, k_tail && kt == nk - 1);
          sx[b][x] = 16 * x + i < rows
                         ? Xs[static_cast<int64_t>(kt) * cap_rows + row_begin + 16 * x + i]
                         : 0.f;
        }
      };
      // Step j is block wave + kWaves j; past this wave's last one the last
      // block is loaded again and not used.
      const int steps = (nk - wave + kWaves - 1) / kWaves;
      if (steps > 0) {
        load_x(0, wave);
#pragma unroll
        for (int f = 0; f < 8; ++f) load_w(f, wave);
      }
      auto step = [&](int j, auto b_c) {
        constexpr int b = decltype(b_c)::value;
        if ((j & 63) == 0) {  // 64 steps' weight scales, one a lane
#pragma unroll
          for (int q = 0; q < 2; ++q) wsv[q] = ws_row[q][min(wave + kWaves * (j + lane), nk - 1)];
        }
        const int next = min(wave + kWaves * (j + 1), nk - 1);
        load_x(b ^ 1, next);
        float s[2][NX];
#pragma unroll
        for (int q = 0; q < 2; ++q)
#pragma unroll
          for (int x = 0; x < NX; ++x)
            s[q][x] = sx[b][x] * __builtin_bit_cast(float, __builtin_amdgcn_readlane(
                                     __builtin_bit_cast(int, wsv[q]), j & 63));
#pragma unroll
        for (int f = 0; f < 8; ++f) {
          f32x4 part[NX];
#pragma unroll
          for (int x = 0; x < NX; ++x) part[x] = mma(wf[f], xf[b][x]);
          load_w(f, next);
#pragma unroll
          for (int x = 0; x < NX; ++x)
#pragma unroll
            for (int r = 0; r < 4; ++r)
              acc[f][x][r] = __builtin_fmaf(part[x][r], s[f >> 2][x], acc[f][x][r]);
          __builtin_amdgcn_sched_barrier(0);
        }
      };
      for (int j = 0; j < steps; j += 2) {
        step(j, std::integral_constant<int, 0>{});
        if (j + 1 < steps) step(j + 1, std::integral_constant<int, 1>{});
      }
      // ---- sums of the waves, in order: [wave][fragment][row block][lane] ----
#pragma unroll
      for (int f = 0; f < 8; ++f)
#pragma unroll
        for (int x = 0; x < NX; ++x) red[((wave * 8 + f) * NX + x) * 64 + lane] = acc[f][x];
      __syncthreads();
      auto total = [&](int f, int x) {
        f32x4 v = red[(f * NX + x) * 64 + lane];
#pragma unroll
        for (int w = 1; w < kWaves; ++w) {
          const f32x4 u = red[((w * 8 + f) * NX + x) * 64 + lane];
#pragma unroll
          for (int r = 0; r < 4; ++r) v[r] += u[r];
        }
        return v;
      };
      // Wave w takes fragment w of each column group.
#pragma unroll
      for (int x = 0; x < NX; ++x) {
        const int row = row_begin + 16 * x + i;
        f32x4 v[2] = {total(wave, x), total(wave + 4, x)};
        if (GATED) {
#pragma unroll
          for (int r = 0; r < 4; ++r) v[0][r] = silu_mul(v[0][r], v[1][r]);
        }
        if (16 * x + i < rows) {
#pragma unroll
          for (int q = 0; q < (GATED ? 1 : 2); ++q) {
            const int c = n0 + 64 * q + 16 * g + 4 * wave;
            if (c < N) store4<KIND>(out, static_cast<int64_t>(row) * N + c, v[q]);
          }
        }
      }
    };
    if (rows <= 16)
      run(std::integral_constant<int, 1>{});
    else
      run(std::integral_constant<int, 2>{});
    // The sums have been read before the next tile's are written.
    __syncthreads();
  }
}

int num_cus() {
  static int cus = 0;
  if (cus == 0) {
    int dev = 0;
    hipDeviceProp_t p;
    if (hipGetDevice(&dev) == hipSuccess && hipGetDeviceProperties(&p, dev) == hipSuccess)
      cus = p.multiProcessorCount;
    if (cus <= 0) cus = 256;
  }
  return cus;
}

template <bool GATED, int KIND>
hipError_t launch_gemm(int n_experts, int64_t cap_rows, int K, int N, const void* xq,
                       const float* xs, const int32_t* offsets, const void* wq, const float* ws,
                       void* out, hipStream_t s) {
  const int n = offsets ? n_experts : 1;
  const int64_t cus = std::max<int64_t>(kXcds, num_cus() / kXcds * kXcds);
  // Small tiles (32 x 128) read the weights once for each 32 rows, large ones
  // (256 x 256) once for each 256, but large ones alone leave CUs idle, and take
  // longer over a block of few rows. Small ones win where they number a CU or
  // less, and, up to 32 rows an expert, where K is long and they are many (of
  // cap_rows, spread evenly: the counts are on the device). Measured, large
  // against small: one expert of 1024 rows, 2048 -> 1024 (256 small tiles),
  // 29 : 15 us; 8 of 14336 -> 4096, 32 rows each (256), 179 : 88; 32 of 7168 ->
  // 2 x 2048, 16 rows each (1024), 199 : 168; but 64 of 512 -> 512, 40 rows each
  // (512), 8 : 13, 40 of 1024 -> 1024, 16 rows each (320), 14 : 17, 8 of 1024 ->
  // 2 x 1024, 96 rows each (384), 12 : 18. (Over 600 such cases the choice is 1 %
  // slower than the better of the two in the mean, at most 1.34 times.)
  const int64_t hit = std::min<int64_t>(cap_rows, n);
  const int64_t small_tiles = hit * ((cap_rows + SM * hit - 1) / (SM * hit)) *
                              ((N + SN / (GATED ? 2 : 1) - 1) / (SN / (GATED ? 2 : 1)));
  const bool small = small_tiles <= cus ||
                     (cap_rows <= SM * hit && K >= 2048 && small_tiles >= 2 * cus);
  const int bm = small ? SM : BM, bn = (small ? SN : BN) / (GATED ? 2 : 1);
  const int64_t mt = std::min<int64_t>(cap_rows, cap_rows / bm + n);
  const int64_t tiles = mt * ((N + bn - 1) / bn);
  const int64_t g = std::min((tiles + kXcds - 1) / kXcds * kXcds, small ? 2 * cus : cus);
  auto* k = small ? fp8_small_kernel<GATED, KIND> : fp8_gemm_kernel<GATED, KIND>;
  k<<<static_cast<unsigned>(g), small ? kSmallThreads : kThreads, 0, s>>>(
      static_cast<const uint8_t*>(xq), xs, offsets, n_experts, cap_rows,
      static_cast<const uint8_t*>(wq), ws, out, K, N);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_gate_up_fp8(int n_experts, int64_t cap_rows, int D, int inter, const void* xq,
                              const float* xs, const int32_t* offsets, const void* wq,
                              const float* ws, void* h, hipStream_t s) {
  if (cap_rows == 0) return hipSuccess;
  return launch_gemm<true, kOutBf16>(n_experts, cap_rows, D, inter, xq, xs, offsets, wq, ws, h, s);
}

hipError_t launch_down_fp8(int n_experts, int64_t cap_rows, int D, int inter, const void* hq,
                           const float* hs, const int32_t* offsets, const void* wq,
                           const float* ws, void* y, bool y_half, hipStream_t s) {
  if (cap_rows == 0) return hipSuccess;
  auto* f = y_half ? launch_gemm<false, kOutF16> : launch_gemm<false, kOutF32>;
  return f(n_experts, cap_rows, inter, D, hq, hs, offsets, wq, ws, y, s);
}

}  // namespace moe

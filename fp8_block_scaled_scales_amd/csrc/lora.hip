// The low-rank adapters of many requests at once, for gfx950:
//
//   out[t] = base[t] + s_l (x[t] A_l^T) B_l^T,  l = the adapter of row t
//
// x, A [groups][rank][K] and B [groups][N][rank] in BF16 or FP16; the rows come
// sorted by adapter (route.hip). Two launches: v = x A^T of every row, the K
// range of a row tile shared by several workgroups (FP32 partial sums in the
// workspace, added in split order by the second), then out.
//
// Bound by HBM: a few rows per adapter read A_l and B_l once, many rows x once
// and out once. With few rows per adapter the operands go from memory straight to
// the matrix instructions' registers; with many that costs the caches four times
// the accesses, since the instruction's layout gives neighbouring lanes
// neighbouring rows: there the first product's operands pass through LDS. The
// outputs always do, so that neighbouring lanes hold neighbouring columns. 64 rows of
// 128 adapters, 7168 to 4096 at rank 16: 5.6 + 6.5 us (19 MB: 3), each a launch and a
// chain of offsets, slots and operands; 8192 of 8, 4096 to 4096 at rank 64: 25 + 45 us
// (0.21 GB: 36), the first 136 tiles in three parts on CUs that hold two workgroups (152
// CUs have two, 104 one), the second with every output through LDS (49 straight), the
// partial sums of v, then a strip's B and base waited for before its stores.
//
// Rounding: v is FP32; it enters the second product as the sum of two 16-bit
// numbers (its rounding and that of the rest, 16 bits of BF16 or 22 of FP16),
// three where the operands are BF16 and out is FP32: rounding it once would
// cost up to 2^-9 of every term, as much as a BF16 out's own rounding where the
// base is small. FP16 rows are scaled by a power of two first, to a largest v in
// [2^14, 2^15): none overflows, and the rest of a small one keeps FP16's whole
// range below it (2^-25 is half its smallest step, 2^-39 of the row's largest: 22
// bits of a v down to 2^-17 of that, 16 at 2^-23). The sum with base is FP32,
// rounded once.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "gemm_common.h"
#include "gemm_groups.h"
#include "quant_common.h"
#include "route_ops.h"

#pragma clang fp contract(off)

namespace dg {

namespace {

typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef _Float16 v8h __attribute__((ext_vector_type(8)));

// D += A B^T on 16 rows of each and 32 of K: lane l has K elements 8 (l / 16) ..
// + 7 of row l % 16 of either operand, and of D the column l % 16 and rows 4 (l
// / 16) .. + 3.
template <int XK>
__device__ __forceinline__ v4f mfma16x32(v4u a, v4u b, v4f c) {
  if constexpr (XK == 1)
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, a), __builtin_bit_cast(v8bf, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(v8h, a), __builtin_bit_cast(v8h, b), c, 0, 0, 0);
}

constexpr int kThreads = 256, kWaves = 4;

// The token of sorted row r, -1 where it has none.
__device__ __forceinline__ int token_of(const LoraArgs& p, int r) {
  const int s = p.slot[r];
  return s >= 0 && s < p.tokens ? s : -1;
}

// v of MT x 16 rows by NR x 16 ranks over a K range: four waves share it.
template <int XK, int MT, int NR>
__global__ __launch_bounds__(kThreads) void lora_shrink(const LoraArgs p, const RowGroups grp) {
  constexpr int BM = 16 * MT;
  __shared__ float red[kWaves][BM][NR * 16 + 1];
  GroupTile t;
  if (!find_tile<BM, 1>(grp, p.splits, t)) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, i16 = lane & 15, q = lane >> 4;
  const int steps = (int)((p.K + 63) / 64), whole = (int)(p.K / 64);
  const int s0 = (int)((int64_t)t.tn * steps / p.splits), s1 = (int)((int64_t)(t.tn + 1) * steps / p.splits);
  const int w0 = s0 + (int)((int64_t)wave * (s1 - s0) / kWaves), w1 = s0 + (int)((int64_t)(wave + 1) * (s1 - s0) / kWaves);
  // Rows past the group's, or without a token, and ranks past the last read a row
  // that there is: their sums are their own and are not kept.
  const uint16_t* const a = static_cast<const uint16_t*>(p.a) + (int64_t)t.group * p.rank * p.K + 16 * q;
  const uint16_t *xr[MT], *ar[NR];
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    const int r = t.tm * BM + m * 16 + i16;
    xr[m] = static_cast<const uint16_t*>(p.x) + (int64_t)max(r < t.rows ? token_of(p, t.row0 + r) : 0, 0) * p.ldx + 16 * q;
  }
#pragma unroll
  for (int n = 0; n < NR; ++n) ar[n] = a + (int64_t)min(n * 16 + i16, p.rank - 1) * p.K;
  v4f acc[MT][NR];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int n = 0; n < NR; ++n) acc[m][n] = (v4f){};
  // 64 of K a step: a lane's two pieces of 8 elements are neighbours, so that the
  // four lanes of a row ask for its whole 128-byte line at once
  auto step = [&](int s, auto in) {
    const int64_t k = (int64_t)s * 64;
    v4u xa[2][MT], ra[2][NR];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int m = 0; m < MT; ++m) xa[h][m] = in(h) ? *reinterpret_cast<const v4u*>(xr[m] + k + 8 * h) : (v4u){};
#pragma unroll
      for (int n = 0; n < NR; ++n) ra[h][n] = in(h) ? *reinterpret_cast<const v4u*>(ar[n] + k + 8 * h) : (v4u){};
    }
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int n = 0; n < NR; ++n) acc[m][n] = mfma16x32<XK>(xa[h][m], ra[h][n], acc[m][n]);
  };
#pragma unroll 2
  for (int s = w0; s < min(w1, whole); ++s) step(s, [](int) { return true; });
  if (w0 <= whole && whole < w1) step(whole, [&](int h) { return (int64_t)whole * 64 + 16 * q + 8 * h < p.K; });
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int n = 0; n < NR; ++n)
#pragma unroll
      for (int v = 0; v < 4; ++v) red[wave][m * 16 + 4 * q + v][n * 16 + i16] = acc[m][n][v];
  __syncthreads();
  for (int i = threadIdx.x; i < BM * NR * 16; i += kThreads) {
    const int m = i / (NR * 16), n = i % (NR * 16), r = t.tm * BM + m;
    if (r < t.rows && n < p.rank) {
      float v = red[0][m][n];
#pragma unroll
      for (int w = 1; w < kWaves; ++w) v += red[w][m][n];
      p.ws[((int64_t)t.tn * p.tokens + t.row0 + r) * p.rank + n] = v;
    }
  }
}

// The same with many rows per adapter: 64 rows of x and the adapter's ranks (RR
// rows of A) go through a ring of LDS slots, 64 of K (128 bytes a row) a step,
// by copies that take a row's line with eight neighbouring lanes. 16-byte chunks
// are swizzled by row as the FP8 product's slabs (key (row % 8) ^ ((row / 8) % 2)).
// A wave has 16 rows and the whole K range. 128 rows a tile, which halve the
// reading of A, take as long (25 us at 8192 x 4096, rank 64, eight adapters): half
// as many workgroups.
constexpr int kTall = 64;

__device__ __forceinline__ void copy16(const uint16_t* src, uint32_t lds) {
  asm volatile(
      "s_mov_b32 m0, %0\n\t"
      "s_nop 0\n\t"
      "global_load_lds_dwordx4 %1, off"
      :
      : "s"(lds), "v"(src)
      : "memory", "m0");
}

template <int LOADS, int MAXS>
__device__ __forceinline__ void wait_copies(int steps) {
  if constexpr (MAXS == 0) {
    DG_WAIT_VMCNT(0);
  } else {
    if (steps >= MAXS) {
      DG_WAIT_VMCNT(LOADS * MAXS);
    } else {
      wait_copies<LOADS, MAXS - 1>(steps);
    }
  }
}

template <int XK, int NR>
__global__ __launch_bounds__(kThreads) void lora_shrink_tall(const LoraArgs p, const RowGroups grp) {
  constexpr int RR = NR < 2 ? 32 : 16 * NR, ROWS = kTall + RR, STAGES = NR > 4 ? 3 : 4;  // two workgroups a CU
  constexpr int GROUPS = ROWS / 8, LOADS = GROUPS / kWaves, SLOT = ROWS * 128;
  static_assert(GROUPS % kWaves == 0, "the same number of copies in every wave");
  __shared__ __attribute__((aligned(1024))) uint8_t ring[STAGES * SLOT];
  GroupTile t;
  if (!find_tile<kTall, 1>(grp, p.splits, t)) return;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), i16 = lane & 15, q = lane >> 4;
  const int whole = (int)(p.K / 64);  // steps of 64; the rest of K goes to the last split
  const int s0 = (int)((int64_t)t.tn * whole / p.splits), steps = (int)((int64_t)(t.tn + 1) * whole / p.splits) - s0;
  const uint16_t* const a = static_cast<const uint16_t*>(p.a) + (int64_t)t.group * p.rank * p.K;
  auto row_of_x = [&](int m) {  // a row that there is where the tile has none: its sums are not kept
    const int r = t.tm * kTall + m;
    return static_cast<const uint16_t*>(p.x) + (int64_t)max(r < t.rows ? token_of(p, t.row0 + r) : 0, 0) * p.ldx;
  };
  auto row_of_a = [&](int n) { return a + (int64_t)min(n, p.rank - 1) * p.K; };
  // this wave's copies of a step: rows 8 g .. 8 g + 7 for g = wave, wave + 4, ...; lane L the chunk that belongs at L % 8 of row L / 8
  const uint16_t* src[LOADS];
#pragma unroll
  for (int i = 0; i < LOADS; ++i) {
    const int row = (i * kWaves + wave) * 8 + (lane >> 3);
    const int chunk = (lane & 7) ^ ((row & 7) ^ ((row >> 3) & 1));
    src[i] = (row < kTall ? row_of_x(row) : row_of_a(row - kTall)) + (int64_t)s0 * 64 + chunk * 8;
  }
  const uint32_t base = (uint32_t)(uintptr_t)(lds_void_t*)ring;
  auto issue = [&](int s) {
#pragma unroll
    for (int i = 0; i < LOADS; ++i)
      copy16(src[i] + (int64_t)s * 64, __builtin_amdgcn_readfirstlane(base + (s % STAGES) * SLOT + (i * kWaves + wave) * 1024));
  };
  v4f acc[NR];
#pragma unroll
  for (int n = 0; n < NR; ++n) acc[n] = (v4f){};
#pragma unroll
  for (int s = 0; s < STAGES - 1; ++s)
    if (s < steps) issue(s);
  auto frag = [&](const uint8_t* slot, int row, int c) {
    return *reinterpret_cast<const v4u*>(slot + row * 128 + ((c ^ ((row & 7) ^ ((row >> 3) & 1))) << 4));
  };
  for (int s = 0; s < steps; ++s) {
    wait_copies<LOADS, STAGES - 2>(min(STAGES - 2, steps - 1 - s));
    __syncthreads();  // step s visible to all waves; the slot of step s - 1 is free
    if (s + STAGES - 1 < steps) issue(s + STAGES - 1);
    const uint8_t* const slot = ring + (s % STAGES) * SLOT;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const v4u xa = frag(slot, wave * 16 + i16, 4 * h + q);
#pragma unroll
      for (int n = 0; n < NR; ++n) acc[n] = mfma16x32<XK>(xa, frag(slot, kTall + n * 16 + i16, 4 * h + q), acc[n]);
    }
    DG_STEP_SYNC_WG();
  }
  if (t.tn == p.splits - 1 && p.K % 64 != 0) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int64_t k = (int64_t)whole * 64 + 32 * h + 8 * q;
      const bool in = k < p.K;
      const v4u xa = in ? *reinterpret_cast<const v4u*>(row_of_x(wave * 16 + i16) + k) : (v4u){};
#pragma unroll
      for (int n = 0; n < NR; ++n)
        acc[n] = mfma16x32<XK>(xa, in ? *reinterpret_cast<const v4u*>(row_of_a(n * 16 + i16) + k) : (v4u){}, acc[n]);
    }
  }
#pragma unroll
  for (int n = 0; n < NR; ++n)
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      const int r = t.tm * kTall + wave * 16 + 4 * q + v;
      if (r < t.rows && n * 16 + i16 < p.rank) p.ws[((int64_t)t.tn * p.tokens + t.row0 + r) * p.rank + n * 16 + i16] = acc[n][v];
    }
}

constexpr int kStrip = 64;  // columns of a wave's step

typedef v4u v4u_at2 __attribute__((aligned(2)));
typedef v4f v4f_at4 __attribute__((aligned(4)));

// 16 bytes of consecutive outputs of a token, from column n on: the base's as
// they are stored (16-bit elements one to a word where the row ends inside).
template <int OK>
struct Out16 {
  static constexpr int B = InKind<OK>::kBytes, PER = 16 / B;
  typedef typename std::conditional<OK == 0, v4f_at4, v4u_at2>::type V;
};

template <int OK>
__device__ __forceinline__ void load_base(const LoraArgs& p, int64_t tok, int64_t n, unsigned (&w)[Out16<OK>::PER]) {
  typedef Out16<OK> O;
#pragma unroll
  for (int e = 0; e < O::PER; ++e) w[e] = 0;
  if (!p.base || n >= p.N) return;
  const char* const base = static_cast<const char*>(p.base) + (tok * p.ldbase + n) * O::B;
  if (n + O::PER <= p.N) {
    const v4u v = __builtin_bit_cast(v4u, *reinterpret_cast<const typename O::V*>(base));
#pragma unroll
    for (int e = 0; e < 4; ++e) w[e] = v[e];
  } else {
#pragma unroll
    for (int e = 0; e < O::PER; ++e) {
      if (n + e >= p.N) break;
      w[e] = OK == 0 ? reinterpret_cast<const uint32_t*>(base)[e] : reinterpret_cast<const uint16_t*>(base)[e];
    }
  }
}

template <int OK>
__device__ __forceinline__ void add_store(const LoraArgs& p, int64_t tok, int64_t n, const float (&d)[Out16<OK>::PER],
                                          const unsigned (&w)[Out16<OK>::PER]) {
  typedef Out16<OK> O;
  if (n >= p.N) return;
  char* const out = static_cast<char*>(p.out) + (tok * p.N + n) * O::B;
  if (n + O::PER <= p.N) {
    float f[O::PER];
    widen_raw(Raw<OK, O::PER>{{w[0], w[1], w[2], w[3]}}, f);
#pragma unroll
    for (int e = 0; e < O::PER; ++e) f[e] += d[e];
    const Raw<OK, O::PER> r = round_raw<OK>(f);
    *reinterpret_cast<typename O::V*>(out) = __builtin_bit_cast(typename O::V, (v4u){r.w[0], r.w[1], r.w[2], r.w[3]});
  } else {
#pragma unroll
    for (int e = 0; e < O::PER; ++e) {
      if (n + e >= p.N) break;
      if constexpr (OK == 0) {
        reinterpret_cast<float*>(out)[e] = __uint_as_float(w[e]) + d[e];
      } else {
        float f[4];
        widen_raw(Raw<OK, 4>{{w[e], 0u}}, f);
        f[0] += d[e];
        reinterpret_cast<uint16_t*>(out)[e] = (uint16_t)round_raw<OK>(f).w[0];
      }
    }
  }
}

// A token without an adapter (its position is no row's), where out is not base: a
// wave, which looks at kCopyTokens, copies its row.
constexpr int kCopyTokens = 8;

template <int OK>
__device__ __forceinline__ void copy_row(const LoraArgs& p, int64_t tok, int lane) {
  constexpr int B = InKind<OK>::kBytes, PER = 16 / B;
  typedef typename std::conditional<OK == 0, v4f_at4, v4u_at2>::type V;
  char* const out = static_cast<char*>(p.out) + tok * p.N * B;
  const char* const base = static_cast<const char*>(p.base) + tok * p.ldbase * B;
  const int64_t whole = p.N / PER;
#pragma unroll 8
  for (int64_t i = lane; i < whole; i += 64) {
    const V v = p.base ? *reinterpret_cast<const V*>(base + 16 * i) : (V){};
    *reinterpret_cast<V*>(out + 16 * i) = v;
  }
  for (int64_t n = whole * PER + lane; n < p.N; n += 64) {
    if constexpr (B == 4) reinterpret_cast<uint32_t*>(out)[n] = p.base ? reinterpret_cast<const uint32_t*>(base)[n] : 0u;
    else reinterpret_cast<uint16_t*>(out)[n] = p.base ? reinterpret_cast<const uint16_t*>(base)[n] : (uint16_t)0;
  }
}

__device__ __forceinline__ float rest_of(float f, float h) {
  const float r = f - h;
  return r == r ? r : 0.0f;
}

// f as TERMS 16-bit numbers: its rounding, that of the rest, ... (an infinite one
// has no rest; a finite one that BF16 would round to infinity leaves what is past
// the largest BF16 to its rest)
template <int XK, int TERMS>
__device__ __forceinline__ void split16(float f, uint16_t (&t)[TERMS]) {
#pragma unroll
  for (int i = 0; i < TERMS; ++i) {
    if constexpr (XK == 1) {
      const __bf16 h = (__bf16)(fabsf(f) < __builtin_inff() ? fminf(fmaxf(f, -0x1.fep127f), 0x1.fep127f) : f);
      t[i] = __builtin_bit_cast(uint16_t, h);
      f = rest_of(f, (float)h);
    } else {
      const _Float16 h = (_Float16)f;
      t[i] = __builtin_bit_cast(uint16_t, h);
      f = rest_of(f, (float)h);
    }
  }
}

template <int XK>
__device__ __forceinline__ float widen16(uint16_t h) {
  if constexpr (XK == 1) return __uint_as_float((unsigned)h << 16);
  else return (float)__builtin_bit_cast(_Float16, h);
}

// out of MT x 16 rows by `strips` x 4 x 64 columns. The rows of B_l are the
// first operand: a lane's four sums are neighbours in a token's row, and pass
// through LDS (16 tokens of a strip at a time, a wave's own) to lanes that hold 16
// bytes of outputs each, a token's 64 columns in neighbouring lanes. KS: 32-wide
// steps of the rank.
template <int XK, int OK, int MT, int KS>
__global__ __launch_bounds__(kThreads) void lora_expand(const LoraArgs p, const RowGroups grp, unsigned tile_wgs, int strips) {
  constexpr int BM = 16 * MT, RP = 32 * KS, LD = RP + 8;  // pitch in 16-bit elements: 16-byte reads of 16 rows on distinct banks
  constexpr int TERMS = XK == 1 && OK == 0 ? 3 : 2;
  __shared__ __attribute__((aligned(16))) uint16_t term[TERMS][BM][LD];
  constexpr int LDP = kStrip + 4;  // pitch of a strip's sums in floats
  __shared__ int back[BM];  // exponents of the rows' scaling
  __shared__ int tokens[BM];
  __shared__ __attribute__((aligned(16))) float sums[kWaves][16][LDP];
  int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, i16 = lane & 15, q = lane >> 4;
  if (blockIdx.x >= tile_wgs) {
    for (int64_t t0 = ((int64_t)(blockIdx.x - tile_wgs) * kWaves + wave) * kCopyTokens; t0 < p.tokens;
         t0 += (int64_t)(gridDim.x - tile_wgs) * kWaves * kCopyTokens) {
      const int row = lane < kCopyTokens && t0 + lane < p.tokens ? p.position[t0 + lane] : 0;
      uint64_t m = __ballot(row < 0 || row >= p.tokens);
      for (; m; m &= m - 1) copy_row<OK>(p, t0 + __builtin_ctzll(m), lane);
    }
    return;
  }
  GroupTile t;
  const int col_tiles = (int)((p.N + kStrip * kWaves * strips - 1) / (kStrip * kWaves * strips));
  if (!find_tile<BM, 1>(grp, col_tiles, t)) return;
  const float scale = p.scale ? p.scale[t.group] : 1.0f;

  for (int m = threadIdx.x; m < BM; m += kThreads) {
    const int r = t.tm * BM + m;
    tokens[m] = r < t.rows ? token_of(p, t.row0 + r) : -1;
  }
  __syncthreads();

  const uint16_t* const b = static_cast<const uint16_t*>(p.b) + (int64_t)t.group * p.N * p.rank;
  // a lane's outputs: PER columns from col on, of tokens RPI apart
  constexpr int PER = Out16<OK>::PER, LPR = kStrip / PER, RPI = 64 / LPR, ITS = 16 / RPI;
  int col = (lane % LPR) * PER, row = lane / LPR;
  auto first_col = [&](int st) { return (((int64_t)t.tn * strips + st) * kWaves + wave) * kStrip; };
  v4u br[KS][4];
  unsigned old[MT][ITS][PER];
  auto load_b = [&](int64_t n0) {  // a strip's rows of B_l
#pragma unroll
    for (int ks = 0; ks < KS; ++ks)
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        // past the last column a column that there is (not stored), past the rank
        // elements that there are (v is zero there)
        const int64_t n = min(n0 + 16 * s + i16, p.N - 1);
        br[ks][s] = *reinterpret_cast<const v4u*>(b + n * p.rank + min(32 * ks + 8 * q, p.rank - 8));
      }
  };
  auto load_bases = [&](int64_t n0) {  // all of its base, ahead of the first store, which may be to the same memory
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int it = 0; it < ITS; ++it) {
        const int tok = tokens[m * 16 + it * RPI + row];
        if (tok >= 0) load_base<OK>(p, tok, n0 + col, old[m][it]);
      }
  };

  // the strip's sums of 16 tokens, to LDS
  auto sums_of = [&](int m) {
    v4f acc[4];
#pragma unroll
    for (int s = 0; s < 4; ++s) acc[s] = (v4f){};
#pragma unroll
    for (int k = TERMS - 1; k >= 0; --k)
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        const v4u h = *reinterpret_cast<const v4u*>(&term[k][m * 16 + i16][32 * ks + 8 * q]);
#pragma unroll
        for (int s = 0; s < 4; ++s) acc[s] = mfma16x32<XK>(br[ks][s], h, acc[s]);
      }
    // a wave's LDS operations are in order: no barrier, but none may be moved
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int s = 0; s < 4; ++s) *reinterpret_cast<v4f*>(&sums[wave][i16][16 * s + 4 * q]) = acc[s];
    __builtin_amdgcn_wave_barrier();
  };
  // a lane's sums of one of them; whether none is NaN (nor infinities of both signs among them)
  auto sums_at = [&](int m, int r, float (&d)[PER]) {
    float all = 0.0f;
#pragma unroll
    for (int e = 0; e < PER; e += 4) {
      const v4f f = *reinterpret_cast<const v4f*>(&sums[wave][r][col + e]);
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        d[e + v] = XK == 2 ? __builtin_amdgcn_ldexpf(f[v], back[m * 16 + r]) : f[v];
        all += f[v];
      }
    }
    return all == all;
  };

  // v of the tile, its terms to LDS: neighbouring threads take neighbouring fours
  // of a row (with a row's fours spread over the passes instead, lines were
  // fetched up to four times)
  {
    constexpr int FOURS = RP / 4, VITS = BM * FOURS / kThreads;
    static_assert(VITS * kThreads == BM * FOURS || VITS == 0, "whole passes");
    const int n = (threadIdx.x % FOURS) * 4;
    v4f v[VITS ? VITS : 1];
#pragma unroll
    for (int i = 0; i < (VITS ? VITS : 1); ++i) {
      const int m = (i * kThreads + threadIdx.x) / FOURS, r = t.tm * BM + m;
      v[i] = (v4f){};
      if (m < BM && r < t.rows && n < p.rank) {
        const float* src = p.ws + ((int64_t)t.row0 + r) * p.rank + n;
#pragma unroll 4
        for (int s = 0; s < p.splits; ++s) v[i] += *reinterpret_cast<const v4f*>(src + (int64_t)s * p.tokens * p.rank);
      }
    }
#pragma unroll
    for (int i = 0; i < (VITS ? VITS : 1); ++i) {
      const int m = (i * kThreads + threadIdx.x) / FOURS;
#pragma unroll
      for (int e = 0; e < 4; ++e) v[i][e] *= scale;
      if constexpr (XK == 2) {
        float top = 0.0f;  // of those that are finite
#pragma unroll
        for (int e = 0; e < 4; ++e) top = fmaxf(top, fabsf(v[i][e]) < __builtin_inff() ? fabsf(v[i][e]) : 0.0f);
#pragma unroll
        for (int d = 1; d < FOURS; d <<= 1) top = fmaxf(top, __shfl_xor(top, d, 64));
        const int up = 15 - __builtin_amdgcn_frexp_expf(top);  // rank 128 and B at its largest: sums below 2^39
        // by exponent: 2^up itself may be past FP32's range
#pragma unroll
        for (int e = 0; e < 4; ++e) v[i][e] = __builtin_amdgcn_ldexpf(v[i][e], up);
        if (n == 0 && m < BM) back[m] = -up;
      }
      if (m < BM) {
        uint16_t f[4][TERMS];
#pragma unroll
        for (int e = 0; e < 4; ++e) split16<XK, TERMS>(v[i][e], f[e]);
#pragma unroll
        for (int k = 0; k < TERMS; ++k)
          *reinterpret_cast<uint2*>(&term[k][m][n]) = make_uint2(f[0][k] | ((unsigned)f[1][k] << 16), f[2][k] | ((unsigned)f[3][k] << 16));
      }
    }
  }
  __syncthreads();

  bool again = false;
  for (int st = 0; st < strips; ++st) {
    const int64_t n0 = first_col(st);
    if (n0 >= p.N) break;
    load_b(n0);  // ahead of v instead: 42.9 -> 45 us
    load_bases(n0);
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      sums_of(m);
#pragma unroll
      for (int it = 0; it < ITS; ++it) {
        const int r = it * RPI + row, tok = tokens[m * 16 + r];
        float d[PER];
        const bool whole = sums_at(m, r, d);
        if (tok >= 0 && whole) add_store<OK>(p, tok, n0 + col, d, old[m][it]);
        again |= tok >= 0 && !whole;
      }
    }
  }
  if (!__any(again)) return;

  // Outputs with a NaN among their sums, which were left as they were. An infinite
  // element of B is NaN times the rest of an element of v that has none, or of the
  // other sign, and times the zeros past the rank: where B holds one, sums that came
  // out NaN are taken again, element by element. (The lane's numbers are worked out
  // anew, so that none is held in a register until here: 8192 x 4096 to 4096 at rank
  // 128, eight adapters, 102 -> 93 us.)
  int tid = threadIdx.x;
  asm volatile("" : "+v"(tid));
  lane = tid & 63, wave = tid >> 6, i16 = lane & 15, q = lane >> 4;
  col = (lane % LPR) * PER, row = lane / LPR;
  for (int st = 0; st < strips; ++st) {
    const int64_t n0 = first_col(st);
    if (n0 >= p.N) return;
    load_b(n0);
    v2u16 top = {};
#pragma unroll
    for (int ks = 0; ks < KS; ++ks)
#pragma unroll
      for (int s = 0; s < 4; ++s)
#pragma unroll
        for (int i = 0; i < 4; ++i) top = __builtin_elementwise_max(top, abs_bits2(br[ks][s][i]));
    const bool beyond = __any(max(top.x, top.y) >= (XK == 1 ? 0x7F80 : 0x7C00));
#pragma unroll 1
    for (int m = 0; m < MT; ++m) {
      sums_of(m);
      unsigned left = 0;  // this lane's outputs that were left
#pragma unroll 1
      for (int it = 0; it < ITS; ++it) {
        float d[PER];
        left |= (unsigned)!sums_at(m, it * RPI + row, d) << it;
      }
      __builtin_amdgcn_wave_barrier();
#pragma unroll 1
      for (int i = 0; beyond && i < 16; ++i) {
        const int c = 16 * (i >> 2) + 4 * q + (i & 3);
        if (n0 + c >= p.N || sums[wave][i16][c] == sums[wave][i16][c]) continue;
        const uint16_t* const bn = b + (n0 + c) * p.rank;
        float sum = 0.0f;
#pragma unroll 1
        for (int r = 0; r < p.rank; ++r) {
          float f = 0.0f;
#pragma unroll
          for (int k = TERMS - 1; k >= 0; --k) f += widen16<XK>(term[k][m * 16 + i16][r]);
          sum = __builtin_fmaf(f, widen16<XK>(bn[r]), sum);
        }
        sums[wave][i16][c] = sum;
      }
      __builtin_amdgcn_wave_barrier();
#pragma unroll 1
      for (int it = 0; it < ITS; ++it) {
        const int r = it * RPI + row, tok = tokens[m * 16 + r];
        if (tok < 0 || !(left >> it & 1)) continue;
        float d[PER];
        unsigned w[PER];
        sums_at(m, r, d);
        load_base<OK>(p, tok, n0 + col, w);
        add_store<OK>(p, tok, n0 + col, d, w);
      }
    }
  }
}

// Workgroups that any lengths of the groups could need.
int64_t most_tiles(const LoraArgs& p, int bm) { return p.tokens / bm + std::min<int64_t>(p.groups, p.tokens); }

template <int XK, int MT, int NR>
hipError_t shrink(const LoraArgs& p, const RowGroups& g, hipStream_t stream) {
  hipLaunchKernelGGL((lora_shrink<XK, MT, NR>), dim3((unsigned)(most_tiles(p, 16 * MT) * p.splits)), dim3(kThreads), 0, stream, p, g);
  return hipGetLastError();
}

template <int XK, int NR>
hipError_t shrink_tall(const LoraArgs& p, const RowGroups& g, hipStream_t stream) {
  hipLaunchKernelGGL((lora_shrink_tall<XK, NR>), dim3((unsigned)(most_tiles(p, kTall) * p.splits)), dim3(kThreads), 0, stream, p, g);
  return hipGetLastError();
}

template <int XK, int MT>
hipError_t shrink_r(const LoraArgs& p, const RowGroups& g, hipStream_t stream) {
  if constexpr (MT == 1) {
    if (p.rank <= 16) return shrink<XK, 1, 1>(p, g, stream);
    if (p.rank <= 32) return shrink<XK, 1, 2>(p, g, stream);
    if (p.rank <= 64) return shrink<XK, 1, 4>(p, g, stream);
    return shrink<XK, 1, 8>(p, g, stream);
  } else {
    if (p.rank <= 16) return shrink_tall<XK, 1>(p, g, stream);
    if (p.rank <= 32) return shrink_tall<XK, 2>(p, g, stream);
    if (p.rank <= 64) return shrink_tall<XK, 4>(p, g, stream);
    return shrink_tall<XK, 8>(p, g, stream);
  }
}

// Columns of a workgroup: as many as leave 1024 workgroups, so that v is brought
// to LDS for few of them.
template <int XK, int OK, int MT, int KS>
hipError_t expand(const LoraArgs& p, const RowGroups& g, hipStream_t stream) {
  const int64_t tiles = most_tiles(p, 16 * MT), cols = (p.N + kStrip * kWaves - 1) / (kStrip * kWaves);
  const int64_t strips = std::max<int64_t>(1, std::min<int64_t>(tiles * cols / 1024, cols));
  const int64_t wgs = tiles * ((cols + strips - 1) / strips);
  const int64_t copies = p.base == p.out ? 0 : std::min<int64_t>((p.tokens + kWaves * kCopyTokens - 1) / (kWaves * kCopyTokens), 1 << 16);
  hipLaunchKernelGGL((lora_expand<XK, OK, MT, KS>), dim3((unsigned)(wgs + copies)), dim3(kThreads), 0, stream, p, g, (unsigned)wgs, (int)strips);
  return hipGetLastError();
}

template <int XK, int OK, int MT>
hipError_t expand_r(const LoraArgs& p, const RowGroups& g, hipStream_t stream) {
  if (p.rank <= 32) return expand<XK, OK, MT, 1>(p, g, stream);
  if (p.rank <= 64) return expand<XK, OK, MT, 2>(p, g, stream);
  return expand<XK, OK, MT, 4>(p, g, stream);
}

template <int XK, int MT>
hipError_t both(const LoraArgs& p, hipStream_t stream) {
  const RowGroups g{p.offsets, p.groups, (int)p.tokens};
  const hipError_t err = shrink_r<XK, MT>(p, g, stream);
  if (err != hipSuccess) return err;
  switch (p.ok) {
    case 0: return expand_r<XK, 0, MT>(p, g, stream);
    case 1: return expand_r<XK, 1, MT>(p, g, stream);
    case 2: return expand_r<XK, 2, MT>(p, g, stream);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace

// 16-row blocks of a tile: 64 rows where a group of the mean length fills them. K = N =
// 4096, 64 rows / 16, in us: 32 tokens of each of 8 adapters at rank 16 14.2 / 12.1, at
// rank 64 17.3 / 14.1; 64 of each 14.8 / 12.7 and 18.4 / 18.7; 64 of each of 64
// adapters 38 / 41 and 53 / 87; 128 of each of 8 16.3 / 16.3 and 20.5 / 22.2.
static int blocks_of(int64_t tokens, int groups) {
  return tokens >= 64ll * groups ? 4 : 1;
}

int lora_splits(int64_t tokens, int64_t K, int groups) {
  const int64_t tiles = tokens / (16 * blocks_of(tokens, groups)) + std::min<int64_t>(groups, tokens);
  const int64_t want = std::max<int64_t>(1, 512 / tiles), most = std::max<int64_t>(1, K / 512);
  return (int)std::min<int64_t>(std::min(want, most), 16);
}

hipError_t launch_lora(const LoraArgs& p, hipStream_t stream) {
  const bool tall = blocks_of(p.tokens, p.groups) == 4;
  if (p.xk == 1) return tall ? both<1, 4>(p, stream) : both<1, 1>(p, stream);
  if (p.xk == 2) return tall ? both<2, 4>(p, stream) : both<2, 1>(p, stream);
  return hipErrorInvalidValue;
}

}  // namespace dg

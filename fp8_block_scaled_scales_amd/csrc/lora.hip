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
// and out once. Operands go from memory straight to the matrix instructions'
// registers: a lane's eight consecutive elements of a row are one 16-byte load,
// and neither operand is used by another wave of the tile.
//
// Rounding: v is FP32; it enters the second product as the sum of two 16-bit
// numbers (its rounding and that of the rest, 16 bits of BF16 or 22 of FP16),
// three where the operands are BF16 and out is FP32: rounding it once would
// cost up to 2^-9 of every term, as much as a BF16 out's own rounding where the
// base is small. FP16 rows are scaled by a power of two first, so that no v
// overflows. The sum with base is FP32, rounded once.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

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

// A token without an adapter, where out is not base: a wave copies its row.
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

// f as TERMS 16-bit numbers: its rounding, that of the rest, ...
template <int XK, int TERMS>
__device__ __forceinline__ void split16(float f, uint16_t (&t)[TERMS]) {
#pragma unroll
  for (int i = 0; i < TERMS; ++i) {
    if constexpr (XK == 1) {
      const __bf16 h = (__bf16)f;
      t[i] = __builtin_bit_cast(uint16_t, h);
      f -= (float)h;
    } else {
      const _Float16 h = (_Float16)f;
      t[i] = __builtin_bit_cast(uint16_t, h);
      f -= (float)h;
    }
  }
}

// The column of row i of the strip's product s (0 .. 3): 32-bit outputs as they
// come, 16-bit ones in pairs of products that share 32 columns.
template <int OK>
__device__ __forceinline__ int strip_col(int s, int i) {
  return OK == 0 ? 16 * s + i : 32 * (s >> 1) + 8 * (i >> 2) + 4 * (s & 1) + (i & 3);
}

// out of MT x 16 rows by `strips` x 4 x 64 columns. The rows of B_l are the
// first operand, so that a lane ends with outputs of one token. Which columns of a
// 64-column strip a product's 16 rows stand for is free (strip_col): those that
// give a lane 16 bytes of consecutive outputs, and four neighbouring lanes 64.
// KS: 32-wide steps of the rank.
template <int XK, int OK, int MT, int KS>
__global__ __launch_bounds__(kThreads) void lora_expand(const LoraArgs p, const RowGroups grp, unsigned tile_wgs, int strips) {
  constexpr int BM = 16 * MT, RP = 32 * KS, LD = RP + 8;  // pitch in 16-bit elements: 16-byte reads of 16 rows on distinct banks
  constexpr int TERMS = XK == 1 && OK == 0 ? 3 : 2;
  __shared__ __attribute__((aligned(16))) uint16_t term[TERMS][BM][LD];
  __shared__ float back[BM];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, i16 = lane & 15, q = lane >> 4;
  if (blockIdx.x >= tile_wgs) {
    for (int64_t tok = (int64_t)(blockIdx.x - tile_wgs) * kWaves + wave; tok < p.tokens; tok += (int64_t)(gridDim.x - tile_wgs) * kWaves)
      if (p.position[tok] < 0) copy_row<OK>(p, tok, lane);
    return;
  }
  GroupTile t;
  const int col_tiles = (int)((p.N + kStrip * kWaves * strips - 1) / (kStrip * kWaves * strips));
  if (!find_tile<BM, 1>(grp, col_tiles, t)) return;
  const float scale = p.scale ? p.scale[t.group] : 1.0f;

  // v of the tile, its terms to LDS: a thread takes TPR-strided fours of one row
  {
    constexpr int TPR = kThreads / BM, FOURS = RP / 4, ITS = (FOURS + TPR - 1) / TPR;
    const int m = threadIdx.x / TPR, c = threadIdx.x % TPR, r = t.tm * BM + m;
    const bool has = r < t.rows;
    v4f v[ITS];
    float top = 0.0f;
#pragma unroll
    for (int i = 0; i < ITS; ++i) {
      const int n = (i * TPR + c) * 4;
      v[i] = (v4f){};
      if (has && n < p.rank) {
        const float* src = p.ws + ((int64_t)t.row0 + r) * p.rank + n;
#pragma unroll 4
        for (int s = 0; s < p.splits; ++s) v[i] += *reinterpret_cast<const v4f*>(src + (int64_t)s * p.tokens * p.rank);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) v[i][e] *= scale;
      top = fmaxf(top, amax4(v[i]));
    }
    float down = 1.0f;
    if constexpr (XK == 2) {
#pragma unroll
      for (int d = 1; d < TPR; d <<= 1) top = fmaxf(top, __shfl_xor(top, d, 64));
      const int e = min(max(__builtin_amdgcn_frexp_expf(top), -100), 100);
      down = __builtin_amdgcn_ldexpf(1.0f, -e);
      if (c == 0) back[m] = __builtin_amdgcn_ldexpf(1.0f, e);
    }
#pragma unroll
    for (int i = 0; i < ITS; ++i) {
      const int n = (i * TPR + c) * 4;
      if (n < RP) {
        uint16_t b[4][TERMS];
#pragma unroll
        for (int e = 0; e < 4; ++e) split16<XK, TERMS>(v[i][e] * down, b[e]);
#pragma unroll
        for (int k = 0; k < TERMS; ++k)
          *reinterpret_cast<uint2*>(&term[k][m][n]) = make_uint2(b[0][k] | ((unsigned)b[1][k] << 16), b[2][k] | ((unsigned)b[3][k] << 16));
      }
    }
  }
  __syncthreads();

  const uint16_t* const b = static_cast<const uint16_t*>(p.b) + (int64_t)t.group * p.N * p.rank;
  int tok[MT];
  float up[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    const int r = t.tm * BM + m * 16 + i16;
    tok[m] = r < t.rows ? token_of(p, t.row0 + r) : -1;
    up[m] = XK == 2 ? back[m * 16 + i16] : 1.0f;
  }
  for (int st = 0; st < strips; ++st) {
    const int64_t n0 = (((int64_t)t.tn * strips + st) * kWaves + wave) * kStrip;
    if (n0 >= p.N) return;
    // a strip's outputs: 64 bytes of 16-bit ones in two pieces per lane, of FP32 in four
    constexpr int PER = Out16<OK>::PER, PIECES = 16 / PER;
    v4u br[KS][4];
#pragma unroll
    for (int ks = 0; ks < KS; ++ks)
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        // past the last column a column that there is (not stored), past the rank
        // elements that there are (v is zero there)
        const int64_t n = min(n0 + strip_col<OK>(s, i16), p.N - 1);
        br[ks][s] = *reinterpret_cast<const v4u*>(b + n * p.rank + min(32 * ks + 8 * q, p.rank - 8));
      }
    // all of the base ahead of the first store, which may be to the same memory
    unsigned old[MT][PIECES][PER];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int h = 0; h < PIECES; ++h)
        if (tok[m] >= 0) load_base<OK>(p, tok[m], n0 + strip_col<OK>(h * (4 / PIECES), 4 * q), old[m][h]);
#pragma unroll
    for (int m = 0; m < MT; ++m) {
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
      if (tok[m] < 0) continue;
#pragma unroll
      for (int h = 0; h < PIECES; ++h) {
        float d[PER];
#pragma unroll
        for (int e = 0; e < PER; ++e) d[e] = acc[h * (4 / PIECES) + e / 4][e % 4] * up[m];
        add_store<OK>(p, tok[m], n0 + strip_col<OK>(h * (4 / PIECES), 4 * q), d, old[m][h]);
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

template <int XK, int MT>
hipError_t shrink_r(const LoraArgs& p, const RowGroups& g, hipStream_t stream) {
  if (p.rank <= 16) return shrink<XK, MT, 1>(p, g, stream);
  if (p.rank <= 32) return shrink<XK, MT, 2>(p, g, stream);
  if (p.rank <= 64) return shrink<XK, MT, 4>(p, g, stream);
  return shrink<XK, (MT > 2 ? 2 : MT), 8>(p, g, stream);
}

// Columns of a workgroup: as many as leave 1024 workgroups, so that v is brought
// to LDS for few of them.
template <int XK, int OK, int MT, int KS>
hipError_t expand(const LoraArgs& p, const RowGroups& g, hipStream_t stream) {
  const int64_t tiles = most_tiles(p, 16 * MT), cols = (p.N + kStrip * kWaves - 1) / (kStrip * kWaves);
  const int64_t strips = std::max<int64_t>(1, std::min<int64_t>(tiles * cols / 1024, cols));
  const int64_t wgs = tiles * ((cols + strips - 1) / strips);
  const int64_t copies = p.base == p.out ? 0 : std::min<int64_t>((p.tokens + kWaves - 1) / kWaves, 1 << 16);
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

// Rows per adapter from which a tile takes 64 of them instead of 16.
static bool tall(int64_t tokens, int groups) { return tokens >= 32ll * groups; }

int lora_splits(int64_t tokens, int64_t K, int groups) {
  const int64_t tiles = tokens / (tall(tokens, groups) ? 64 : 16) + std::min<int64_t>(groups, tokens);
  const int64_t want = std::max<int64_t>(1, 512 / tiles), most = std::max<int64_t>(1, K / 512);
  return (int)std::min<int64_t>(std::min(want, most), 16);
}

hipError_t launch_lora(const LoraArgs& p, hipStream_t stream) {
  const bool t = tall(p.tokens, p.groups);
  if (p.xk == 1) return t ? both<1, 4>(p, stream) : both<1, 1>(p, stream);
  if (p.xk == 2) return t ? both<2, 4>(p, stream) : both<2, 1>(p, stream);
  return hipErrorInvalidValue;
}

}  // namespace dg

// The product's epilogue with a residual (compiled form EPI = 3 of every
// kernel class):
//
//   z = C + bias[j];  pre = bf16(z);  out = bf16(act(z) + residual)
//
// all in FP32 with one rounding into each output. The accumulators pass through
// LDS as FP32 (the plain forms stage BF16), so that each thread then holds
// consecutive outputs of a row: the residual is read and pre and out are
// written 16 bytes at a time, and the activation is code for eight values, not
// for every accumulator register, which lets one compiled form take every
// activation and residual type. Rows of any pitch and base keep the 16-byte
// accesses (global memory takes them at any address; the types below carry
// the elements' own alignment): only the last few columns go one by one.
//
// Bound by HBM at the ends of tiles that all CUs reach together: 8192^3 takes
// 474.9 us with bias, BF16 residual and pre (268 MB more, 45 us at a copy's
// rate) and 501.7 with GELU too, where the plain product takes 433.7 (one set of
// operands; with three sets in turn 520 and 454).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "activation.h"
#include "gemm_common.h"
#include "quant_common.h"

namespace dg {

// Passed by value after the plain arguments; the other forms read none of it.
struct EpiArgs {
  const float* bias;  // [N] or null
  const void* res;    // [M][N], row pitch ldres elements, of kind res_kind; may be out itself
  uint16_t* out;
  uint16_t* pre;      // [M][N] BF16 or null
  int64_t ldres;
  int res_kind;       // 0 FP32, 1 BF16, 2 FP16, 3 none
  int act;            // 0 none, 1 ReLU, 2 GELU, 3 SiLU, 4 GELU (tanh form)
};

// Four words at the alignment of the elements they hold.
typedef v4f v4f_at4 __attribute__((aligned(4)));
typedef unsigned v2u_at2 __attribute__((ext_vector_type(2), aligned(2)));
typedef unsigned v4u_at2 __attribute__((ext_vector_type(4), aligned(2)));

// The residual of NV (4 or 8) consecutive outputs as loaded, so that a load
// long before its use waits for nothing: FP32 words; 16-bit elements two to a
// word, or one to a word (the low half) where the row ends inside.
template <int NV>
struct RawResidual {
  unsigned w[NV];
};

template <bool ONCE, class V>
__device__ __forceinline__ V load_wide(const V* p) {
  if constexpr (ONCE) return __builtin_nontemporal_load(p);
  else return *p;
}

// From (row, col) on; row < M and col < N. ONCE (here and below): nontemporal
// 16-byte accesses.
template <int NV, bool ONCE = false>
__device__ __forceinline__ void load_residual(const EpiArgs& e, int64_t row, int col, int N, RawResidual<NV>& r) {
  if (e.res_kind == 3) return;
  const int64_t at = row * e.ldres + col;
  if (col + NV <= N) {
    if (e.res_kind == 0) {
      const float* src = static_cast<const float*>(e.res) + at;
#pragma unroll
      for (int q = 0; q < NV / 4; ++q) {
        const v4f v = load_wide<ONCE>(reinterpret_cast<const v4f_at4*>(src + 4 * q));
#pragma unroll
        for (int t = 0; t < 4; ++t) r.w[4 * q + t] = __float_as_uint(v[t]);
      }
    } else {
      const uint16_t* src = static_cast<const uint16_t*>(e.res) + at;
      if constexpr (NV == 8) {
        const v4u v = load_wide<ONCE>(reinterpret_cast<const v4u_at2*>(src));
#pragma unroll
        for (int t = 0; t < 4; ++t) r.w[t] = v[t];
      } else {
        const v2u_at2 v = *reinterpret_cast<const v2u_at2*>(src);
        r.w[0] = v.x;
        r.w[1] = v.y;
      }
    }
  } else {
#pragma unroll
    for (int t = 0; t < NV; ++t) {
      if (col + t >= N) break;
      r.w[t] = e.res_kind == 0 ? static_cast<const unsigned*>(e.res)[at + t] : static_cast<const uint16_t*>(e.res)[at + t];
    }
  }
}

// z += the residual, those outputs past column N - 1 left as they are.
template <int NV>
__device__ __forceinline__ void add_residual(const EpiArgs& e, int col, int N, const RawResidual<NV>& r, float (&z)[NV]) {
  const bool whole = col + NV <= N;
  auto half = [&](unsigned w) { return (float)__builtin_bit_cast(v2h, w).x; };
  switch (e.res_kind) {  // the same for the whole launch
    case 0:
#pragma unroll
      for (int t = 0; t < NV; ++t)
        if (whole || col + t < N) z[t] += __uint_as_float(r.w[t]);
      break;
    case 1:
#pragma unroll
      for (int t = 0; t < NV; ++t) {
        const unsigned w = whole ? (t & 1 ? r.w[t / 2] & 0xFFFF0000u : r.w[t / 2] << 16) : r.w[t] << 16;
        if (whole || col + t < N) z[t] += __uint_as_float(w);
      }
      break;
    case 2:
#pragma unroll
      for (int t = 0; t < NV; ++t) {
        const unsigned w = whole ? (t & 1 ? r.w[t / 2] >> 16 : r.w[t / 2]) : r.w[t];
        if (whole || col + t < N) z[t] += half(w);
      }
      break;
    default: break;
  }
}

// The bias of NV columns from col on (zero without a bias and past N - 1).
template <int NV>
__device__ __forceinline__ void load_bias(const EpiArgs& e, int col, int N, float (&b)[NV]) {
#pragma unroll
  for (int t = 0; t < NV; ++t) b[t] = e.bias && col + t < N ? e.bias[col + t] : 0.0f;
}

template <int NV, bool ONCE>
__device__ __forceinline__ void store_bf16(uint16_t* base, int64_t row, int col, int N, const float (&f)[NV]) {
  uint16_t* dst = base + row * N + col;
  unsigned w[NV / 2];
#pragma unroll
  for (int t = 0; t < NV / 2; ++t) w[t] = bf16_bits(f[2 * t]) | ((unsigned)bf16_bits(f[2 * t + 1]) << 16);
  if (col + NV <= N) {
    if constexpr (NV == 8 && ONCE)
      __builtin_nontemporal_store((v4u_at2){w[0], w[1], w[2], w[3]}, reinterpret_cast<v4u_at2*>(dst));
    else if constexpr (NV == 8) *reinterpret_cast<v4u_at2*>(dst) = (v4u){w[0], w[1], w[2], w[3]};
    else *reinterpret_cast<v2u_at2*>(dst) = (v2u_at2){w[0], w[1]};
  } else {
#pragma unroll
    for (int t = 0; t < NV; ++t)
      if (col + t < N) dst[t] = (uint16_t)(w[t >> 1] >> (16 * (t & 1)));
  }
}

// pre and out of NV outputs from their products c, bias b and residual r.
template <int NV, bool ONCE = false>
__device__ __forceinline__ void residual_store(const EpiArgs& e, int64_t row, int col, int N, const float (&c)[NV],
                                               const float (&b)[NV], const RawResidual<NV>& r) {
  float z[NV];
#pragma unroll
  for (int t = 0; t < NV; ++t) z[t] = c[t] + b[t];
  if (e.pre) store_bf16<NV, ONCE>(e.pre, row, col, N, z);
  switch (e.act) {  // the same for the whole launch
    case 1:
#pragma unroll
      for (int t = 0; t < NV; ++t) z[t] = act_fn<1>(z[t]);
      break;
    case 2:
#pragma unroll
      for (int t = 0; t < NV; ++t) z[t] = act_fn<2>(z[t]);
      break;
    case 3:
#pragma unroll
      for (int t = 0; t < NV; ++t) z[t] = act_fn<3>(z[t]);
      break;
    case 4:
#pragma unroll
      for (int t = 0; t < NV; ++t) z[t] = act_fn<4>(z[t]);
      break;
    default: break;
  }
  add_residual<NV>(e, col, N, r, z);
  store_bf16<NV, ONCE>(e.out, row, col, N, z);
}

// A tile's epilogue in passes: a pass is GR rows of each wave row's WTM rows
// (the pass's first at `first`), BN columns from n0, in LDS as FP32 (pitch LDF
// floats), stored by all NT threads, ITS rows each. A thread's columns are the
// same in every pass.
template <int BN_, int LDF_, int NT_, int WM_, int WTM_, int GR_, bool ONCE = false>
struct ResidualTile {
  static constexpr int BN = BN_, LDF = LDF_, NT = NT_, WTM = WTM_, GR = GR_;
  static constexpr int RPI = NT / (BN / 8), ITS = WM_ * GR / RPI;
  static_assert(NT % (BN / 8) == 0 && (WM_ * GR) % RPI == 0, "rows split evenly over the threads");

  const EpiArgs& e;
  int m0, n0, M, N;

  __device__ __forceinline__ int col() const { return (threadIdx.x % (BN / 8)) * 8; }
  // the thread's row in LDS and in the output of iteration `it`
  __device__ __forceinline__ int row(int it) const { return it * RPI + (int)threadIdx.x / (BN / 8); }
  __device__ __forceinline__ int64_t out_row(int r, int first) const { return m0 + (r / GR) * WTM + first + r % GR; }

  // The pass's residual: loaded a pass ahead, so that its latency passes
  // behind the pass before it.
  __device__ __forceinline__ void load(int first, RawResidual<8> (&res)[ITS]) const {
#pragma unroll
    for (int it = 0; it < ITS; ++it) {
      const int64_t gr = out_row(row(it), first);
      if (gr < M && n0 + col() < N) load_residual<8, ONCE>(e, gr, n0 + col(), N, res[it]);
    }
  }

  __device__ __forceinline__ void store(const float* tile, int first, const float (&bias)[8], const RawResidual<8> (&res)[ITS]) const {
    const int c = col();
#pragma unroll
    for (int it = 0; it < ITS; ++it) {
      const int r = row(it);
      const int64_t gr = out_row(r, first);
      if (gr >= M || n0 + c >= N) continue;
      const v4f lo = *reinterpret_cast<const v4f*>(tile + r * LDF + c);
      const v4f hi = *reinterpret_cast<const v4f*>(tile + r * LDF + c + 4);
      const float p[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
      residual_store<8, ONCE>(e, gr, n0 + c, N, p, bias, res[it]);
    }
  }
};

}  // namespace dg

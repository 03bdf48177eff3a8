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
// activation and residual type.
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
  int vec;            // 16-byte accesses: bit 0 out, bit 1 pre, bit 2 residual
};

// The residual of NV (4 or 8) outputs from (row, col) on, in FP32; those past
// column N - 1 are zero. row < M and col < N.
template <int NV>
__device__ __forceinline__ void load_residual(const EpiArgs& e, int64_t row, int col, int N, float (&r)[NV]) {
#pragma unroll
  for (int t = 0; t < NV; ++t) r[t] = 0.0f;
  if (e.res_kind == 3) return;
  const int64_t at = row * e.ldres + col;
  if ((e.vec & 4) && col + NV <= N) {
    if (e.res_kind == 0) {
      const v4f* src = reinterpret_cast<const v4f*>(static_cast<const float*>(e.res) + at);
#pragma unroll
      for (int t = 0; t < NV; ++t) r[t] = src[t / 4][t % 4];
    } else {
      unsigned w[NV / 2];
      const uint16_t* src = static_cast<const uint16_t*>(e.res) + at;
      if constexpr (NV == 8) {
        const v4u v = *reinterpret_cast<const v4u*>(src);
#pragma unroll
        for (int t = 0; t < 4; ++t) w[t] = v[t];
      } else {
        const uint2 v = *reinterpret_cast<const uint2*>(src);
        w[0] = v.x;
        w[1] = v.y;
      }
#pragma unroll
      for (int t = 0; t < NV / 2; ++t) {
        const v2h h = __builtin_bit_cast(v2h, w[t]);
        r[2 * t] = e.res_kind == 1 ? __uint_as_float(w[t] << 16) : (float)h.x;
        r[2 * t + 1] = e.res_kind == 1 ? __uint_as_float(w[t] & 0xFFFF0000u) : (float)h.y;
      }
    }
  } else {
#pragma unroll
    for (int t = 0; t < NV; ++t) {
      if (col + t >= N) break;
      if (e.res_kind == 0) r[t] = static_cast<const float*>(e.res)[at + t];
      else if (e.res_kind == 1) r[t] = __uint_as_float((unsigned)static_cast<const uint16_t*>(e.res)[at + t] << 16);
      else r[t] = (float)static_cast<const _Float16*>(e.res)[at + t];
    }
  }
}

// The bias of NV columns from col on (zero without a bias and past N - 1).
template <int NV>
__device__ __forceinline__ void load_bias(const EpiArgs& e, int col, int N, float (&b)[NV]) {
#pragma unroll
  for (int t = 0; t < NV; ++t) b[t] = e.bias && col + t < N ? e.bias[col + t] : 0.0f;
}

template <int NV>
__device__ __forceinline__ void store_bf16(uint16_t* base, bool vec, int64_t row, int col, int N, const float (&f)[NV]) {
  uint16_t* dst = base + row * N + col;
  unsigned w[NV / 2];
#pragma unroll
  for (int t = 0; t < NV / 2; ++t) w[t] = bf16_bits(f[2 * t]) | ((unsigned)bf16_bits(f[2 * t + 1]) << 16);
  if (vec && col + NV <= N) {
    if constexpr (NV == 8) *reinterpret_cast<v4u*>(dst) = (v4u){w[0], w[1], w[2], w[3]};
    else *reinterpret_cast<uint2*>(dst) = make_uint2(w[0], w[1]);
  } else {
#pragma unroll
    for (int t = 0; t < NV; ++t)
      if (col + t < N) dst[t] = (uint16_t)(w[t >> 1] >> (16 * (t & 1)));
  }
}

// pre and out of NV outputs from their products c, bias b and residual r.
template <int NV>
__device__ __forceinline__ void residual_store(const EpiArgs& e, int64_t row, int col, int N, const float (&c)[NV],
                                               const float (&b)[NV], const float (&r)[NV]) {
  float z[NV];
#pragma unroll
  for (int t = 0; t < NV; ++t) z[t] = c[t] + b[t];
  if (e.pre) store_bf16<NV>(e.pre, e.vec & 2, row, col, N, z);
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
#pragma unroll
  for (int t = 0; t < NV; ++t) z[t] += r[t];
  store_bf16<NV>(e.out, e.vec & 1, row, col, N, z);
}

// One pass of a tile's epilogue: the rows that are in LDS as FP32 (pitch LDF
// floats, GR rows of each wave row's WTM, the pass's first at `first`), BN
// columns from n0, by all NT threads. A thread's columns are the same in every
// pass; bias: theirs.
template <int BN, int LDF, int NT, int WM, int WTM, int GR>
__device__ __forceinline__ void residual_pass(const EpiArgs& e, const float* tile, int m0, int n0, int first, int M, int N,
                                              const float (&bias)[8]) {
  constexpr int RPI = NT / (BN / 8), ITS = WM * GR / RPI;
  static_assert(NT % (BN / 8) == 0 && (WM * GR) % RPI == 0, "rows split evenly over the threads");
  const int c = (threadIdx.x % (BN / 8)) * 8, r0 = threadIdx.x / (BN / 8);
  if (n0 + c >= N) return;
#pragma unroll
  for (int it = 0; it < ITS; ++it) {
    const int r = it * RPI + r0;
    const int64_t gr = m0 + (r / GR) * WTM + first + r % GR;
    if (gr >= M) continue;
    const v4f lo = *reinterpret_cast<const v4f*>(tile + r * LDF + c);
    const v4f hi = *reinterpret_cast<const v4f*>(tile + r * LDF + c + 4);
    const float p[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
    float res[8];
    load_residual<8>(e, gr, n0 + c, N, res);
    residual_store<8>(e, gr, n0 + c, N, p, bias, res);
  }
}

}  // namespace dg

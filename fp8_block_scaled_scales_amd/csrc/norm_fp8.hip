// Root-mean-square norm with the residual's addition and FP8 output, and its
// backward pass, for gfx950.
//
// Forward, per row of `cols` elements (all in FP32 unless said otherwise):
//   h    = round(x + residual) to the residual's type (no residual: h = x);
//          the norm is of the stream as it is stored, so a later reader of h
//          sees the values that were normed
//   rstd = 1 / sqrt(mean(h^2) + eps)
//   y    = (h * rstd) * w
//   per g-wide segment: scale = amax|y| / fmax, q = FP8(y / scale) by the
//          quantiser's rule (quant_common.h), from the FP32 y: the one
//          rounding on the way to the codes is the codes' own
// and, where a backward pass will need them, y in x's type and rstd.
//
// Backward, with n = h * rstd, u = dy * w:
//   dx = rstd * (u - n * mean(u * n)) + dh,  dw = sum over rows of dy * n
// (dh the gradient that reaches the stream past the norm; dx is the gradient
// of x and of the residual alike).
//
// Both are bound by HBM: 8 to 12 operations per element against 3 (BF16 without a
// residual) to 17 bytes (FP32 with residual and y). A row stays in registers
// between its reduction and its use, so each input is read once: 8192 x 8192 in
// BF16 takes 98 us forward with y (606 MB, 6.2 TB/s) and 90 us backward (537 MB,
// 5.9 TB/s, the addition of the partial rows included), 2000 x 16384 with an FP32
// stream 62.6 (5.8 TB/s) and 88.2 us (5.2 TB/s), where a copy reaches 5.9 TB/s;
// one row of 7168 takes 3.0 us, 64 rows backward 3.4 us.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "layer_ops.h"
#include "quant_common.h"

// Fused multiply-adds are written out, so that a row's result does not depend on
// which of the kernels below its call takes (the row's sum has one order for
// each row length up to the longest that registers hold).
#pragma clang fp contract(off)

namespace dg {

namespace {

// Sum over the RT threads that share a row, in every one of them: RT = 64 is
// one wave; else the waves meet through LDS (red: RT / 64 floats of the row's
// own, free again after the workgroup's next barrier), added in wave order. t:
// the thread's place in its row.
template <int RT>
__device__ __forceinline__ float row_sum(float v, float* red, int t) {
  v = wave_sum(v);
  if constexpr (RT > 64) {
    DG_STEP_SYNC_WG();
    if ((t & 63) == 0) red[t >> 6] = v;
    __syncthreads();
    v = red[0];
#pragma unroll
    for (int i = 1; i < RT / 64; ++i) v += red[i];
    DG_STEP_SYNC_WG();
  }
  return v;
}

template <int K, int E>
__device__ __forceinline__ float sum_sq(const Raw<K, E>& r, float s) {
  float f[E];
  widen_raw(r, f);
#pragma unroll
  for (int i = 0; i < E; ++i) s = __builtin_fmaf(f[i], f[i], s);
  return s;
}

// h's elements from ex of x and er of the residual on, in h's kind.
template <int XK, int RK, int E, bool ONCE = false>
__device__ __forceinline__ Raw<RK == kAbsent ? XK : RK, E> stream_of(const NormArgs& p, int64_t ex, int64_t er) {
  const Raw<XK, E> x = load_raw<XK, E, ONCE>(p.x, ex);
  if constexpr (RK == kAbsent) {
    return x;
  } else {
    float a[E], b[E];
    widen_raw(x, a);
    widen_raw(load_raw<RK, E, ONCE>(p.res, er), b);
#pragma unroll
    for (int i = 0; i < E; ++i) a[i] += b[i];
    return round_raw<RK>(a);
  }
}

template <int E>
__device__ __forceinline__ void load_w(const float* w, int c, float (&f)[E]) {
  widen_raw(load_raw<0, E>(w, c), f);
}

// The outputs of E elements of row `row` from column c on: segments are whole
// lane groups (segment_max), so every lane of a group comes here.
template <int XK, int HK, int E, bool ONCE = false>
__device__ __forceinline__ void emit(const NormArgs& p, const Raw<HK, E>& h, float rstd, int64_t row, int c) {
  float y[E], w[E];
  load_w(p.w, c, w);
  widen_raw(h, y);
#pragma unroll
  for (int i = 0; i < E; ++i) y[i] = y[i] * rstd * w[i];
  const float amax = segment_max<E>(amax_of(y), p.gran);
  const float s = block_scale(amax, format_max(p.fmt));
  const int64_t e = row * p.cols + c;
  store_codes<ONCE>(p.q + e, y, s, 1.0f / s, p.fmt);
  if ((c & (p.gran - 1)) == 0) p.scales[row * p.segs + (c >> p.gshift)] = s;
  if (p.y) store_raw<ONCE>(p.y, e, round_raw<XK>(y));
}

constexpr int unit_of_norm(int xk, int rk) { return unit_of(xk, rk == kAbsent ? xk : rk); }

// RT threads per row, 8 C elements per thread (RT * C * 8 >= cols) in units of E
// elements.
template <int XK, int RK, int RT, int C, bool ONCE>
__global__ __launch_bounds__(RT < 256 ? 256 : RT) void rmsnorm_quant(const NormArgs p) {
  constexpr int HK = RK == kAbsent ? XK : RK, E = unit_of_norm(XK, RK), U = 8 * C / E;
  constexpr int ROWS = RT < 256 ? 256 / RT : 1;
  __shared__ float red[ROWS][RT / 64];
  const int t = threadIdx.x % RT, team = threadIdx.x / RT;
  const int64_t row = p.row0 + (int64_t)blockIdx.x * ROWS + team;
  if (RT == 64 && row >= p.rows) return;  // whole waves, and no barrier follows
  const int units = row < p.rows ? (int)(p.cols / E) : 0;  // a team past the last row only meets the barrier
  Raw<HK, E> h[U];
  float ss = 0.0f;
#pragma unroll
  for (int i = 0; i < U; ++i) {
    const int c = E * (i * RT + t);
    if (i * RT + t < units) h[i] = stream_of<XK, RK, E, ONCE>(p, row * p.ldx + c, row * p.ldres + c);
  }
#pragma unroll
  for (int i = 0; i < U; ++i) {
    if (i * RT + t < units) {
      ss = sum_sq(h[i], ss);
      if (RK != kAbsent) store_raw<ONCE>(p.h, row * p.cols + E * (i * RT + t), h[i]);
    }
  }
  ss = row_sum<RT>(ss, red[team], t);
  const float rstd = 1.0f / sqrtf(ss / (float)p.cols + p.eps);
  if (p.rstd && t == 0 && units) p.rstd[row] = rstd;
#pragma unroll
  for (int i = 0; i < U; ++i)
    if (i * RT + t < units) emit<XK, HK, E, ONCE>(p, h[i], rstd, row, E * (i * RT + t));
}

// Rows longer than the registers of a workgroup hold: the row is read twice,
// the second time mostly from L2 (as stored in h where there is a residual:
// each thread reads what it wrote itself).
template <int XK, int RK>
__global__ __launch_bounds__(1024) void rmsnorm_quant_long(const NormArgs p) {
  constexpr int HK = RK == kAbsent ? XK : RK, RT = 1024, E = unit_of_norm(XK, RK);
  __shared__ float red[RT / 64];
  const int64_t row = p.row0 + blockIdx.x;
  const int units = (int)(p.cols / E);
  float ss = 0.0f;
  for (int u = threadIdx.x; u < units; u += RT) {
    const Raw<HK, E> h = stream_of<XK, RK, E>(p, row * p.ldx + E * u, row * p.ldres + E * u);
    ss = sum_sq(h, ss);
    if (RK != kAbsent) store_raw(p.h, row * p.cols + E * u, h);
  }
  ss = row_sum<RT>(ss, red, (int)threadIdx.x);
  const float rstd = 1.0f / sqrtf(ss / (float)p.cols + p.eps);
  if (p.rstd && threadIdx.x == 0) p.rstd[row] = rstd;
  for (int u = threadIdx.x; u < units; u += RT) {
    const Raw<HK, E> h =
        RK == kAbsent ? load_raw<HK, E>(p.x, row * p.ldx + E * u) : load_raw<HK, E>(p.h, row * p.cols + E * u);
    emit<XK, HK, E>(p, h, rstd, row, E * u);
  }
}

// One launch, or several where a grid's threads would pass 2^32 - 1; `wg_rows`
// rows per workgroup of NT threads.
template <int NT, class K, class Args>
hipError_t launch_by_rows(K kernel, const Args& p, int wg_rows, hipStream_t stream) {
  const int64_t most = 0xffffffffll / NT;
  for (int64_t r0 = 0; r0 < p.rows; r0 += most * wg_rows) {
    Args q = p;
    q.row0 = r0;
    const int64_t wgs = std::min<int64_t>(most, (p.rows - r0 + wg_rows - 1) / wg_rows);
    hipLaunchKernelGGL(kernel, dim3((unsigned)wgs), dim3(NT), 0, stream, q);
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
  }
  return hipSuccess;
}

template <int XK, int RK, int RT, int C>
hipError_t launch_rows(const NormArgs& p, hipStream_t stream) {
  constexpr int ROWS = RT < 256 ? 256 / RT : 1, NT = RT * ROWS;
  // kOnceBytes: 8192x8192 in BF16 85.6 -> 81.4 us nontemporally, 2622x14976
  // (training) 69.9 -> 59.7, 4000x16384 85.0 -> 78.6; 300x4096 4.3 -> 4.5
  if (p.rows * p.cols * (InKind<XK>::kBytes + (RK == kAbsent ? 0 : InKind<RK % kAbsent>::kBytes)) >= kOnceBytes)
    return launch_by_rows<NT>(rmsnorm_quant<XK, RK, RT, C, true>, p, ROWS, stream);
  return launch_by_rows<NT>(rmsnorm_quant<XK, RK, RT, C, false>, p, ROWS, stream);
}

// Threads per row: one chunk each as long as 1024 reach, which leaves the
// fewest bytes waiting at each row's barrier and gives a single row the most
// lanes. Two or four chunks per thread: 8192x2048 23.2 -> 25.6 and 30.2 us,
// 8192x8192 (training) 105 -> 110 and 120, one row of 7168 3.2 -> 3.6 and 4.8;
// half of the lanes idle: 4096x4096 24.2 -> 30.0, 8192x1024 12.1 -> 13.3.
template <int XK, int RK>
hipError_t launch_norm_k(const NormArgs& p, hipStream_t stream) {
  if (p.cols <= 512) return launch_rows<XK, RK, 64, 1>(p, stream);
  if (p.cols <= 1024) return launch_rows<XK, RK, 128, 1>(p, stream);
  if (p.cols <= 2048) return launch_rows<XK, RK, 256, 1>(p, stream);
  if (p.cols <= 4096) return launch_rows<XK, RK, 512, 1>(p, stream);
  if (p.cols <= 8192) return launch_rows<XK, RK, 1024, 1>(p, stream);
  if (p.cols <= 16384) return launch_rows<XK, RK, 1024, 2>(p, stream);
  if (p.cols <= 32768) return launch_rows<XK, RK, 1024, 4>(p, stream);
  return launch_by_rows<1024>(rmsnorm_quant_long<XK, RK>, p, 1, stream);
}

template <int XK>
hipError_t launch_norm_x(const NormArgs& p, hipStream_t stream) {
  switch (p.rk) {
    case 0: return launch_norm_k<XK, 0>(p, stream);
    case 1: return launch_norm_k<XK, 1>(p, stream);
    case 2: return launch_norm_k<XK, 2>(p, stream);
    case kAbsent: return launch_norm_k<XK, kAbsent>(p, stream);
    default: return hipErrorInvalidValue;
  }
}

// ---- backward -----------------------------------------------------------------

// s plus u * n of E elements, one after the other.
template <int DK, int HK, int E>
__device__ __forceinline__ float row_part(const Raw<DK, E>& dy, const Raw<HK, E>& h, const float (&w)[E], float rstd, float s) {
  float g[E], n[E];
  widen_raw(dy, g);
  widen_raw(h, n);
#pragma unroll
  for (int k = 0; k < E; ++k) s = __builtin_fmaf(g[k] * w[k], n[k] * rstd, s);
  return s;
}

// dx of E elements from the row's mean of u * n.
template <bool ONCE = false, int DK, int HK, int E>
__device__ __forceinline__ void store_dx(const NormBwdArgs& p, const Raw<DK, E>& dy, const Raw<HK, E>& h, const Raw<HK, E>& dh,
                                         const float (&w)[E], float rstd, float mean, int64_t e) {
  float g[E], n[E], d[E];
  widen_raw(dy, g);
  widen_raw(h, n);
  widen_raw(dh, d);
#pragma unroll
  for (int k = 0; k < E; ++k) d[k] = __builtin_fmaf(rstd, __builtin_fmaf(-(n[k] * rstd), mean, g[k] * w[k]), d[k]);
  store_raw<ONCE>(p.dx, e, round_raw<HK>(d));
}

template <int HK, int E, bool ONCE = false>
__device__ __forceinline__ Raw<HK, E> load_dh(const NormBwdArgs& p, int64_t row, int c) {
  return p.dh ? load_raw<HK, E, ONCE>(p.dh, row * p.lddh + c) : Raw<HK, E>{};
}

// Few rows, one launch and no workspace: the first `col_wgs` workgroups add
// dy * n over all rows, 64 columns each (eight lanes of eight columns, 128 rows
// at a time, their sums added through LDS in a fixed order); the others take a
// row per RT threads. dy and h are read twice, the second time from L2.
template <int DK, int HK, int RT, int C>
__global__ __launch_bounds__(1024) void rmsnorm_bwd_few(const NormBwdArgs p, int col_wgs) {
  constexpr int NT = 1024, ROWS = NT / RT, CL = 8, RL = NT / CL;
  __shared__ float red[RL][8 * CL];
  if ((int)blockIdx.x < col_wgs) {
    const int rl = threadIdx.x / CL, c = (blockIdx.x * CL + threadIdx.x % CL) * 8;
    float acc[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) acc[k] = 0.0f;
#pragma unroll 4
    for (int64_t r = rl; r < p.rows; r += RL) {
      float g[8], h[8];
      widen_raw(load_raw<DK, 8>(p.dy, r * p.lddy + c), g);
      widen_raw(load_raw<HK, 8>(p.h, r * p.ldh + c), h);
      const float rstd = p.rstd[r];
#pragma unroll
      for (int k = 0; k < 8; ++k) acc[k] = __builtin_fmaf(g[k], h[k] * rstd, acc[k]);
    }
    column_sums_of_lanes<RL, CL>(acc, red, p.dw + blockIdx.x * (8 * CL));
    return;
  }
  const int t = threadIdx.x % RT, team = threadIdx.x / RT;
  const int64_t row = (int64_t)(blockIdx.x - col_wgs) * ROWS + team;
  constexpr int E = unit_of(DK, HK), U = 8 * C / E;
  const int units = row < p.rows ? (int)(p.cols / E) : 0;  // a team past the last row only meets the barrier
  const float rstd = units ? p.rstd[row] : 0.0f;
  Raw<DK, E> dy[U];
  Raw<HK, E> h[U], dh[U];
  float w[U][E], s = 0.0f;
#pragma unroll
  for (int i = 0; i < U; ++i) {
    const int c = E * (i * RT + t);
    if (i * RT + t < units) {
      dy[i] = load_raw<DK, E>(p.dy, row * p.lddy + c);
      h[i] = load_raw<HK, E>(p.h, row * p.ldh + c);
      dh[i] = load_dh<HK, E>(p, row, c);
      load_w(p.w, c, w[i]);
    }
  }
#pragma unroll
  for (int i = 0; i < U; ++i)
    if (i * RT + t < units) s = row_part(dy[i], h[i], w[i], rstd, s);
  s = row_sum<RT>(s, &red[0][0] + team * (RT / 64), t) / (float)p.cols;
#pragma unroll
  for (int i = 0; i < U; ++i)
    if (i * RT + t < units) store_dx(p, dy[i], h[i], dh[i], w[i], rstd, s, row * p.cols + E * (i * RT + t));
}

// Many rows: every team of RT threads takes rows team, team + teams, ...; its
// threads keep the same columns throughout, so w and the columns' sums of dy * n
// stay in registers and every input is read once. The next row is loaded
// before this row's reduction; two chunks per thread of FP32 rows do not all
// fit 128 registers, so there dh is loaded with its own row and, where dy is
// FP32 too, h as well, and w is read again for every row (from L2). A workgroup writes its
// columns' sums as one partial row (its four teams' added through LDS where
// RT = 64).
template <int DK, int HK, int RT, int C, bool ONCE>
__global__ __launch_bounds__(RT < 256 ? 256 : RT) void rmsnorm_bwd_many(const NormBwdArgs p) {
  constexpr int NT = RT < 256 ? 256 : RT, TEAMS = NT / RT;
  __shared__ float red[2][RT / 64];
  __shared__ float sums[TEAMS > 1 ? TEAMS : 1][TEAMS > 1 ? 512 : 1];
  constexpr int E = unit_of(DK, HK), U = 8 * C / E;
  constexpr int BYTES = InKind<DK>::kBytes + 2 * InKind<HK>::kBytes;
  constexpr bool DH_AHEAD = C == 1 || BYTES <= 6, KEEP_W = C == 1 || BYTES <= 10, H_AHEAD = KEEP_W;
  const int t = threadIdx.x % RT, team = threadIdx.x / RT;
  const int64_t teams = (int64_t)gridDim.x * TEAMS;
  const int units = (int)(p.cols / E);
  float w[U][E], acc[U][E];
  Raw<DK, E> dy[U];
  Raw<HK, E> h[U], dh[U];
  float rstd = 0.0f;
  auto load_row = [&](int64_t row, Raw<DK, E>(&dy)[U], Raw<HK, E>(&h)[U], Raw<HK, E>(&dh)[U], float& rstd) {
    rstd = p.rstd[row];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int c = E * (i * RT + t);
      if (i * RT + t < units) {
        dy[i] = load_raw<DK, E, ONCE>(p.dy, row * p.lddy + c);
        if (H_AHEAD) h[i] = load_raw<HK, E, ONCE>(p.h, row * p.ldh + c);
        if (DH_AHEAD) dh[i] = load_dh<HK, E, ONCE>(p, row, c);
      }
    }
  };
  int64_t row = (int64_t)blockIdx.x * TEAMS + team;
  if (row < p.rows) load_row(row, dy, h, dh, rstd);
#pragma unroll
  for (int i = 0; i < U; ++i) {
#pragma unroll
    for (int k = 0; k < E; ++k) acc[i][k] = 0.0f;
    if (KEEP_W && i * RT + t < units) load_w(p.w, E * (i * RT + t), w[i]);
  }
  for (int it = 0; row < p.rows; row += teams, ++it) {
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int c = E * (i * RT + t);
      if (i * RT + t < units) {
        if (!KEEP_W) load_w(p.w, c, w[i]);
        if (!H_AHEAD) h[i] = load_raw<HK, E, ONCE>(p.h, row * p.ldh + c);
        if (!DH_AHEAD) dh[i] = load_dh<HK, E, ONCE>(p, row, c);
        float g[E], n[E];
        widen_raw(dy[i], g);
        widen_raw(h[i], n);
#pragma unroll
        for (int k = 0; k < E; ++k) {
          n[k] *= rstd;
          s = __builtin_fmaf(g[k] * w[i][k], n[k], s);
          acc[i][k] = __builtin_fmaf(g[k], n[k], acc[i][k]);
        }
      }
    }
    Raw<DK, E> dy1[U];
    Raw<HK, E> h1[U], dh1[U];
    float rstd1 = 0.0f;
    const bool more = row + teams < p.rows;
    if (more) load_row(row + teams, dy1, h1, dh1, rstd1);
    // two areas in turn: a wave writes one again only after the other's barrier
    s = row_sum<RT>(s, red[it & 1], t) / (float)p.cols;
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int c = E * (i * RT + t);
      if (i * RT + t < units) {
        if (!KEEP_W) load_w(p.w, c, w[i]);
        store_dx<ONCE>(p, dy[i], h[i], dh[i], w[i], rstd, s, row * p.cols + c);
      }
    }
    if (more) {
#pragma unroll
      for (int i = 0; i < U; ++i) {
        dy[i] = dy1[i];
        if (H_AHEAD) h[i] = h1[i];
        if (DH_AHEAD) dh[i] = dh1[i];
      }
      rstd = rstd1;
    }
  }
  float* const part = p.ws + (int64_t)blockIdx.x * p.cols;
  if constexpr (TEAMS > 1) {
    static_assert(C == 1 && RT * 8 <= 512, "a team's columns fit its row of sums");
#pragma unroll
    for (int i = 0; i < U; ++i)
      if (i * RT + t < units) {
#pragma unroll
        for (int k = 0; k < E; ++k) sums[team][E * (i * RT + t) + k] = acc[i][k];
      }
    __syncthreads();
    DG_STEP_SYNC_WG();
    for (int c = threadIdx.x; c < (int)p.cols; c += NT) {
      float v = sums[0][c];
#pragma unroll
      for (int i = 1; i < TEAMS; ++i) v += sums[i][c];
      part[c] = v;
    }
  } else {
#pragma unroll
    for (int i = 0; i < U; ++i)
      if (i * RT + t < units) store_raw(part, E * (i * RT + t), round_raw<0>(acc[i]));
  }
}

// Rows longer than the registers of a workgroup hold: dx with the row read
// twice, the columns' sums by rmsnorm_bwd_cols.
template <int DK, int HK>
__global__ __launch_bounds__(1024) void rmsnorm_bwd_rows_long(const NormBwdArgs p) {
  constexpr int RT = 1024, E = unit_of(DK, HK);
  __shared__ float red[RT / 64];
  const int64_t row = p.row0 + blockIdx.x;
  const int units = (int)(p.cols / E);
  const float rstd = p.rstd[row];
  float s = 0.0f;
  for (int u = threadIdx.x; u < units; u += RT) {
    float w[E];
    load_w(p.w, E * u, w);
    s = row_part(load_raw<DK, E>(p.dy, row * p.lddy + E * u), load_raw<HK, E>(p.h, row * p.ldh + E * u), w, rstd, s);
  }
  s = row_sum<RT>(s, red, (int)threadIdx.x) / (float)p.cols;
  for (int u = threadIdx.x; u < units; u += RT) {
    float w[E];
    load_w(p.w, E * u, w);
    store_dx(p, load_raw<DK, E>(p.dy, row * p.lddy + E * u), load_raw<HK, E>(p.h, row * p.ldh + E * u),
             load_dh<HK, E>(p, row, E * u), w, rstd, s, row * p.cols + E * u);
  }
}

// Column sums of dy * n over a range of rows, 512 columns per workgroup: 64
// lanes of eight columns, four waves taking the range's rows in turn, their
// sums added through LDS in wave order.
template <int DK, int HK>
__global__ __launch_bounds__(256) void rmsnorm_bwd_cols(const NormBwdArgs p, float* out, int col_groups, int ranges) {
  __shared__ float red[4][512];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int cg = blockIdx.x % col_groups, rr = blockIdx.x / col_groups;
  const int64_t c = (int64_t)cg * 512 + lane * 8;
  const int64_t r0 = p.rows * rr / ranges, r1 = p.rows * (rr + 1) / ranges;
  float acc[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) acc[k] = 0.0f;
  if (c < p.cols) {
    for (int64_t r = r0 + wave; r < r1; r += 4) {
      float g[8], h[8];
      widen_raw(load_raw<DK, 8>(p.dy, r * p.lddy + c), g);
      widen_raw(load_raw<HK, 8>(p.h, r * p.ldh + c), h);
      const float rstd = p.rstd[r];
#pragma unroll
      for (int k = 0; k < 8; ++k) acc[k] = __builtin_fmaf(g[k], h[k] * rstd, acc[k]);
    }
  }
#pragma unroll
  for (int k = 0; k < 8; ++k) red[wave][lane * 8 + k] = acc[k];
  __syncthreads();
  DG_STEP_SYNC_WG();
  for (int i = threadIdx.x; i < 512; i += 256) {
    const int64_t col = (int64_t)cg * 512 + i;
    if (col < p.cols) out[rr * p.cols + col] = ((red[0][i] + red[1][i]) + red[2][i]) + red[3][i];
  }
}

// The backward pass's form and its number of partial rows of dw.
constexpr int64_t kLongCols = 16384;  // what rmsnorm_bwd_many holds
// Few rows: up to 2048 of them and 6M elements (dy and h then stay in the L2s
// between their two readings) rmsnorm_bwd_few's one launch beats two: 139x1216
// 2.9 us against 6.0, 512x4096 6.7 against 9.8, 1024x2048 7.6 against 10.0;
// 2000x2048 13.3 against 13.2, 1024x8192 17.8 against 17.4, 1024x16384 39.6
// against 33.6 (BF16; two launches with kTeamRows).
constexpr int64_t kFewRows = 2048, kFewElements = 6ll << 20;

// Rows that a team takes at least, so that the partial rows stay few beside the
// rows: 2000x2048 15.5 us at one, 13.2 at four, 12.6 at eight; 3022x768 11.9,
// 11.4 and 12.8.
constexpr int64_t kTeamRows = 4;

struct BwdPlan {
  bool few;
  int rt;           // threads per row
  int64_t partial;  // partial rows (one: the sums go straight to dw)
};

BwdPlan bwd_plan(int64_t rows, int64_t cols) {
  BwdPlan b;
  b.rt = cols <= 512 ? 64 : cols <= 2048 ? 256 : cols <= 4096 ? 512 : 1024;
  b.few = cols <= kLongCols && rows <= kFewRows && rows * cols <= kFewElements;
  if (b.few) {
    b.partial = 1;
  } else if (cols <= kLongCols) {
    // 1024 threads per CU
    const int64_t wg_rows = b.rt < 256 ? 256 / b.rt : 1, wgs = 256 * (1024 / (b.rt < 256 ? 256 : b.rt));
    b.partial = std::min<int64_t>((rows + wg_rows * kTeamRows - 1) / (wg_rows * kTeamRows), wgs);
  } else {
    // about 1024 workgroups of rmsnorm_bwd_cols, at least 16 rows each
    b.partial = std::max<int64_t>(1, std::min<int64_t>(1024 / ((cols + 511) / 512), (rows + 15) / 16));
  }
  return b;
}

template <int DK, int HK, int RT, int C>
void launch_bwd(const NormBwdArgs& p, const BwdPlan& b, hipStream_t stream) {
  if (b.few) {
    constexpr int ROWS = 1024 / RT;
    const int col_wgs = (int)(p.cols / 64);
    hipLaunchKernelGGL((rmsnorm_bwd_few<DK, HK, RT, C>), dim3((unsigned)(col_wgs + (p.rows + ROWS - 1) / ROWS)), dim3(1024), 0,
                       stream, p, col_wgs);
  } else {
    // From 128 MB of inputs on nontemporally: 8192x8192 in BF16 100.8 -> 90.6 us,
    // 7459x5376 64.8 -> 61.7, 2000x16384 with an FP32 stream 96.4 -> 92.7 (967x9600
    // with one, 93 MB: 32.1 -> 33.9); not where w is read for every row (FP32 dy
    // and stream, 2000x16384: 111 -> 118).
    constexpr bool W_AGAIN = C > 1 && DK == 0 && HK == 0;
    const dim3 grid((unsigned)b.partial), block(RT < 256 ? 256 : RT);
    const int64_t bytes = p.rows * p.cols * (InKind<DK>::kBytes + (p.dh ? 2 : 1) * InKind<HK>::kBytes);
    if (!W_AGAIN && bytes >= 2 * kOnceBytes)
      hipLaunchKernelGGL((rmsnorm_bwd_many<DK, HK, RT, C, !W_AGAIN>), grid, block, 0, stream, p);
    else
      hipLaunchKernelGGL((rmsnorm_bwd_many<DK, HK, RT, C, false>), grid, block, 0, stream, p);
  }
}

template <int DK, int HK>
hipError_t launch_norm_bwd_k(const NormBwdArgs& p, hipStream_t stream) {
  const BwdPlan b = bwd_plan(p.rows, p.cols);
  NormBwdArgs q = p;
  const bool direct = b.partial == 1;
  if (direct) q.ws = p.dw;  // one partial row is dw itself
  if (p.cols > kLongCols) {
    const int64_t col_groups = (p.cols + 511) / 512;
    hipLaunchKernelGGL((rmsnorm_bwd_cols<DK, HK>), dim3((unsigned)(col_groups * b.partial)), dim3(256), 0, stream, q, q.ws,
                       (int)col_groups, (int)b.partial);
    const hipError_t err = launch_by_rows<1024>(rmsnorm_bwd_rows_long<DK, HK>, q, 1, stream);
    if (err != hipSuccess) return err;
  } else if (b.rt == 64) {
    launch_bwd<DK, HK, 64, 1>(q, b, stream);
  } else if (b.rt == 256) {
    launch_bwd<DK, HK, 256, 1>(q, b, stream);
  } else if (b.rt == 512) {
    launch_bwd<DK, HK, 512, 1>(q, b, stream);
  } else if (p.cols <= 8192) {
    launch_bwd<DK, HK, 1024, 1>(q, b, stream);
  } else {
    launch_bwd<DK, HK, 1024, 2>(q, b, stream);
  }
  const hipError_t err = hipGetLastError();
  if (err != hipSuccess || direct) return err;
  return launch_column_sum(p.ws, b.partial, p.cols, p.dw, stream);
}

template <int DK>
hipError_t launch_norm_bwd_d(const NormBwdArgs& p, hipStream_t stream) {
  switch (p.hk) {
    case 0: return launch_norm_bwd_k<DK, 0>(p, stream);
    case 1: return launch_norm_bwd_k<DK, 1>(p, stream);
    case 2: return launch_norm_bwd_k<DK, 2>(p, stream);
    default: return hipErrorInvalidValue;
  }
}

// CL lanes of four columns per workgroup, 1024 / CL groups of lanes taking the
// partial rows in turn (eight loads in flight each), then added over the wave's
// groups by shuffles and over the 16 waves through LDS, in order.
template <int CL>
__global__ __launch_bounds__(1024) void column_sum(const float* __restrict__ part, int64_t n, int64_t cols,
                                                   float* __restrict__ out) {
  __shared__ float red[16][4 * CL];
  const int cl = threadIdx.x % CL, grp = threadIdx.x / CL, wave = threadIdx.x >> 6;
  const float* src = part + (int64_t)blockIdx.x * (4 * CL) + cl * 4;
  v4f s = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 8
  for (int64_t r = grp; r < n; r += 1024 / CL) s += *reinterpret_cast<const v4f*>(src + r * cols);
#pragma unroll
  for (int k = 0; k < 4; ++k) {
#pragma unroll
    for (int d = CL; d < 64; d *= 2) s[k] += __shfl_xor(s[k], d, 64);
    if ((threadIdx.x & 63) < CL) red[wave][cl * 4 + k] = s[k];
  }
  __syncthreads();
  DG_STEP_SYNC_WG();
  if (threadIdx.x < 4 * CL) {
    float v = red[0][threadIdx.x];
#pragma unroll
    for (int i = 1; i < 16; ++i) v += red[i][threadIdx.x];
    out[(int64_t)blockIdx.x * (4 * CL) + threadIdx.x] = v;
  }
}

}  // namespace

// Below 4096 columns 64 of them to a workgroup would leave most CUs idle: with
// 16 the whole backward of 3867 x 768 takes 12.0 us for 13.3, of 30000 x 512
// 28.3 for 29.5; at 4096 columns the wider pieces are ahead (5000 rows: 37.2 for
// 38.3, 2000 x 16384: 88.5 for 92.0).
hipError_t launch_column_sum(const float* part, int64_t n, int64_t cols, float* out, hipStream_t stream) {
  if (cols >= 4096) hipLaunchKernelGGL(column_sum<16>, dim3((unsigned)(cols / 64)), dim3(1024), 0, stream, part, n, cols, out);
  else hipLaunchKernelGGL(column_sum<4>, dim3((unsigned)(cols / 16)), dim3(1024), 0, stream, part, n, cols, out);
  return hipGetLastError();
}

hipError_t launch_norm(const NormArgs& p, hipStream_t stream) {
  switch (p.xk) {
    case 0: return launch_norm_x<0>(p, stream);
    case 1: return launch_norm_x<1>(p, stream);
    case 2: return launch_norm_x<2>(p, stream);
    default: return hipErrorInvalidValue;
  }
}

int64_t norm_bwd_workspace(int64_t rows, int64_t cols) {
  const int64_t n = bwd_plan(rows, cols).partial;
  return n > 1 ? n * cols * (int64_t)sizeof(float) : 0;
}

hipError_t launch_norm_bwd(const NormBwdArgs& p, hipStream_t stream) {
  switch (p.dk) {
    case 0: return launch_norm_bwd_d<0>(p, stream);
    case 1: return launch_norm_bwd_d<1>(p, stream);
    case 2: return launch_norm_bwd_d<2>(p, stream);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace dg

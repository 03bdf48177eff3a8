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
// Both are bound by HBM: 8 to 12 operations per element against 5 to 13
// bytes. A row stays in registers between its reduction and its use, so each
// input is read once.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "layer_ops.h"
#include "quant_common.h"

namespace dg {

namespace {

// Sum over the RT threads that share a row, in every one of them: RT = 64 is
// one wave; else the workgroup's waves meet through LDS (red: RT / 64 floats,
// free again after the next barrier), added in wave order.
template <int RT>
__device__ __forceinline__ float row_sum(float v, float* red) {
  v = wave_sum(v);
  if constexpr (RT > 64) {
    const int t = threadIdx.x;
    if ((t & 63) == 0) red[t >> 6] = v;
    __syncthreads();
    v = red[0];
#pragma unroll
    for (int i = 1; i < RT / 64; ++i) v += red[i];
  }
  return v;
}

template <int K>
__device__ __forceinline__ float sum_sq8(const Raw8<K>& r) {
  float f[8];
  widen8(r, f);
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) s = __builtin_fmaf(f[i], f[i], s);
  return s;
}

// h's eight elements from e_x of x and e_r of the residual, in h's kind.
template <int XK, int RK>
__device__ __forceinline__ Raw8<RK == kAbsent ? XK : RK> stream8(const NormArgs& p, int64_t ex, int64_t er) {
  const Raw8<XK> x = load8<XK>(p.x, ex);
  if constexpr (RK == kAbsent) {
    return x;
  } else {
    float a[8], b[8];
    widen8(x, a);
    widen8(load8<RK>(p.res, er), b);
#pragma unroll
    for (int i = 0; i < 8; ++i) a[i] += b[i];
    return round8<RK>(a);
  }
}

// The outputs of eight elements of row `row` from column c on: segments are
// whole lane groups (segment_max), so every lane of a group comes here.
template <int XK, int HK>
__device__ __forceinline__ void emit8(const NormArgs& p, const Raw8<HK>& h, const float (&w)[8], float rstd, int64_t row,
                                      int c) {
  float y[8];
  widen8(h, y);
#pragma unroll
  for (int i = 0; i < 8; ++i) y[i] = y[i] * rstd * w[i];
  const float amax = segment_max(amax8(y), p.gran);
  const float s = block_scale(amax, format_max(p.fmt));
  const int64_t e = row * p.cols + c;
  *reinterpret_cast<v2i*>(p.q + e) = encode8(y, s, 1.0f / s, p.fmt);
  if ((c & (p.gran - 1)) == 0) p.scales[row * p.segs + (c >> p.gshift)] = s;
  if (p.y) store8<XK>(p.y, e, round8<XK>(y));
}

__device__ __forceinline__ void load_w8(const float* w, int c, float (&f)[8]) { widen8(load8<0>(w, c), f); }

// RT threads per row, C eight-element chunks per thread (RT * C * 8 >= cols).
template <int XK, int RK, int RT, int C>
__global__ __launch_bounds__(RT < 256 ? 256 : RT) void rmsnorm_quant(const NormArgs p) {
  constexpr int HK = RK == kAbsent ? XK : RK;
  constexpr int ROWS = RT < 256 ? 256 / RT : 1;
  __shared__ float red[RT / 64];
  const int t = threadIdx.x % RT;
  const int64_t row = (int64_t)blockIdx.x * ROWS + threadIdx.x / RT;
  if (row >= p.rows) return;  // RT = 64 only: whole waves, and no barrier follows
  const int chunks = (int)(p.cols / 8);
  Raw8<HK> h[C];
  float ss = 0.0f;
#pragma unroll
  for (int i = 0; i < C; ++i) {
    const int ch = i * RT + t;
    if (ch < chunks) h[i] = stream8<XK, RK>(p, row * p.ldx + 8 * ch, row * p.ldres + 8 * ch);
  }
#pragma unroll
  for (int i = 0; i < C; ++i) {
    const int ch = i * RT + t;
    if (ch < chunks) {
      ss += sum_sq8(h[i]);
      if (RK != kAbsent) store8<HK>(p.h, row * p.cols + 8 * ch, h[i]);
    }
  }
  ss = row_sum<RT>(ss, red);
  const float rstd = 1.0f / sqrtf(ss / (float)p.cols + p.eps);
  if (p.rstd && t == 0) p.rstd[row] = rstd;
#pragma unroll
  for (int i = 0; i < C; ++i) {
    const int ch = i * RT + t;
    if (ch < chunks) {
      float w[8];
      load_w8(p.w, 8 * ch, w);
      emit8<XK, HK>(p, h[i], w, rstd, row, 8 * ch);
    }
  }
}

// Rows longer than the registers of a workgroup hold: the row is read twice,
// the second time mostly from L2 (as stored in h where there is a residual:
// each thread reads what it wrote itself).
template <int XK, int RK>
__global__ __launch_bounds__(1024) void rmsnorm_quant_long(const NormArgs p) {
  constexpr int HK = RK == kAbsent ? XK : RK, RT = 1024;
  __shared__ float red[RT / 64];
  const int t = threadIdx.x;
  const int64_t row = blockIdx.x;
  const int chunks = (int)(p.cols / 8);
  float ss = 0.0f;
  for (int ch = t; ch < chunks; ch += RT) {
    const Raw8<HK> h = stream8<XK, RK>(p, row * p.ldx + 8 * ch, row * p.ldres + 8 * ch);
    ss += sum_sq8(h);
    if (RK != kAbsent) store8<HK>(p.h, row * p.cols + 8 * ch, h);
  }
  ss = row_sum<RT>(ss, red);
  const float rstd = 1.0f / sqrtf(ss / (float)p.cols + p.eps);
  if (p.rstd && t == 0) p.rstd[row] = rstd;
  for (int ch = t; ch < chunks; ch += RT) {
    float w[8];
    load_w8(p.w, 8 * ch, w);
    const Raw8<HK> h = RK == kAbsent ? load8<HK>(p.x, row * p.ldx + 8 * ch) : load8<HK>(p.h, row * p.cols + 8 * ch);
    emit8<XK, HK>(p, h, w, rstd, row, 8 * ch);
  }
}

template <int XK, int RK, int RT, int C>
hipError_t launch_rows(const NormArgs& p, hipStream_t stream) {
  constexpr int ROWS = RT < 256 ? 256 / RT : 1;
  hipLaunchKernelGGL((rmsnorm_quant<XK, RK, RT, C>), dim3((unsigned)((p.rows + ROWS - 1) / ROWS)),
                     dim3(RT < 256 ? 256 : RT), 0, stream, p);
  return hipGetLastError();
}

template <int XK, int RK>
hipError_t launch_norm_k(const NormArgs& p, hipStream_t stream) {
  if (p.cols <= 512) return launch_rows<XK, RK, 64, 1>(p, stream);
  if (p.cols <= 2048) return launch_rows<XK, RK, 256, 1>(p, stream);
  if (p.cols <= 8192) return launch_rows<XK, RK, 1024, 1>(p, stream);
  if (p.cols <= 16384) return launch_rows<XK, RK, 1024, 2>(p, stream);
  if (p.cols <= 32768) return launch_rows<XK, RK, 1024, 4>(p, stream);
  hipLaunchKernelGGL((rmsnorm_quant_long<XK, RK>), dim3((unsigned)p.rows), dim3(1024), 0, stream, p);
  return hipGetLastError();
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

// dx of one row per RT threads.
template <int DK, int HK, int RT, int C>
__global__ __launch_bounds__(RT < 256 ? 256 : RT) void rmsnorm_bwd_rows(const NormBwdArgs p) {
  constexpr int ROWS = RT < 256 ? 256 / RT : 1;
  __shared__ float red[RT / 64];
  const int t = threadIdx.x % RT;
  const int64_t row = (int64_t)blockIdx.x * ROWS + threadIdx.x / RT;
  if (row >= p.rows) return;  // RT = 64 only: whole waves, and no barrier follows
  const int chunks = (int)(p.cols / 8);
  const float rstd = p.rstd[row];
  float u[C][8], n[C][8];
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < C; ++i) {
    const int ch = i * RT + t;
    if (ch < chunks) {
      float w[8];
      widen8(load8<DK>(p.dy, row * p.lddy + 8 * ch), u[i]);
      widen8(load8<HK>(p.h, row * p.ldh + 8 * ch), n[i]);
      load_w8(p.w, 8 * ch, w);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        n[i][k] *= rstd;
        u[i][k] *= w[k];
        s = __builtin_fmaf(u[i][k], n[i][k], s);
      }
    }
  }
  s = row_sum<RT>(s, red) / (float)p.cols;
#pragma unroll
  for (int i = 0; i < C; ++i) {
    const int ch = i * RT + t;
    if (ch < chunks) {
      float d[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) d[k] = 0.0f;
      if (p.dh) widen8(load8<HK>(p.dh, row * p.lddh + 8 * ch), d);
#pragma unroll
      for (int k = 0; k < 8; ++k) d[k] = __builtin_fmaf(rstd, u[i][k] - n[i][k] * s, d[k]);
      store8<HK>(p.dx, row * p.cols + 8 * ch, round8<HK>(d));
    }
  }
}

// The same for rows longer than a workgroup's registers, read twice.
template <int DK, int HK>
__global__ __launch_bounds__(1024) void rmsnorm_bwd_rows_long(const NormBwdArgs p) {
  constexpr int RT = 1024;
  __shared__ float red[RT / 64];
  const int64_t row = blockIdx.x;
  const int chunks = (int)(p.cols / 8);
  const float rstd = p.rstd[row];
  float s = 0.0f;
  for (int pass = 0; pass < 2; ++pass) {
    for (int ch = threadIdx.x; ch < chunks; ch += RT) {
      float u[8], n[8], w[8];
      widen8(load8<DK>(p.dy, row * p.lddy + 8 * ch), u);
      widen8(load8<HK>(p.h, row * p.ldh + 8 * ch), n);
      load_w8(p.w, 8 * ch, w);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        n[k] *= rstd;
        u[k] *= w[k];
      }
      if (pass == 0) {
#pragma unroll
        for (int k = 0; k < 8; ++k) s = __builtin_fmaf(u[k], n[k], s);
      } else {
        float d[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) d[k] = 0.0f;
        if (p.dh) widen8(load8<HK>(p.dh, row * p.lddh + 8 * ch), d);
#pragma unroll
        for (int k = 0; k < 8; ++k) d[k] = __builtin_fmaf(rstd, u[k] - n[k] * s, d[k]);
        store8<HK>(p.dx, row * p.cols + 8 * ch, round8<HK>(d));
      }
    }
    if (pass == 0) s = row_sum<RT>(s, red) / (float)p.cols;
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
      widen8(load8<DK>(p.dy, r * p.lddy + c), g);
      widen8(load8<HK>(p.h, r * p.ldh + c), h);
      const float rstd = p.rstd[r];
#pragma unroll
      for (int k = 0; k < 8; ++k) acc[k] = __builtin_fmaf(g[k], h[k] * rstd, acc[k]);
    }
  }
#pragma unroll
  for (int k = 0; k < 8; ++k) red[wave][lane * 8 + k] = acc[k];
  __syncthreads();
  for (int i = threadIdx.x; i < 512; i += 256) {
    const int64_t col = (int64_t)cg * 512 + i;
    if (col < p.cols) out[rr * p.cols + col] = ((red[0][i] + red[1][i]) + red[2][i]) + red[3][i];
  }
}

// Row ranges of the column sums: about 1024 workgroups, at least 16 rows each.
int64_t bwd_ranges(int64_t rows, int64_t cols) {
  const int64_t col_groups = (cols + 511) / 512;
  const int64_t r = 1024 / col_groups, most = (rows + 15) / 16;
  return r < 1 ? 1 : r < most ? r : most;
}

template <int DK, int HK, int RT, int C>
void launch_bwd_rows(const NormBwdArgs& p, hipStream_t stream) {
  constexpr int ROWS = RT < 256 ? 256 / RT : 1;
  hipLaunchKernelGGL((rmsnorm_bwd_rows<DK, HK, RT, C>), dim3((unsigned)((p.rows + ROWS - 1) / ROWS)),
                     dim3(RT < 256 ? 256 : RT), 0, stream, p);
}

template <int DK, int HK>
hipError_t launch_norm_bwd_k(const NormBwdArgs& p, hipStream_t stream) {
  // the column sums first: dx may be written over dh, never over dy or h
  const int64_t ranges = bwd_ranges(p.rows, p.cols), col_groups = (p.cols + 511) / 512;
  hipLaunchKernelGGL((rmsnorm_bwd_cols<DK, HK>), dim3((unsigned)(col_groups * ranges)), dim3(256), 0, stream, p,
                     ranges > 1 ? p.ws : p.dw, (int)col_groups, (int)ranges);
  if (p.cols <= 512) launch_bwd_rows<DK, HK, 64, 1>(p, stream);
  else if (p.cols <= 2048) launch_bwd_rows<DK, HK, 256, 1>(p, stream);
  else if (p.cols <= 8192) launch_bwd_rows<DK, HK, 1024, 1>(p, stream);
  else if (p.cols <= 16384) launch_bwd_rows<DK, HK, 1024, 2>(p, stream);
  else hipLaunchKernelGGL((rmsnorm_bwd_rows_long<DK, HK>), dim3((unsigned)p.rows), dim3(1024), 0, stream, p);
  const hipError_t err = hipGetLastError();
  if (err != hipSuccess || ranges == 1) return err;
  return launch_column_sum(p.ws, ranges, p.cols, p.dw, stream);
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

// 64 columns per workgroup, four groups of 64 threads taking the partial rows
// in turn (eight loads in flight each), then added through LDS in group order.
__global__ __launch_bounds__(256) void column_sum(const float* __restrict__ part, int64_t n, int64_t cols,
                                                  float* __restrict__ out) {
  __shared__ float red[4][64];
  const int lane = threadIdx.x & 63, grp = threadIdx.x >> 6;
  const int64_t c = (int64_t)blockIdx.x * 64 + lane;
  float s = 0.0f;
#pragma unroll 8
  for (int64_t r = grp; r < n; r += 4) s += part[r * cols + c];
  red[grp][lane] = s;
  __syncthreads();
  if (grp == 0) out[c] = ((red[0][lane] + red[1][lane]) + red[2][lane]) + red[3][lane];
}

}  // namespace

hipError_t launch_column_sum(const float* part, int64_t n, int64_t cols, float* out, hipStream_t stream) {
  hipLaunchKernelGGL(column_sum, dim3((unsigned)(cols / 64)), dim3(256), 0, stream, part, n, cols, out);
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
  const int64_t ranges = bwd_ranges(rows, cols);
  return ranges > 1 ? ranges * cols * (int64_t)sizeof(float) : 0;
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

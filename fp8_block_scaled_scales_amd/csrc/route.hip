// Rows to the group that each chose and back (experts, adapters), for gfx950:
//
//   sort      a stable counting sort of the slots (token t's choice j is slot t k
//             + j) by group: where each slot's row is, and which slot a row has
//   rows      FP8 codes and factors of w x in sorted order, every token read once
//   combine   out[t] = res[t] + sum over j of w[t,j] y[position[t,j]]
//   weights   dw[t,j] = <x[t], y[position[t,j]]>
//
// rows and combine are each other's gradients (combine without weights is the
// gradient of the dispatch, rows of dout with the weights that of the combine).
// All are bound by HBM.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "quant_common.h"
#include "route_ops.h"

#pragma clang fp contract(off)

namespace dg {

namespace {

// ---- the sort -----------------------------------------------------------------

constexpr int kMaxGroups = 1024;  // the library's DG_MAX_GROUPS
constexpr int kSortThreads = 1024, kSortWaves = kSortThreads / 64;

// Slots that one workgroup sorts alone; beyond, chunks of at least kChunk slots,
// at most 256 of them, are counted by one launch and placed by a second.
constexpr int64_t kOneSort = 8192, kChunk = 4096;

int64_t sort_chunk(int64_t n) { return std::max<int64_t>(kChunk, ((n + 255) / 256 + 1023) / 1024 * 1024); }

template <class T>
__device__ __forceinline__ int group_of(const T* ids, int64_t i, int64_t end, int groups) {
  if (i >= end) return -1;
  const T v = ids[i];
  return v >= 0 && v < (T)groups ? (int)v : -1;
}

template <class T>
__global__ __launch_bounds__(kSortThreads) void route_count(const SortArgs p) {
  __shared__ int count[kMaxGroups];
  for (int e = threadIdx.x; e < p.groups; e += kSortThreads) count[e] = 0;
  __syncthreads();
  const int64_t first = (int64_t)blockIdx.x * p.per, end = min(first + p.per, p.n);
  const T* ids = static_cast<const T*>(p.ids);
  for (int64_t i = first + threadIdx.x; i < end; i += kSortThreads) {
    const int e = group_of(ids, i, end, p.groups);
    if (e >= 0) atomicAdd(&count[e], 1);  // whole numbers: the same sum in any order
  }
  __syncthreads();
  for (int e = threadIdx.x; e < p.groups; e += kSortThreads) p.hist[(int64_t)blockIdx.x * p.groups + e] = count[e];
}

// One workgroup, or one per chunk after route_count. A wave takes a contiguous
// run of its chunk's slots, 64 at a time: a slot's row is its group's start, the
// group's slots in earlier chunks, earlier waves' runs and earlier steps, and
// those of lower lanes, found by comparing keys bit by bit with ballots.
template <class T>
__global__ __launch_bounds__(kSortThreads) void route_place(const SortArgs p) {
  __shared__ int count[kSortWaves * kMaxGroups];  // [wave][group]: first counts, then the wave's next place
  __shared__ int part_all[kSortThreads], part_before[kSortThreads];
  __shared__ int start[kMaxGroups + 1], fill[kMaxGroups];
  __shared__ int wave_sum_of[kSortWaves];
  const int G = p.groups, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int chunk = blockIdx.x;
  const int64_t first = (int64_t)chunk * p.per, last = min(first + p.per, p.n);
  const int64_t run = ((last - first + kSortWaves - 1) / kSortWaves + 63) / 64 * 64;
  const int64_t lo = min(first + wave * run, last), hi = min(lo + run, last);
  const T* ids = static_cast<const T*>(p.ids);

  for (int i = tid; i < kSortWaves * G; i += kSortThreads) count[i] = 0;
  __syncthreads();
  for (int64_t i = lo + lane; i < hi; i += 64) {
    const int e = group_of(ids, i, hi, G);
    if (e >= 0) atomicAdd(&count[wave * G + e], 1);
  }
  // all chunks' counts, and those of the chunks before: the chunks shared out over the threads that a power of two of groups leaves
  if (p.chunks) {
    const int wide = G <= 1 ? 1 : 1 << (32 - __builtin_clz(G - 1)), parts = kSortThreads / wide;
    const int e = tid % wide;
    int all = 0, before = 0;
    if (e < G) {
#pragma unroll 4
      for (int c = tid / wide; c < p.chunks; c += parts) {
        const int v = p.hist[(int64_t)c * G + e];
        all += v;
        before += c < chunk ? v : 0;
      }
    }
    part_all[tid] = all;
    part_before[tid] = before;
  }
  __syncthreads();
  int total = 0, before = 0;
  if (tid < G) {
    int sum = 0;
#pragma unroll
    for (int w = 0; w < kSortWaves; ++w) {
      const int v = count[w * G + tid];
      count[w * G + tid] = sum;
      sum += v;
    }
    total = sum;
    if (p.chunks) {
      const int wide = G <= 1 ? 1 : 1 << (32 - __builtin_clz(G - 1));
      total = 0;
      for (int i = tid; i < kSortThreads; i += wide) {
        total += part_all[i];
        before += part_before[i];
      }
    }
  }
  // starts: an exclusive scan of the aligned totals
  const int aligned = (total + p.align - 1) / p.align * p.align;
  int upto = aligned;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int v = __shfl_up(upto, d, 64);
    if (lane >= d) upto += v;
  }
  if (lane == 63) wave_sum_of[wave] = upto;
  __syncthreads();
  for (int w = 0; w < wave; ++w) upto += wave_sum_of[w];
  if (tid < G) {
    start[tid] = upto - aligned;
    fill[tid] = upto - aligned + total;  // where the group's rows without a slot begin
    if (tid == G - 1) start[G] = upto;
    for (int w = 0; w < kSortWaves; ++w) count[w * G + tid] += upto - aligned + before;
    if (chunk == 0) {
      p.offsets[tid] = upto - aligned;
      if (tid == G - 1) p.offsets[G] = upto;
    }
  }
  __syncthreads();

  const int bits = 32 - __builtin_clz(G);
  for (int64_t i0 = lo; i0 < hi; i0 += 64) {
    const int64_t i = i0 + lane;
    const int e = group_of(ids, i, hi, G);
    uint64_t same = __ballot(e >= 0);
    for (int b = 0; b < bits; ++b) {
      const bool one = (e >> b) & 1;
      const uint64_t m = __ballot(one);
      same &= one ? m : ~m;
    }
    const int rank = __builtin_popcountll(same & ((1ull << lane) - 1));
    int at = -1;
    if (e >= 0) {
      const int next = count[wave * G + e];
      at = next + rank;
      __builtin_amdgcn_wave_barrier();
      if (rank == 0) count[wave * G + e] = next + __builtin_popcountll(same);
      p.slot[at] = (int)i;
    }
    __builtin_amdgcn_wave_barrier();
    if (i < hi) p.position[i] = at;
  }

  // rows without a slot: -1 between a group's last row and the next group, -2 behind the last
  const int waves = (int)gridDim.x * kSortWaves;
  for (int e = chunk * kSortWaves + wave; e < G; e += waves)
    for (int r = fill[e] + lane; r < start[e + 1]; r += 64) p.slot[r] = -1;
  for (int64_t r = start[G] + (int64_t)chunk * kSortThreads + tid; r < p.rows; r += (int64_t)gridDim.x * kSortThreads)
    p.slot[r] = -2;
}

template <class T>
hipError_t launch_sort_t(const SortArgs& p, hipStream_t stream) {
  if (p.chunks) {
    hipLaunchKernelGGL((route_count<T>), dim3(p.chunks), dim3(kSortThreads), 0, stream, p);
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
  }
  hipLaunchKernelGGL((route_place<T>), dim3(p.chunks ? p.chunks : 1), dim3(kSortThreads), 0, stream, p);
  return hipGetLastError();
}

// ---- rows as FP8 codes --------------------------------------------------------

template <int FMT, int E>
__device__ __forceinline__ void codes_fmt(const float (&y)[E], float s, int (&c)[E / 4]) {
  const bool fast = recip_ok(s);
  const float inv = 1.0f / s;
#pragma unroll
  for (int i = 0; i < E / 4; ++i) {
    const v4f v = {y[4 * i], y[4 * i + 1], y[4 * i + 2], y[4 * i + 3]};
    if (fast) c[i] = encode4<FMT, true>(v, s, inv);
    else c[i] = encode4<FMT, false>(v, s, inv);
  }
}

template <int E>
__device__ __forceinline__ void codes_of(const float (&y)[E], float s, int fmt, int (&c)[E / 4]) {
  if (fmt == 1) codes_fmt<1>(y, s, c);
  else codes_fmt<0>(y, s, c);
}

template <int E>
__device__ __forceinline__ void put_codes(uint8_t* q, const int (&c)[E / 4]) {
  if constexpr (E == 8) *reinterpret_cast<v2i*>(q) = (v2i){c[0], c[1]};
  else *reinterpret_cast<int*>(q) = c[0];
}

// Rows between a group's last and the next group: codes of zero, factors of
// one. A wave looks at 64 rows.
__device__ __forceinline__ void pad_rows(const RouteQuantArgs& p, int64_t wave, int lane) {
  const int64_t r0 = wave * 64;
  const int s = r0 + lane < p.rows ? p.slot[r0 + lane] : -2;
  uint64_t m = __ballot(s == -1);
  const int64_t segs = p.cols / p.gran;
  while (m) {
    const int64_t r = r0 + __builtin_ctzll(m);
    m &= m - 1;
    for (int64_t c = lane * 16; c < p.cols; c += 64 * 16) *reinterpret_cast<v4u*>(p.q + r * p.cols + c) = (v4u){};
    for (int64_t c = lane; c < segs; c += 64) p.scales[r * segs + c] = 1.0f;
  }
}

constexpr int kRowThreads = 256;

// 1 x g: a lane takes E columns of a token and writes their codes to every row
// that the token has.
template <int XK, bool W>
__global__ __launch_bounds__(kRowThreads) void route_rows(const RouteQuantArgs p, int64_t units, unsigned unit_wgs) {
  constexpr int E = unit_of(XK, 1);
  if (blockIdx.x >= unit_wgs) {
    const int64_t wave = (int64_t)(blockIdx.x - unit_wgs) * (kRowThreads / 64) + (threadIdx.x >> 6);
    const int64_t waves = (int64_t)(gridDim.x - unit_wgs) * (kRowThreads / 64);
    for (int64_t w = wave; w * 64 < p.rows; w += waves) pad_rows(p, w, threadIdx.x & 63);
    return;
  }
  const int64_t per = p.cols / E, segs = p.cols / p.gran;
  // whole segments are live or not, so each reduction stays inside live lanes
  for (int64_t u = (int64_t)blockIdx.x * kRowThreads + threadIdx.x; u < units; u += (int64_t)unit_wgs * kRowThreads) {
    const int64_t t = u / per, c = (u - t * per) * E;
    float x[E];
    widen_raw(load_raw<XK, E>(p.x, t * p.ldx + c), x);
    const float top = segment_max<E>(amax_of(x), p.gran);
    const bool leads = (c & (p.gran - 1)) == 0;
    float s = block_scale(top, format_max(p.fmt));
    int code[E / 4];
    if constexpr (!W) codes_of(x, s, p.fmt, code);
    for (int j = 0; j < p.k; ++j) {
      const int r = p.position[t * p.k + j];
      if (r < 0 || r >= p.rows) continue;
      if constexpr (W) {
        // rounding keeps order: the largest |w x| is that of the largest |x|
        const float w = p.weights[t * p.k + j];
        s = block_scale(fabsf(top * w), format_max(p.fmt));
        float y[E];
#pragma unroll
        for (int i = 0; i < E; ++i) y[i] = x[i] * w;
        codes_of(y, s, p.fmt, code);
      }
      put_codes<E>(p.q + (int64_t)r * p.cols + c, code);
      if (leads) p.scales[(int64_t)r * segs + c / p.gran] = s;
    }
  }
}

// g x g: one block of sorted rows per workgroup, its values in registers between
// amax and codes.
template <int XK, int G, int NT, bool W>
__global__ __launch_bounds__(NT) void route_blocks(const RouteQuantArgs p) {
  constexpr int E = 8, ROW_L = G / E, RPP = NT / ROW_L, PASSES = G / RPP;
  static_assert(PASSES * RPP == G, "passes");
  __shared__ float red[NT / 64];
  const int64_t ncb = p.cols / G;
  const int64_t rb = blockIdx.x / ncb, cb = blockIdx.x % ncb;
  if (p.slot[rb * G] == -2) return;  // behind the last group
  const int t = threadIdx.x, rsub = t / ROW_L, cl = t % ROW_L;
  const int64_t c = cb * G + cl * E;
  const int64_t slots = p.tokens * p.k;
  float z[PASSES][E];
  float top = 0.0f;
#pragma unroll
  for (int i = 0; i < PASSES; ++i) {
    const int64_t r = rb * G + i * RPP + rsub;
    const int s = r < p.rows ? p.slot[r] : -2;
#pragma unroll
    for (int k = 0; k < E; ++k) z[i][k] = 0.0f;
    if (s >= 0 && s < slots) {
      widen_raw(load_raw<XK, E>(p.x, (int64_t)((unsigned)s / (unsigned)p.k) * p.ldx + c), z[i]);
      if constexpr (W) {
        const float w = p.weights[s];
#pragma unroll
        for (int k = 0; k < E; ++k) z[i][k] *= w;
      }
    }
    top = fmaxf(top, amax_of(z[i]));
  }
  top = group_max<64>(top);
  if ((t & 63) == 0) red[t >> 6] = top;
  __syncthreads();
  DG_STEP_SYNC_WG();
  top = red[0];
#pragma unroll
  for (int w = 1; w < NT / 64; ++w) top = fmaxf(top, red[w]);
  const float s = block_scale(top, format_max(p.fmt));
  if (t == 0) p.scales[rb * ncb + cb] = s;
#pragma unroll
  for (int i = 0; i < PASSES; ++i) {
    const int64_t r = rb * G + i * RPP + rsub;
    if (r < p.rows && p.slot[r] != -2) {
      int code[E / 4];
      codes_of(z[i], s, p.fmt, code);
      put_codes<E>(p.q + r * p.cols + c, code);
    }
  }
}

constexpr int64_t kMaxWgs = 1 << 20;

template <int XK, bool W>
hipError_t launch_rows_w(const RouteQuantArgs& p, hipStream_t stream) {
  if (p.block_rows == 1) {
    constexpr int E = unit_of(XK, 1);
    const int64_t units = p.tokens * (p.cols / E);
    const int64_t wgs = std::min((units + kRowThreads - 1) / kRowThreads, kMaxWgs);
    const int64_t pads = std::min<int64_t>((p.rows + kRowThreads - 1) / kRowThreads, kMaxWgs);
    hipLaunchKernelGGL((route_rows<XK, W>), dim3((unsigned)(wgs + pads)), dim3(kRowThreads), 0, stream, p, units, (unsigned)wgs);
  } else {
    const dim3 grid((unsigned)(((p.rows + p.gran - 1) / p.gran) * (p.cols / p.gran)));
    if (p.gran == 64) hipLaunchKernelGGL((route_blocks<XK, 64, 256, W>), grid, dim3(256), 0, stream, p);
    else if (p.gran == 128) hipLaunchKernelGGL((route_blocks<XK, 128, 512, W>), grid, dim3(512), 0, stream, p);
    else hipLaunchKernelGGL((route_blocks<XK, 256, 1024, W>), grid, dim3(1024), 0, stream, p);
  }
  return hipGetLastError();
}

template <int XK>
hipError_t launch_rows(const RouteQuantArgs& p, hipStream_t stream) {
  return p.weights ? launch_rows_w<XK, true>(p, stream) : launch_rows_w<XK, false>(p, stream);
}

// ---- the combine --------------------------------------------------------------

template <int YK, int OK>
__global__ __launch_bounds__(kRowThreads) void route_combine(const CombineArgs p, int64_t units) {
  constexpr int E = unit_of(YK, OK);
  const int64_t per = p.cols / E;
  for (int64_t u = (int64_t)blockIdx.x * kRowThreads + threadIdx.x; u < units; u += (int64_t)gridDim.x * kRowThreads) {
    const int64_t t = u / per, c = (u - t * per) * E;
    float acc[E];
#pragma unroll
    for (int i = 0; i < E; ++i) acc[i] = 0.0f;
#pragma unroll 4
    for (int j = 0; j < p.k; ++j) {
      const int r = p.position[t * p.k + j];
      if (r < 0 || r >= p.rows) continue;
      const float w = p.weights ? p.weights[t * p.k + j] : 1.0f;
      float y[E];
      widen_raw(load_raw<YK, E>(p.y, (int64_t)r * p.ldy + c), y);
#pragma unroll
      for (int i = 0; i < E; ++i) acc[i] = __builtin_fmaf(w, y[i], acc[i]);
    }
    if (p.res) {
      float f[E];
      widen_raw(load_raw<OK, E>(p.res, t * p.ldres + c), f);
#pragma unroll
      for (int i = 0; i < E; ++i) acc[i] += f[i];
    }
    store_raw(p.out, t * p.cols + c, round_raw<OK>(acc));
  }
}

template <int YK, int OK>
hipError_t launch_combine_k(const CombineArgs& p, hipStream_t stream) {
  const int64_t units = p.tokens * (p.cols / unit_of(YK, OK));
  const int64_t wgs = std::min((units + kRowThreads - 1) / kRowThreads, kMaxWgs);
  hipLaunchKernelGGL((route_combine<YK, OK>), dim3((unsigned)wgs), dim3(kRowThreads), 0, stream, p, units);
  return hipGetLastError();
}

template <int YK>
hipError_t launch_combine_y(const CombineArgs& p, hipStream_t stream) {
  switch (p.ok) {
    case 0: return launch_combine_k<YK, 0>(p, stream);
    case 1: return launch_combine_k<YK, 1>(p, stream);
    case 2: return launch_combine_k<YK, 2>(p, stream);
    default: return hipErrorInvalidValue;
  }
}

// ---- the gradient of the weights ----------------------------------------------

// A workgroup takes a token, eight of its rows at a time: x once per eight rows.
template <int XK, int YK>
__global__ __launch_bounds__(kRowThreads) void route_weight_grad(const WeightGradArgs p) {
  constexpr int E = unit_of(XK, YK), J = 8;
  __shared__ float red[kRowThreads / 64][J];
  const int tid = threadIdx.x, wave = tid >> 6;
  for (int64_t t = blockIdx.x; t < p.tokens; t += gridDim.x) {
    for (int j0 = 0; j0 < p.k; j0 += J) {
      int r[J];
      float acc[J];
#pragma unroll
      for (int j = 0; j < J; ++j) {
        r[j] = j0 + j < p.k ? p.position[t * p.k + j0 + j] : -1;
        if (r[j] >= p.rows) r[j] = -1;
        acc[j] = 0.0f;
      }
      for (int64_t c = tid * E; c < p.cols; c += kRowThreads * E) {
        float x[E];
        widen_raw(load_raw<XK, E>(p.x, t * p.ldx + c), x);
#pragma unroll
        for (int j = 0; j < J; ++j) {
          if (r[j] < 0) continue;
          float y[E];
          widen_raw(load_raw<YK, E>(p.y, (int64_t)r[j] * p.ldy + c), y);
#pragma unroll
          for (int i = 0; i < E; ++i) acc[j] = __builtin_fmaf(x[i], y[i], acc[j]);
        }
      }
      __syncthreads();
#pragma unroll
      for (int j = 0; j < J; ++j) {
        const float v = wave_sum(acc[j]);
        if ((tid & 63) == 0) red[wave][j] = v;
      }
      __syncthreads();
      if (tid < J && j0 + tid < p.k) {
        float v = red[0][tid];
#pragma unroll
        for (int w = 1; w < kRowThreads / 64; ++w) v += red[w][tid];
        p.dw[t * p.k + j0 + tid] = v;
      }
    }
  }
}

template <int XK>
hipError_t launch_weight_grad_x(const WeightGradArgs& p, hipStream_t stream) {
  const dim3 grid((unsigned)std::min<int64_t>(p.tokens, kMaxWgs)), block(kRowThreads);
  switch (p.yk) {
    case 0: hipLaunchKernelGGL((route_weight_grad<XK, 0>), grid, block, 0, stream, p); break;
    case 1: hipLaunchKernelGGL((route_weight_grad<XK, 1>), grid, block, 0, stream, p); break;
    case 2: hipLaunchKernelGGL((route_weight_grad<XK, 2>), grid, block, 0, stream, p); break;
    default: return hipErrorInvalidValue;
  }
  return hipGetLastError();
}

}  // namespace

int64_t sort_workspace(int64_t n, int groups) {
  if (n <= kOneSort) return 0;
  const int64_t per = sort_chunk(n);
  return (n + per - 1) / per * groups * (int64_t)sizeof(int);
}

hipError_t launch_sort(const SortArgs& args, hipStream_t stream) {
  SortArgs p = args;
  p.per = (int)(p.n <= kOneSort ? p.n : sort_chunk(p.n));
  p.chunks = p.n <= kOneSort ? 0 : (int)((p.n + p.per - 1) / p.per);
  return p.wide ? launch_sort_t<int64_t>(p, stream) : launch_sort_t<int32_t>(p, stream);
}

int64_t route_quant_workspace(int64_t, int64_t, int, int) { return 0; }

hipError_t launch_route_quant(const RouteQuantArgs& p, hipStream_t stream) {
  switch (p.xk) {
    case 0: return launch_rows<0>(p, stream);
    case 1: return launch_rows<1>(p, stream);
    case 2: return launch_rows<2>(p, stream);
    default: return hipErrorInvalidValue;
  }
}

hipError_t launch_combine(const CombineArgs& p, hipStream_t stream) {
  switch (p.yk) {
    case 0: return launch_combine_y<0>(p, stream);
    case 1: return launch_combine_y<1>(p, stream);
    case 2: return launch_combine_y<2>(p, stream);
    default: return hipErrorInvalidValue;
  }
}

hipError_t launch_weight_grad(const WeightGradArgs& p, hipStream_t stream) {
  switch (p.xk) {
    case 0: return launch_weight_grad_x<0>(p, stream);
    case 1: return launch_weight_grad_x<1>(p, stream);
    case 2: return launch_weight_grad_x<2>(p, stream);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace dg

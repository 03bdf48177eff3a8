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
// Bound by HBM, but for the coding of g x g blocks by tokens, whose k codes per
// element read make it arithmetic. Times are of 8192 tokens, 8 of 64 groups each,
// 4096 columns in BF16, unless a comment says otherwise; HBM copies at 5.9 TB/s.

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

// Slots that one workgroup sorts alone (calls of 2048, 4096 and 8192 slots 5.6, 7.0
// and 10.2 us, in chunks 8.3, 8.3 and 8.5); beyond, chunks of at least kChunk slots,
// at most 256 of them, are counted by one launch and placed by a second.
constexpr int64_t kOneSort = 4096, kChunk = 1024;

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
// those of lower lanes, found by comparing keys bit by bit with ballots: no
// atomics, so the order is always the slots' own. 3.7 us for 8 slots (a launch and
// its barriers), 4.9 + 6.2 for 65536 (chunks of 4096 slots: 9.6).
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

// quant_common.h's div_by_scale in five instructions: the remainder is taken
// with its sign turned (q s - x), which leaves a zero the sign of x by itself (q =
// -0 gives a remainder of +0, and -(+0) inv + -0 is -0), so no sign is copied.
__device__ __forceinline__ float quotient(float x, float s, float inv) {
  float q = x * inv;
  q = __builtin_fmaf(-__builtin_fmaf(q, s, -x), inv, q);
  return __builtin_fmaf(-__builtin_fmaf(q, s, -x), inv, q);
}

// The same in three, for BF16 and FP16 values and the factor of their own block's
// largest: one correction gives RN(x / s) for each of the 2^20 pairs of mantissas
// of x and of the largest value (all tried; the largest finite value of either
// format is 7 times a power of two). The exponents play no part while the
// remainder, down to 2^-48 of an x that does not code to zero, stays normal: s
// from 2^-60 to 2^60. (Coding x m (1 - e) and x m (1 + e) instead, m = w / s, and
// dividing where the codes differ: 85 us of 94 with weights, but 127 of 78 without,
// where exact ties are common.)
__device__ __forceinline__ float quotient_of_block(float x, float s, float inv) {
  const float q = x * inv;
  return __builtin_fmaf(-__builtin_fmaf(q, s, -x), inv, q);
}

// A wave whose factors all have normal reciprocals divides by them; where one has
// not, every lane of it takes the quantisers' two ways (the same codes). SHORT:
// quotient_of_block's values.
template <int FMT, bool SHORT, int E>
__device__ __forceinline__ void codes_fmt(const float (&y)[E], float s, float inv, int (&c)[E / 4]) {
  const bool fast = recip_ok(s);
  if constexpr (SHORT) {
    if (__all(s >= 0x1p-60f && s <= 0x1p60f)) {
#pragma unroll
      for (int i = 0; i < E / 4; ++i) {
        const int lo = cvt2<FMT, false>(quotient_of_block(y[4 * i], s, inv), quotient_of_block(y[4 * i + 1], s, inv), 0);
        c[i] = cvt2<FMT, true>(quotient_of_block(y[4 * i + 2], s, inv), quotient_of_block(y[4 * i + 3], s, inv), lo);
      }
      return;
    }
  }
  if (!SHORT && __all(fast)) {
#pragma unroll
    for (int i = 0; i < E / 4; ++i) {
      const int lo = cvt2<FMT, false>(quotient(y[4 * i], s, inv), quotient(y[4 * i + 1], s, inv), 0);
      c[i] = cvt2<FMT, true>(quotient(y[4 * i + 2], s, inv), quotient(y[4 * i + 3], s, inv), lo);
    }
  } else {
#pragma unroll
    for (int i = 0; i < E / 4; ++i) {
      const v4f v = {y[4 * i], y[4 * i + 1], y[4 * i + 2], y[4 * i + 3]};
      if (fast) c[i] = encode4<FMT, true>(v, s, inv);
      else c[i] = encode4<FMT, false>(v, s, inv);
    }
  }
}

// The codes of y / s, inv = 1 / s. SHORT: y as it was read, of 16 bits.
template <bool SHORT, int E>
__device__ __forceinline__ void codes_of(const float (&y)[E], float s, float inv, int fmt, int (&c)[E / 4]) {
  if (fmt == 1) codes_fmt<1, SHORT>(y, s, inv, c);
  else codes_fmt<0, SHORT>(y, s, inv, c);
}

template <bool ONCE, int E>
__device__ __forceinline__ void put_codes(uint8_t* q, const int (&c)[E / 4]) {
  if constexpr (E == 8) {
    if constexpr (ONCE) __builtin_nontemporal_store((v2i){c[0], c[1]}, reinterpret_cast<v2i*>(q));
    else *reinterpret_cast<v2i*>(q) = (v2i){c[0], c[1]};
  } else {
    if constexpr (ONCE) __builtin_nontemporal_store(c[0], reinterpret_cast<int*>(q));
    else *reinterpret_cast<int*>(q) = c[0];
  }
}

// Rows between a group's last and the next group: codes of zero and, with a
// factor per row, factors of one. A wave looks at kPadRows rows. 8 / 64 of them, in
// us: 4 x 6 of 7168 to 19 groups of 128 rows with the weights' gradient 14.5 / 31.2, 81 x
// 2 of 1280 to 44 of 16 10.8 / 15.3, 8192 x 8 of 4096 to 64 of 128 80 / 89, of 1 77.5 /
// 77.8; 65536 x 8 of 256 72 / 69.
constexpr int kPadRows = 8;

__device__ __forceinline__ void pad_rows(const RouteQuantArgs& p, int64_t wave, int lane) {
  const int64_t r0 = wave * kPadRows;
  const int s = lane < kPadRows && r0 + lane < p.rows ? p.slot[r0 + lane] : -2;
  uint64_t m = __ballot(s == -1);
  const int64_t segs = p.cols / p.gran;
  while (m) {
    const int64_t r = r0 + __builtin_ctzll(m);
    m &= m - 1;
    for (int64_t c = lane * 16; c < p.cols; c += 64 * 16) *reinterpret_cast<v4u*>(p.q + r * p.cols + c) = (v4u){};
    if (p.block_rows == 1)
      for (int64_t c = lane; c < segs; c += 64) p.scales[r * segs + c] = 1.0f;
  }
}

constexpr int kRowThreads = 256, kRowWaves = kRowThreads / 64;

// How a wave of the token kernels takes its share: U units of E columns per
// lane, 64 E apart, from column `c0` of token `t` on.
template <int E, int U>
struct Piece {
  int64_t c0;
  __device__ __forceinline__ int64_t col(int u, int lane) const { return c0 + (int64_t)(u * 64 + lane) * E; }
};

// The tokens' rows, codes of every one of them: a wave takes a piece of a token,
// whose k rows and weights its lanes load at once, in flight with the token's
// columns. OWN: 1 x g, the factors are the token's own segments' (with weights:
// each row's, since |w x| is largest where |x| is: rounding keeps order);
// otherwise the factors of g x g blocks are in scales already. Sorted rows taken
// by their own waves instead would read x k times. 69 us (0.34 GB: 57; the vector ALU
// busy 79% of the cycles; with two corrections of every quotient 78 us), with weights,
// whose quotients need both, 94 (84%); 1 x g, 2000 x 2 rows of 7168 in FP32 with
// weights 22.5 (86 MB: 15; 33 while a wave cleared up to 64 rows between groups;
// sharing the factors' divisions over a segment's lanes changed nothing).
template <int XK, bool W, bool OWN, int U, bool ONCE>
__global__ __launch_bounds__(kRowThreads) void route_rows(const RouteQuantArgs p, int pieces, int token_wgs) {
  constexpr int E = unit_of(XK, 1);
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int unit_wgs = pieces * token_wgs;
  if ((int)blockIdx.x >= unit_wgs) {
    const int64_t first = (int64_t)((int)blockIdx.x - unit_wgs) * kRowWaves + wave, step = (int64_t)((int)gridDim.x - unit_wgs) * kRowWaves;
    for (int64_t w = first; w * kPadRows < p.rows; w += step) pad_rows(p, w, lane);
    return;
  }
  const Piece<E, U> piece{(int64_t)((int)blockIdx.x % pieces) * (64 * E * U)};
  const int64_t segs = p.cols / p.gran;
  const int gshift = 31 - __builtin_clz(p.gran);
  const float fmax = format_max(p.fmt);
  const float* const invs = p.ws + p.tokens * segs;  // of g x g blocks
  for (int64_t t = (int64_t)((int)blockIdx.x / pieces) * kRowWaves + wave; t < p.tokens; t += (int64_t)token_wgs * kRowWaves) {
    int rows = lane < p.k ? p.position[t * p.k + lane] : -1;
    float ws = W && lane < p.k ? p.weights[t * p.k + lane] : 0.0f;
    float x[U][E], top[U], own[U];
    int code[U][E / 4];
    bool live[U];  // whole segments are live or not, so each reduction stays inside live lanes
#pragma unroll
    for (int u = 0; u < U; ++u) {
      live[u] = piece.col(u, lane) < p.cols;
      if (live[u]) widen_raw(load_raw<XK, E, ONCE>(p.x, t * p.ldx + piece.col(u, lane)), x[u]);
    }
    // g x g: the factors of the next of the token's rows are on their way while one is coded
    float s[U], inv[U], s1[U], inv1[U];
    auto fetch = [&](int r) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int64_t at = (int64_t)(r >> gshift) * segs + (piece.col(u, lane) >> gshift);
        const bool has = live[u] && r >= 0 && r < p.rows;
        s1[u] = has ? p.scales[at] : 1.0f;
        inv1[u] = has ? invs[at] : 1.0f;
      }
    };
    if constexpr (!OWN) fetch(__builtin_amdgcn_readlane(rows, 0));
    if constexpr (OWN) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (!live[u]) continue;
        top[u] = segment_max<E>(amax_of(x[u]), p.gran);
        if constexpr (!W) {
          own[u] = block_scale(top[u], fmax);
          codes_of<XK != 0>(x[u], own[u], 1.0f / own[u], p.fmt, code[u]);
        }
      }
    }
    for (int j = 0; j < p.k; ++j) {
      const int r = __builtin_amdgcn_readlane(rows, j & 63);
      const float w = W ? __int_as_float(__builtin_amdgcn_readlane(__float_as_int(ws), j & 63)) : 1.0f;
      if (j + 1 < p.k && ((j + 1) & 63) == 0) {  // more than 64 choices
        rows = j + 1 + lane < p.k ? p.position[t * p.k + j + 1 + lane] : -1;
        if constexpr (W) ws = j + 1 + lane < p.k ? p.weights[t * p.k + j + 1 + lane] : 0.0f;
      }
      if constexpr (!OWN) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
          s[u] = s1[u];
          inv[u] = inv1[u];
        }
        if (j + 1 < p.k) fetch(__builtin_amdgcn_readlane(rows, (j + 1) & 63));
      }
      if (r < 0 || r >= p.rows) continue;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (!live[u]) continue;
        const int64_t c = piece.col(u, lane);
        if constexpr (W || !OWN) {
          float y[E];
#pragma unroll
          for (int i = 0; i < E; ++i) y[i] = W ? x[u][i] * w : x[u][i];
          if constexpr (OWN) {
            s[u] = block_scale(fabsf(top[u] * w), fmax);
            inv[u] = 1.0f / s[u];
          }
          codes_of<XK != 0 && !W>(y, s[u], inv[u], p.fmt, code[u]);
        } else {
          s[u] = own[u];
        }
        put_codes<ONCE, E>(p.q + (int64_t)r * p.cols + c, code[u]);
        if (OWN && (c & (p.gran - 1)) == 0) p.scales[(int64_t)r * segs + (c >> gshift)] = s[u];
      }
    }
  }
}

// Every token's segment maxima, for the factors of g x g blocks. 16.6 us (67 MB: 11).
template <int XK, int U>
__global__ __launch_bounds__(kRowThreads) void route_maxima(const RouteQuantArgs p, int pieces, int token_wgs) {
  constexpr int E = unit_of(XK, 1);
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const Piece<E, U> piece{(int64_t)((int)blockIdx.x % pieces) * (64 * E * U)};
  const int64_t segs = p.cols / p.gran;
  for (int64_t t = (int64_t)((int)blockIdx.x / pieces) * kRowWaves + wave; t < p.tokens; t += (int64_t)token_wgs * kRowWaves) {
    Raw<XK, E> raw[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (piece.col(u, lane) < p.cols) raw[u] = load_raw<XK, E>(p.x, t * p.ldx + piece.col(u, lane));
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t c = piece.col(u, lane);
      if (c >= p.cols) continue;
      float x[E];
      widen_raw(raw[u], x);
      const float top = segment_max<E>(amax_of(x), p.gran);
      if ((c & (p.gran - 1)) == 0) p.ws[t * segs + c / p.gran] = top;
    }
  }
}

// The factors of g x g blocks of sorted rows from the tokens' maxima, and their
// reciprocals (behind the maxima) for the many divisions that follow: a
// workgroup takes a row of blocks, 32 of them, its threads 32 rows at a time. 9.1 us,
// the latency of slot, then maximum, four times over: a load stays under the test of
// its index, and is waited for there before the next.
constexpr int kFactorThreads = 1024;

template <bool W>
__global__ __launch_bounds__(kFactorThreads) void route_factors(const RouteQuantArgs p, int seg_wgs) {
  constexpr int CL = 32, RL = kFactorThreads / CL;
  __shared__ float red[RL][CL];
  const int64_t segs = p.cols / p.gran;
  const int64_t rb = (int)blockIdx.x / seg_wgs;
  if (p.slot[rb * p.gran] == -2) return;  // behind the last group
  const int cl = threadIdx.x % CL, rl = threadIdx.x / CL;
  const int64_t seg = (int64_t)((int)blockIdx.x % seg_wgs) * CL + cl;
  const int64_t slots = p.tokens * p.k, end = min(rb * p.gran + p.gran, p.rows);
  float top = 0.0f;
  if (seg < segs) {
#pragma unroll 8
    for (int64_t r = rb * p.gran + rl; r < end; r += RL) {
      const int s = p.slot[r];
      if (s < 0 || s >= slots) continue;
      float v = p.ws[(int64_t)((unsigned)s / (unsigned)p.k) * segs + seg];
      if constexpr (W) v = fabsf(v * p.weights[s]);
      top = fmaxf(top, v);
    }
  }
  red[rl][cl] = top;
  __syncthreads();
  if (rl == 0 && seg < segs) {
#pragma unroll
    for (int i = 1; i < RL; ++i) top = fmaxf(top, red[i][cl]);
    const float s = block_scale(top, format_max(p.fmt));
    p.scales[rb * segs + seg] = s;
    p.ws[p.tokens * segs + rb * segs + seg] = 1.0f / s;
  }
}

// g x g: one block of sorted rows per workgroup, its values in registers between
// amax and codes. 4096 x 2 rows of 7168 at g = 128: 54 us with the sort (0.18 GB: 30).
// A pass loads its slot, then its row, and each is waited for before the next pass's:
// eight trips in a row before the maximum.
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
  const float s = block_scale(top, format_max(p.fmt)), inv = 1.0f / s;
  if (t == 0) p.scales[rb * ncb + cb] = s;
#pragma unroll
  for (int i = 0; i < PASSES; ++i) {
    const int64_t r = rb * G + i * RPP + rsub;
    if (r < p.rows && p.slot[r] != -2) {
      int code[E / 4];
      codes_of<XK != 0 && !W>(z[i], s, inv, p.fmt, code);
      put_codes<false, E>(p.q + r * p.cols + c, code);
    }
  }
}

constexpr int64_t kMaxWgs = 1 << 20;

// g x g blocks by tokens: three launches that read every token twice, instead of
// one that gathers every row of a block (and reads it twice). It pays where a
// token has several rows and the codes are many; rows are those allocated, since the
// host does not know how many of them groups have, and those between groups are
// cleared by either. Sort and dispatch of BF16 rows to groups of 128, by tokens / by
// blocks, in us: 1024 x 8 of 4096 to 64 groups 33.0 / 31.2, 2048 x 8 44.5 / 48.2, 8192 x 8
// 95 / 160; 4096 x 2 of 7168 to 8 61.5 / 53.8, 8192 x 2 87 / 93, 16384 x 2 of 4096 93 / 104;
// 4096 x 4 of 7168 to 16 64 / 81; 64 x 8 of 8192 to 64, of whose rows most are between
// groups, 24.7 / 26.4.
constexpr int64_t kByTokens = 1ll << 26;

bool by_tokens(int64_t tokens, int64_t rows, int64_t cols) { return (rows - tokens) * cols >= kByTokens; }

// Units per lane: four where that leaves the chip enough waves (32 a CU). Sort and
// dispatch to 1 x g, one / four, in us: 1024 x 2 of 4096 in BF16 12.5 / 12.5, 2000 x
// 2 of 7168 20.4 / 22.5, in FP32 28.8 / 25.6; 8192 x 2 of 4096 42.9 / 43.8, to g x g
// 57.9 / 57.8.
template <int E>
int units_per_lane(int64_t tokens, int64_t cols) {
  return cols >= 64 * E * 4 && tokens * (cols / (64 * E * 4)) >= 8192 ? 4 : 1;
}

template <int XK, bool W, bool OWN, int U>
hipError_t launch_tokens(const RouteQuantArgs& p, hipStream_t stream) {
  constexpr int E = unit_of(XK, 1);
  const int64_t pieces = (p.cols + 64 * E * U - 1) / (64 * E * U);
  const int64_t tokens = std::min((p.tokens + kRowWaves - 1) / kRowWaves, std::max<int64_t>(1, kMaxWgs / pieces));
  const int64_t pads = std::min<int64_t>((p.rows + kRowWaves * kPadRows - 1) / (kRowWaves * kPadRows), kMaxWgs);
  if constexpr (!OWN) {
    hipLaunchKernelGGL((route_maxima<XK, U>), dim3((unsigned)(pieces * tokens)), dim3(kRowThreads), 0, stream, p, (int)pieces, (int)tokens);
    hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
    const int64_t segs = (p.cols / p.gran + 31) / 32;
    hipLaunchKernelGGL((route_factors<W>), dim3((unsigned)((p.rows + p.gran - 1) / p.gran * segs)), dim3(kFactorThreads), 0, stream, p, (int)segs);
    err = hipGetLastError();
    if (err != hipSuccess) return err;
  }
  const dim3 grid((unsigned)(pieces * tokens + pads));
  // past the caches: 8192 x 8 of 4096 to 1 x g 82 -> 78 us, 4096 x 8 48 -> 44, 2048 x 8 25.2 -> 27.8
  if (p.rows * p.cols + p.tokens * p.cols * InKind<XK>::kBytes >= 2 * kOnceBytes)
    hipLaunchKernelGGL((route_rows<XK, W, OWN, U, true>), grid, dim3(kRowThreads), 0, stream, p, (int)pieces, (int)tokens);
  else
    hipLaunchKernelGGL((route_rows<XK, W, OWN, U, false>), grid, dim3(kRowThreads), 0, stream, p, (int)pieces, (int)tokens);
  return hipGetLastError();
}

template <int XK, bool W>
hipError_t launch_rows_w(const RouteQuantArgs& p, hipStream_t stream) {
  const bool four = units_per_lane<unit_of(XK, 1)>(p.tokens, p.cols) == 4;
  if (p.block_rows == 1) return four ? launch_tokens<XK, W, true, 4>(p, stream) : launch_tokens<XK, W, true, 1>(p, stream);
  if (by_tokens(p.tokens, p.rows, p.cols)) return four ? launch_tokens<XK, W, false, 4>(p, stream) : launch_tokens<XK, W, false, 1>(p, stream);
  const dim3 grid((unsigned)(((p.rows + p.gran - 1) / p.gran) * (p.cols / p.gran)));
  if (p.gran == 64) hipLaunchKernelGGL((route_blocks<XK, 64, 256, W>), grid, dim3(256), 0, stream, p);
  else if (p.gran == 128) hipLaunchKernelGGL((route_blocks<XK, 128, 512, W>), grid, dim3(512), 0, stream, p);
  else hipLaunchKernelGGL((route_blocks<XK, 256, 1024, W>), grid, dim3(1024), 0, stream, p);
  return hipGetLastError();
}

template <int XK>
hipError_t launch_rows(const RouteQuantArgs& p, hipStream_t stream) {
  return p.weights ? launch_rows_w<XK, true>(p, stream) : launch_rows_w<XK, false>(p, stream);
}

// ---- the combine --------------------------------------------------------------
//
// A thread takes 16 bytes of out and the same columns of its token's k rows, one
// after the other: a row's load is under the test of its position and is waited for
// before the next position's, 2 k trips in a row, which the waves of a large call hide
// and those of a small one do not. 116 us (0.60 GB: 102); 64 x 8 rows 4.4 (5.2 MB: 0.9).

template <int YK, int OK, bool ONCE>
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
      widen_raw(load_raw<YK, E, ONCE>(p.y, (int64_t)r * p.ldy + c), y);
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
  // past the caches: 8192 x 8 rows of 4096 in BF16 121 -> 120 us, 2048 x 8 34.4 -> 32.1, 1024 x 8 12.7 -> 17.0
  if (p.tokens * p.k * p.cols * InKind<YK>::kBytes >= 2 * kOnceBytes)
    hipLaunchKernelGGL((route_combine<YK, OK, true>), dim3((unsigned)wgs), dim3(kRowThreads), 0, stream, p, units);
  else
    hipLaunchKernelGGL((route_combine<YK, OK, false>), dim3((unsigned)wgs), dim3(kRowThreads), 0, stream, p, units);
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

// A workgroup takes a token, eight of its rows at a time: x once per eight rows, whose
// loads follow one another (the many workgroups' overlap). 101 us (0.60 GB: 102); 2000 x 2
// of 7168, x in FP32, 20.4 (115 MB: 19).
template <int XK, int YK, bool ONCE>
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
          widen_raw(load_raw<YK, E, ONCE>(p.y, (int64_t)r[j] * p.ldy + c), y);
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

template <int XK, int YK>
hipError_t launch_weight_grad_k(const WeightGradArgs& p, hipStream_t stream) {
  const dim3 grid((unsigned)std::min<int64_t>(p.tokens, kMaxWgs)), block(kRowThreads);
  // past the caches: with the rows' codes 8192 x 8 of 4096 in BF16 223 -> 206 us, 1024
  // x 8 41.9 -> 36.0, 512 x 8 34.1 -> 35.7
  if (p.tokens * p.k * p.cols * InKind<YK>::kBytes >= kOnceBytes)
    hipLaunchKernelGGL((route_weight_grad<XK, YK, true>), grid, block, 0, stream, p);
  else
    hipLaunchKernelGGL((route_weight_grad<XK, YK, false>), grid, block, 0, stream, p);
  return hipGetLastError();
}

template <int XK>
hipError_t launch_weight_grad_x(const WeightGradArgs& p, hipStream_t stream) {
  switch (p.yk) {
    case 0: return launch_weight_grad_k<XK, 0>(p, stream);
    case 1: return launch_weight_grad_k<XK, 1>(p, stream);
    case 2: return launch_weight_grad_k<XK, 2>(p, stream);
    default: return hipErrorInvalidValue;
  }
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

int64_t route_quant_workspace(int64_t tokens, int64_t cols, int64_t rows, int gran, int block_rows) {
  return block_rows != 1 && by_tokens(tokens, rows, cols) ? 4 * (tokens + (rows + gran - 1) / gran) * (cols / gran) : 0;
}

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

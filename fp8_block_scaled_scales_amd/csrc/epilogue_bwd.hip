// The gradient through the product's epilogue out = act(C + bias) [+
// residual], for gfx950: dz = dout * act'(pre), written as FP8 codes with
// block factors for the next products, with dbias = sum over rows of dz.
//
// pre is the BF16 pre-activation the forward product kept; dz is FP32, from it
// the codes (the quantiser's rule, quant_common.h), dbias and, where asked for,
// dz itself in dout's type. With g x g blocks the codes serve the gradient of
// the activations and, read transposed, that of the weights.
//
// Bound by HBM (dout 2 or 4, pre 2 bytes in, 1 out per element): 8192 x 8192 in
// BF16 with GELU takes 70 us, 4.8 TB/s, where ReLU, with a tenth of the
// arithmetic, takes 67.
//
// Either way a thread keeps the same eight columns, so it holds their sums over
// its rows in FP32; a workgroup adds its threads' sums through LDS in a fixed
// order and writes one partial row, and column_sum adds the partial rows.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "activation.h"
#include "layer_ops.h"
#include "quant_common.h"

namespace dg {

namespace {

// dz of eight elements (ACT 0: dout itself).
template <int DK, int ACT, bool ONCE = false>
__device__ __forceinline__ void grad8(const EpiBwdArgs& p, int64_t row, int64_t c, float (&z)[8]) {
  widen8(load8<DK, ONCE>(p.dout, row * p.lddout + c), z);
  if constexpr (ACT != 0) {
    float pre[8];
    widen8(load8<1, ONCE>(p.pre, row * p.ldpre + c), pre);
#pragma unroll
    for (int i = 0; i < 8; ++i) z[i] *= act_grad<ACT>(pre[i]);
  }
}

// One g x g block per workgroup of NT threads; dz in registers between the amax
// and the encode. ONCE: nontemporal loads of the inputs and stores of the codes.
template <int DK, int ACT, int G, int NT, bool ONCE>
__global__ __launch_bounds__(NT) void epi_bwd_blocks(const EpiBwdArgs p, float* part) {
  constexpr int ROW_L = G / 8;    // lanes per block row
  constexpr int RPP = NT / ROW_L;  // block rows covered by one pass
  constexpr int PASSES = G / RPP;
  static_assert(PASSES * RPP == G, "passes");
  __shared__ float red[NT / 64];
  __shared__ float sums[RPP][G];
  const int ncb = (int)(p.cols / G);
  const int rb = blockIdx.x / ncb, cb = blockIdx.x % ncb;
  const int t = threadIdx.x, rsub = t / ROW_L, cl = t % ROW_L;
  const int64_t c = (int64_t)cb * G + cl * 8;

  float z[PASSES][8], acc[8];
  float amax = 0.0f;
#pragma unroll
  for (int k = 0; k < 8; ++k) acc[k] = 0.0f;
#pragma unroll
  for (int i = 0; i < PASSES; ++i) {
    const int64_t r = (int64_t)rb * G + i * RPP + rsub;
    if (r < p.rows) {
      grad8<DK, ACT, ONCE>(p, r, c, z[i]);
      amax = fmaxf(amax, amax8(z[i]));
#pragma unroll
      for (int k = 0; k < 8; ++k) acc[k] += z[i][k];
    }
  }
  amax = group_max<64>(amax);
  if ((t & 63) == 0) red[t >> 6] = amax;
  if (part) {
#pragma unroll
    for (int k = 0; k < 8; ++k) sums[rsub][cl * 8 + k] = acc[k];
  }
  __syncthreads();
  amax = red[0];
#pragma unroll
  for (int w = 1; w < NT / 64; ++w) amax = fmaxf(amax, red[w]);
  const float s = block_scale(amax, format_max(p.fmt));
  const float inv = 1.0f / s;
  if (t == 0) p.scales[blockIdx.x] = s;
#pragma unroll
  for (int i = 0; i < PASSES; ++i) {
    const int64_t r = (int64_t)rb * G + i * RPP + rsub;
    if (r < p.rows) {
      v2i* const q = reinterpret_cast<v2i*>(p.q + r * p.cols + c);
      if constexpr (ONCE) __builtin_nontemporal_store(encode8(z[i], s, inv, p.fmt), q);
      else *q = encode8(z[i], s, inv, p.fmt);
      if (p.dz) store8<DK>(p.dz, r * p.cols + c, round8<DK>(z[i]));
    }
  }
  if (part && t < G) {
    float v = sums[0][t];
#pragma unroll
    for (int i = 1; i < RPP; ++i) v += sums[i][t];
    part[(int64_t)rb * p.cols + (int64_t)cb * G + t] = v;
  }
}

// 1 x g: 512 columns per workgroup, its 16 waves (NW) a row each. The rows a
// workgroup takes lie ranges * NW apart, so that all workgroups advance through
// memory together: contiguous row ranges kept 128 distant places of it open at
// once and took 86 us where this takes 78 (8192 x 8192, BF16, GELU). Several
// rows in flight per wave measured slower (85), fewer waves per workgroup the
// same but for more partial rows (2000 x 7168, FP32: 23.0 us at 4 waves, 21.3
// at 16).
constexpr int NW = 16;

template <int DK, int ACT>
__global__ __launch_bounds__(64 * NW) void epi_bwd_rows(const EpiBwdArgs p, float* part, int col_groups, int ranges) {
  __shared__ float sums[NW][512];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int cg = blockIdx.x % col_groups, rr = blockIdx.x / col_groups;
  const int64_t c = (int64_t)cg * 512 + lane * 8;
  const int gshift = 31 - __builtin_clz(p.gran);
  const int64_t segs = p.cols >> gshift;
  float acc[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) acc[k] = 0.0f;
  if (c < p.cols) {  // whole segments are live or not, so each reduction stays inside live lanes
    for (int64_t r = (int64_t)NW * rr + wave; r < p.rows; r += (int64_t)NW * ranges) {
      float z[8];
      grad8<DK, ACT>(p, r, c, z);
#pragma unroll
      for (int k = 0; k < 8; ++k) acc[k] += z[k];
      const float s = block_scale(segment_max(amax8(z), p.gran), format_max(p.fmt));
      *reinterpret_cast<v2i*>(p.q + r * p.cols + c) = encode8(z, s, 1.0f / s, p.fmt);
      if (((int)c & (p.gran - 1)) == 0) p.scales[r * segs + (c >> gshift)] = s;
      if (p.dz) store8<DK>(p.dz, r * p.cols + c, round8<DK>(z));
    }
  }
  if (!part) return;
#pragma unroll
  for (int k = 0; k < 8; ++k) sums[wave][lane * 8 + k] = acc[k];
  __syncthreads();
  const int64_t col = (int64_t)cg * 512 + threadIdx.x;
  if (threadIdx.x < 512 && col < p.cols) {
    float v = sums[0][threadIdx.x];
#pragma unroll
    for (int w = 1; w < NW; ++w) v += sums[w][threadIdx.x];
    part[rr * p.cols + col] = v;
  }
}

// Partial rows of dbias: one per row of blocks (g x g), or per workgroup of a
// column group (1 x g): two workgroups per CU over all, a row per wave at least.
int64_t partial_rows(int64_t rows, int64_t cols, int gran, int block_rows) {
  if (block_rows != 1) return (rows + gran - 1) / gran;
  const int64_t r = 512 / ((cols + 511) / 512), most = (rows + NW - 1) / NW;
  return r < 1 ? 1 : r < most ? r : most;
}

// Inputs of 64 MB and more (twice the L2s) are loaded, and their codes stored,
// nontemporally: 8192 x 8192 in BF16 at g = 128 73.4 -> 68.0 us, at g = 64 72.7
// -> 69.4 us; a matrix of 16 MB was 5% slower that way.
constexpr int64_t kOnceBytes = 64ll << 20;

template <int DK, int ACT, int G, int NT>
void launch_blocks(const EpiBwdArgs& p, float* part, hipStream_t stream) {
  const dim3 grid((unsigned)(((p.rows + G - 1) / G) * (p.cols / G)));
  if (p.rows * p.cols * (InKind<DK>::kBytes + (ACT ? 2 : 0)) >= kOnceBytes)
    hipLaunchKernelGGL((epi_bwd_blocks<DK, ACT, G, NT, true>), grid, dim3(NT), 0, stream, p, part);
  else
    hipLaunchKernelGGL((epi_bwd_blocks<DK, ACT, G, NT, false>), grid, dim3(NT), 0, stream, p, part);
}

// Threads per block. At g = 128 512 (four pieces of eight elements per thread)
// overlap better in a long launch of 16-bit blocks (8192 x 8192 in BF16 68.8 us
// against 72.8 at 1024 and 76 at 256), 1024 are faster for FP32 blocks (4096 x
// 4096 25.5 -> 23.7 us) and while there are at most four blocks per CU (1024 x
// 4096 in BF16 10.1 -> 9.6 us). 256 neighbouring columns per workgroup, which
// would make the row pieces 512 bytes, measured 84 us: fewer, larger
// workgroups overlap their loads and stores less.
template <int DK, int ACT>
hipError_t launch_act(const EpiBwdArgs& p, hipStream_t stream) {
  const int64_t n = partial_rows(p.rows, p.cols, p.gran, p.block_rows);
  float* const part = !p.dbias ? nullptr : n > 1 ? p.ws : p.dbias;
  if (p.block_rows == 1) {
    const int64_t col_groups = (p.cols + 511) / 512;
    hipLaunchKernelGGL((epi_bwd_rows<DK, ACT>), dim3((unsigned)(col_groups * n)), dim3(64 * NW), 0, stream, p, part,
                       (int)col_groups, (int)n);
  } else if (p.gran == 64) {
    launch_blocks<DK, ACT, 64, 256>(p, part, stream);
  } else if (p.gran == 128) {
    if (DK == 0 || ((p.rows + 127) / 128) * (p.cols / 128) <= 1024) launch_blocks<DK, ACT, 128, 1024>(p, part, stream);
    else launch_blocks<DK, ACT, 128, 512>(p, part, stream);
  } else {
    launch_blocks<DK, ACT, 256, 1024>(p, part, stream);
  }
  const hipError_t err = hipGetLastError();
  if (err != hipSuccess || !p.dbias || n == 1) return err;
  return launch_column_sum(p.ws, n, p.cols, p.dbias, stream);
}

template <int DK>
hipError_t launch_kind(const EpiBwdArgs& p, hipStream_t stream) {
  switch (p.act) {
    case 0: return launch_act<DK, 0>(p, stream);
    case 1: return launch_act<DK, 1>(p, stream);
    case 2: return launch_act<DK, 2>(p, stream);
    case 3: return launch_act<DK, 3>(p, stream);
    case 4: return launch_act<DK, 4>(p, stream);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace

int64_t epi_bwd_workspace(int64_t rows, int64_t cols, int gran, int block_rows) {
  const int64_t n = partial_rows(rows, cols, gran, block_rows);
  return n > 1 ? n * cols * (int64_t)sizeof(float) : 0;
}

hipError_t launch_epi_bwd(const EpiBwdArgs& p, hipStream_t stream) {
  switch (p.dk) {
    case 0: return launch_kind<0>(p, stream);
    case 1: return launch_kind<1>(p, stream);
    case 2: return launch_kind<2>(p, stream);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace dg

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
// BF16 with GELU takes 70 us with dbias, 65 without (5.2 TB/s, and the vector
// ALU 88% busy), where ReLU, with a fraction of the arithmetic, takes 66 with it.
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

// dz of E elements (ACT 0: dout itself).
template <int ACT, int DK, int E>
__device__ __forceinline__ void grad(const Raw<DK, E>& dout, const Raw<1, E>& pre, float (&z)[E]) {
  widen_raw(dout, z);
  if constexpr (ACT != 0) {
    float f[E];
    widen_raw(pre, f);
#pragma unroll
    for (int i = 0; i < E; ++i) z[i] *= act_grad<ACT>(f[i]);
  }
}

template <int DK, int ACT, int E, bool ONCE = false>
__device__ __forceinline__ void grad(const EpiBwdArgs& p, int64_t row, int64_t c, float (&z)[E]) {
  const Raw<DK, E> dout = load_raw<DK, E, ONCE>(p.dout, row * p.lddout + c);
  Raw<1, E> pre = {};
  if constexpr (ACT != 0) pre = load_raw<1, E, ONCE>(p.pre, row * p.ldpre + c);
  grad<ACT>(dout, pre, z);
}

// Where the launches are short, dbias without a second one: the first workgroups
// of the grid take kFewCols columns each over all rows (four lanes of eight
// columns, NT / 4 rows at a time) and compute dz once more, its inputs then
// coming from L2. 64 columns would leave the arithmetic of 1091 x 768 on 12 CUs
// (12.5 us; 8.0 at 32, 6.6 at 16), 16 columns read 32-byte pieces (328 x 3328
// 5.9 us at 64, 5.1 at 32, 6.5 at 16).
constexpr int kFewCols = 32;

template <int DK, int ACT, int NT>
__device__ __forceinline__ void few_rows_dbias(const EpiBwdArgs& p, int group) {
  constexpr int CL = kFewCols / 8, RL = NT / CL;
  __shared__ float red[RL][8 * CL];
  const int rl = threadIdx.x / CL, c = (group * CL + threadIdx.x % CL) * 8;
  float acc[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) acc[k] = 0.0f;
  constexpr int U = 2;  // rows in flight per thread
  for (int64_t r0 = rl; r0 < p.rows; r0 += U * RL) {
    Raw<DK, 8> d[U];
    Raw<1, 8> pre[U] = {};
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t r = r0 + u * RL < p.rows ? r0 + u * RL : r0;  // past the end: a row again, not counted
      d[u] = load_raw<DK, 8>(p.dout, r * p.lddout + c);
      if (ACT != 0) pre[u] = load_raw<1, 8>(p.pre, r * p.ldpre + c);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float z[8];
      grad<ACT>(d[u], pre[u], z);
      if (r0 + u * RL < p.rows) {
#pragma unroll
        for (int k = 0; k < 8; ++k) acc[k] += z[k];
      }
    }
  }
  column_sums_of_lanes<RL, CL>(acc, red, p.dbias + group * kFewCols);
}

// The same as a launch of its own, before the codes: dz written over dout would
// change dout under the sums. NT as in the launch with the codes, so that the
// order of the sums is that one's.
template <int DK, int ACT, int NT>
__global__ __launch_bounds__(NT) void epi_bwd_dbias(const EpiBwdArgs p) {
  few_rows_dbias<DK, ACT, NT>(p, blockIdx.x);
}

// How a launch treats its data: FEW: dbias by few_rows_dbias in the same launch;
// ONCE: nontemporal loads of the inputs and stores of the codes.
enum Form { kPlain = 0, kFew = 1, kOnce = 2 };

// One g x g block per workgroup of NT threads; dz in registers between the amax
// and the encode.
template <int DK, int ACT, int G, int NT, int FORM>
__global__ __launch_bounds__(NT) void epi_bwd_blocks(const EpiBwdArgs p, float* part, int col_wgs) {
  constexpr bool ONCE = FORM == kOnce;
  if constexpr (FORM == kFew) {
    if ((int)blockIdx.x < col_wgs) return few_rows_dbias<DK, ACT, NT>(p, blockIdx.x);
  }
  const int block = blockIdx.x - (FORM == kFew ? col_wgs : 0);
  constexpr int E = 8;  // four for FP32: twice the passes, 8192 x 8192 81.6 -> 85.2 us
  constexpr int ROW_L = G / E;    // lanes per block row
  constexpr int RPP = NT / ROW_L;  // block rows covered by one pass
  constexpr int PASSES = G / RPP;
  static_assert(PASSES * RPP == G, "passes");
  __shared__ float red[NT / 64];
  __shared__ float sums[FORM == kFew ? 1 : RPP][G];
  const int ncb = (int)(p.cols / G);
  const int rb = block / ncb, cb = block % ncb;
  const int t = threadIdx.x, rsub = t / ROW_L, cl = t % ROW_L;
  const int64_t c = (int64_t)cb * G + cl * E;

  float z[PASSES][E], acc[E];
  float amax = 0.0f;
#pragma unroll
  for (int k = 0; k < E; ++k) acc[k] = 0.0f;
#pragma unroll
  for (int i = 0; i < PASSES; ++i) {
    const int64_t r = (int64_t)rb * G + i * RPP + rsub;
    if (r < p.rows) {
      grad<DK, ACT, E, ONCE>(p, r, c, z[i]);
      amax = fmaxf(amax, amax_of(z[i]));
#pragma unroll
      for (int k = 0; k < E; ++k) acc[k] += z[i][k];
    }
  }
  amax = group_max<64>(amax);
  if ((t & 63) == 0) red[t >> 6] = amax;
  if (FORM != kFew && part) {
#pragma unroll
    for (int k = 0; k < E; ++k) sums[rsub][cl * E + k] = acc[k];
  }
  __syncthreads();
  DG_STEP_SYNC_WG();
  amax = red[0];
#pragma unroll
  for (int w = 1; w < NT / 64; ++w) amax = fmaxf(amax, red[w]);
  DG_STEP_SYNC_WG();
  const float s = block_scale(amax, format_max(p.fmt));
  const float inv = 1.0f / s;
  if (t == 0) p.scales[block] = s;
#pragma unroll
  for (int i = 0; i < PASSES; ++i) {
    const int64_t r = (int64_t)rb * G + i * RPP + rsub;
    if (r < p.rows) {
      store_codes<ONCE>(p.q + r * p.cols + c, z[i], s, inv, p.fmt);
      if (p.dz) store_raw<ONCE>(p.dz, r * p.cols + c, round_raw<DK>(z[i]));
    }
  }
  if (FORM != kFew && part && t < G) {
    float v = sums[0][t];
#pragma unroll
    for (int i = 1; i < RPP; ++i) v += sums[i][t];
    part[(int64_t)rb * p.cols + (int64_t)cb * G + t] = v;
  }
}

// 1 x g: 64 units of columns per workgroup, its 16 waves (NW) a row each. The rows a
// workgroup takes lie ranges * NW apart, so that all workgroups advance through
// memory together: contiguous row ranges kept 128 distant places of it open at
// once and took 86 us where this takes 78 (8192 x 8192, BF16, GELU). Several
// rows in flight per wave measured slower (85), fewer waves per workgroup the
// same but for more partial rows (2000 x 7168, FP32: 23.0 us at 4 waves, 21.3
// at 16).
constexpr int NW = 16;
constexpr int row_cols(int dk) { return 64 * unit_of(dk, 1); }  // columns of a workgroup

template <int DK, int ACT, int FORM>
__global__ __launch_bounds__(64 * NW) void epi_bwd_rows(const EpiBwdArgs p, float* part, int col_groups, int ranges,
                                                        int col_wgs) {
  if constexpr (FORM == kFew) {
    if ((int)blockIdx.x < col_wgs) return few_rows_dbias<DK, ACT, 64 * NW>(p, blockIdx.x);
  }
  const int block = blockIdx.x - (FORM == kFew ? col_wgs : 0);
  constexpr int E = unit_of(DK, 1), COLS = row_cols(DK);
  __shared__ float sums[FORM == kFew ? 1 : NW][COLS];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int cg = block % col_groups, rr = block / col_groups;
  const int64_t c = (int64_t)cg * COLS + lane * E;
  const int gshift = 31 - __builtin_clz(p.gran);
  const int64_t segs = p.cols >> gshift;
  float acc[E];
#pragma unroll
  for (int k = 0; k < E; ++k) acc[k] = 0.0f;
  if (c < p.cols) {  // whole segments are live or not, so each reduction stays inside live lanes
    for (int64_t r = (int64_t)NW * rr + wave; r < p.rows; r += (int64_t)NW * ranges) {
      float z[E];
      grad<DK, ACT>(p, r, c, z);
#pragma unroll
      for (int k = 0; k < E; ++k) acc[k] += z[k];
      const float s = block_scale(segment_max<E>(amax_of(z), p.gran), format_max(p.fmt));
      store_codes(p.q + r * p.cols + c, z, s, 1.0f / s, p.fmt);
      if (((int)c & (p.gran - 1)) == 0) p.scales[r * segs + (c >> gshift)] = s;
      if (p.dz) store_raw(p.dz, r * p.cols + c, round_raw<DK>(z));
    }
  }
  if (FORM == kFew || !part) return;
#pragma unroll
  for (int k = 0; k < E; ++k) sums[wave][lane * E + k] = acc[k];
  __syncthreads();
  DG_STEP_SYNC_WG();
  const int64_t col = (int64_t)cg * COLS + threadIdx.x;
  if (threadIdx.x < COLS && col < p.cols) {
    float v = sums[0][threadIdx.x];
#pragma unroll
    for (int w = 1; w < NW; ++w) v += sums[w][threadIdx.x];
    part[rr * p.cols + col] = v;
  }
}

// Row ranges of the 1 x g form: two workgroups per CU over all, a row per wave at
// least.
int64_t row_ranges(int64_t rows, int64_t cols, int dk) {
  const int64_t r = 512 / ((cols + row_cols(dk) - 1) / row_cols(dk)), most = (rows + NW - 1) / NW;
  return r < 1 ? 1 : r < most ? r : most;
}

// Rows and elements up to which dbias comes from the same launch (BF16, GELU or
// its tanh form): 215 x 384 3.7 us against 6.4 in two launches, 328 x 3328 5.1
// against 7.0, 1091 x 768 8.0 against 8.4, 218 x 13184 7.3 against 6.9, 1024 x
// 4096 12.3 against 9.6.
constexpr int64_t kFewRows = 1024, kFewElements = 3ll << 19;

bool few_rows(int64_t rows, int64_t cols) { return rows <= kFewRows && rows * cols <= kFewElements; }

// Partial rows of dbias (one: the sums go straight to it): a row of blocks each
// (g x g), or a row range each (1 x g).
int64_t partial_rows(int64_t rows, int64_t cols, int gran, int block_rows, int dk) {
  const int64_t n = block_rows == 1 ? row_ranges(rows, cols, dk) : (rows + gran - 1) / gran;
  return few_rows(rows, cols) ? 1 : n;
}

// kOnceBytes: 8192 x 8192 in BF16 at g = 128 73.4 -> 68.0 us nontemporally, at g
// = 64 72.7 -> 69.4 us; a matrix of 16 MB was 5% slower that way.
template <int DK, int ACT, int G, int NT>
void launch_blocks(const EpiBwdArgs& p, float* part, hipStream_t stream) {
  const dim3 grid((unsigned)(((p.rows + G - 1) / G) * (p.cols / G)));
  if (p.rows * p.cols * (InKind<DK>::kBytes + (ACT ? 2 : 0)) >= kOnceBytes)
    hipLaunchKernelGGL((epi_bwd_blocks<DK, ACT, G, NT, kOnce>), grid, dim3(NT), 0, stream, p, part, 0);
  else
    hipLaunchKernelGGL((epi_bwd_blocks<DK, ACT, G, NT, kPlain>), grid, dim3(NT), 0, stream, p, part, 0);
}

template <int DK, int ACT, int G, int NT>
void launch_blocks_few(const EpiBwdArgs& p, int col_wgs, hipStream_t stream) {
  const dim3 grid((unsigned)(((p.rows + G - 1) / G) * (p.cols / G) + col_wgs));
  hipLaunchKernelGGL((epi_bwd_blocks<DK, ACT, G, NT, kFew>), grid, dim3(NT), 0, stream, p, nullptr, col_wgs);
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
  const int64_t n = partial_rows(p.rows, p.cols, p.gran, p.block_rows, DK);
  float* part = !p.dbias ? nullptr : n > 1 ? p.ws : p.dbias;
  // one row of blocks (or one range) has dbias' sums already
  const int64_t ranges = row_ranges(p.rows, p.cols, DK);
  bool few = p.dbias && few_rows(p.rows, p.cols) && (p.block_rows == 1 ? ranges > 1 : p.rows > p.gran);
  if (few && p.dz == p.dout) {
    const dim3 grid((unsigned)(p.cols / kFewCols));
    if (p.block_rows == 64) hipLaunchKernelGGL((epi_bwd_dbias<DK, ACT, 512>), grid, dim3(512), 0, stream, p);
    else hipLaunchKernelGGL((epi_bwd_dbias<DK, ACT, 1024>), grid, dim3(1024), 0, stream, p);
    few = false;
    part = nullptr;
  }
  const int col_wgs = few ? (int)(p.cols / kFewCols) : 0;
  const int64_t blocks = ((p.rows + p.gran - 1) / p.gran) * (p.cols / p.gran);
  if (p.block_rows == 1) {
    const int64_t col_groups = (p.cols + row_cols(DK) - 1) / row_cols(DK);
    const dim3 grid((unsigned)(col_groups * ranges + col_wgs));
    if (few)
      hipLaunchKernelGGL((epi_bwd_rows<DK, ACT, kFew>), grid, dim3(64 * NW), 0, stream, p, nullptr, (int)col_groups,
                         (int)ranges, col_wgs);
    else
      hipLaunchKernelGGL((epi_bwd_rows<DK, ACT, kPlain>), grid, dim3(64 * NW), 0, stream, p, part, (int)col_groups,
                         (int)ranges, 0);
  } else if (p.gran == 64) {
    if (few) launch_blocks_few<DK, ACT, 64, 512>(p, col_wgs, stream);
    else launch_blocks<DK, ACT, 64, 256>(p, part, stream);
  } else if (p.gran == 128) {
    if (few) launch_blocks_few<DK, ACT, 128, 1024>(p, col_wgs, stream);
    else if (DK == 0 || blocks <= 1024) launch_blocks<DK, ACT, 128, 1024>(p, part, stream);
    else launch_blocks<DK, ACT, 128, 512>(p, part, stream);
  } else {
    if (few) launch_blocks_few<DK, ACT, 256, 1024>(p, col_wgs, stream);
    else launch_blocks<DK, ACT, 256, 1024>(p, part, stream);
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
  const int64_t n = partial_rows(rows, cols, gran, block_rows, 1);  // 16-bit types have at least FP32's ranges
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

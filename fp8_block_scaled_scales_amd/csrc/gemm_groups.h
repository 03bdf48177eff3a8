// Products over groups of rows (experts): which group and tile a workgroup of
// the GEMM kernels takes, from offsets that stay on the GPU. Group e's rows are
// offsets[e] .. offsets[e+1] - 1 of the sorted rows.
//
//   RowGroups    out rows of group e = A rows of group e times B_e: the groups
//                cut M, and every group has its own B and B factors
//   DepthGroups  out_e = (A rows of group e)^T (B rows of group e): the groups
//                cut K, and every group has its own out
//
// The host knows the number of rows and groups, not the groups' lengths: it
// launches as many workgroups as any lengths could need, and those beyond the
// tiles that there are end at once.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gemm_epilogue.h"

namespace dg {

struct NoGroups {
  static constexpr int kKind = 0;
};

struct RowGroups {
  static constexpr int kKind = 1;
  const int* offsets;  // [n + 1]
  int n;
  int rows;            // of A and out: no offset is taken past it
};

struct DepthGroups {
  static constexpr int kKind = 2;
  const int* offsets;
  int n;
  int rows;
};

// The start and length of group e. Offsets that do not ascend or leave 0 ..
// rows give a shorter or empty group, never a row outside.
template <class GRP>
__device__ __forceinline__ void group_range(const GRP& g, int e, int& row0, int& len) {
  const int lo = min(max(g.offsets[e], 0), g.rows), hi = min(max(g.offsets[e + 1], lo), g.rows);
  row0 = lo;
  len = hi - lo;
}

struct GroupTile {
  int group, row0, rows;  // the group's rows
  int tm, tn;             // tile row and column inside the group
};

// The tile of workgroup blockIdx.x: false (for the whole workgroup) where
// there is none. Tiles are numbered group by group, inside a group as a raster
// of GROUP_M tile rows (map_tile); each XCD takes a contiguous run of the tiles
// that there are, so a group's B stays in as few L2s as possible. Every wave
// finds its tile by itself: lane l adds the tiles of groups c*l .. c*l + c - 1
// (c = ceil(n / 64)), a scan over the lanes finds the lane, and at most c steps
// the group.
template <int BM, int GROUP_M>
__device__ __forceinline__ bool find_tile(const RowGroups& g, int tiles_n, GroupTile& t) {
  const int lane = threadIdx.x & 63;
  const int per = (g.n + 63) >> 6;
  int mine = 0;
  for (int i = 0; i < per; ++i) {
    const int e = lane * per + i;
    if (e < g.n) {
      int row0, len;
      group_range(g, e, row0, len);
      mine += (len + BM - 1) / BM;
    }
  }
  int upto = mine;  // inclusive scan
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int v = __shfl_up(upto, d, 64);
    if (lane >= d) upto += v;
  }
  const int total = __builtin_amdgcn_readlane(upto, 63) * tiles_n;
  int pid = blockIdx.x;
  if (pid >= total) return false;
  const int xcd = pid & 7, local = pid >> 3, q = total >> 3, r = total & 7;
  pid = (xcd < r ? xcd * (q + 1) : r * (q + 1) + (xcd - r) * q) + local;
  const int at = pid / tiles_n;  // tile rows before it, over all groups
  const uint64_t before = __ballot(upto <= at);  // lanes whose groups all come before
  const int l = __builtin_popcountll(before);
  int base = __builtin_amdgcn_readlane(upto - mine, l);
  int e = l * per, row0, len, tiles_m;
  for (;; ++e) {
    group_range(g, e, row0, len);
    tiles_m = (len + BM - 1) / BM;
    if (at < base + tiles_m || e + 1 >= g.n) break;
    base += tiles_m;
  }
  t.group = __builtin_amdgcn_readfirstlane(e);
  t.row0 = __builtin_amdgcn_readfirstlane(row0);
  t.rows = __builtin_amdgcn_readfirstlane(len);
  const int in = pid - base * tiles_n, strip = GROUP_M * tiles_n;
  const int first = in / strip * GROUP_M, high = min(tiles_m - first, GROUP_M), rest = in % strip;
  t.tm = __builtin_amdgcn_readfirstlane(first + rest % high);
  t.tn = __builtin_amdgcn_readfirstlane(rest / high);
  return true;
}

// For DepthGroups: every group has the same tiles_m x tiles_n tiles, and each
// XCD takes an eighth of every group's raster, since a group's length is the
// work of its tiles: whole groups per XCD would leave the XCDs of short groups
// idle. Where a group has too few tiles for every XCD, the next group begins
// with those that had none.
__host__ __device__ constexpr int64_t depth_tiles_per_xcd(int64_t tiles) { return (tiles + 7) / 8; }

template <int GROUP_M>
__device__ __forceinline__ bool find_tile(const DepthGroups& g, int tiles_m, int tiles_n, GroupTile& t) {
  const int tiles = tiles_m * tiles_n, per = (int)depth_tiles_per_xcd(tiles);
  const int xcd = blockIdx.x & 7, local = blockIdx.x >> 3;
  t.group = local / per;
  const int used = (tiles + per - 1) / per;
  const int in = ((xcd + t.group * used) & 7) * per + local % per;
  if (in >= tiles || t.group >= g.n) return false;
  const int strip = GROUP_M * tiles_n;
  const int first = in / strip * GROUP_M, high = min(tiles_m - first, GROUP_M), rest = in % strip;
  t.tm = first + rest % high;
  t.tn = rest / high;
  group_range(g, t.group, t.row0, t.rows);
  return true;
}

// The kernel's arguments as they are for the tile's group alone. sg: rows of a
// factor block; rowa: a factor per row of A.
template <class GRP>
__device__ __forceinline__ void enter_group(const GroupTile& t, int sg, bool rowa, const uint8_t* __restrict__& a,
                                            const uint8_t* __restrict__& b, const float* __restrict__& sa,
                                            const float* __restrict__& sb, uint16_t* __restrict__& out, EpiArgs& epi,
                                            int& M, int& N, int& K) {
  if constexpr (GRP::kKind == 1) {
    const int nks = K / sg;
    a += (int64_t)t.row0 * K;
    sa += (int64_t)(rowa ? t.row0 : t.row0 / sg) * nks;
    b += (int64_t)t.group * N * K;
    sb += (int64_t)t.group * ((N + sg - 1) / sg) * nks;
    epi.out += (int64_t)t.row0 * N;
    if (epi.pre) epi.pre += (int64_t)t.row0 * N;
    M = t.rows;
  } else {
    a += (int64_t)t.row0 * M;
    b += (int64_t)t.row0 * N;
    sa += (int64_t)(t.row0 / sg) * ((M + sg - 1) / sg);
    sb += (int64_t)(t.row0 / sg) * ((N + sg - 1) / sg);
    out += (int64_t)t.group * M * N;
    K = t.rows;
  }
}

}  // namespace dg

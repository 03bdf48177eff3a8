// The products of groups of rows (gemm_groups.h), out rows of group e = act(A
// rows of group e times B_e^T) with the pre-activation where it is kept: the
// streaming, 64x64 and tiled entries, B stored [N,K] or [K,N]; the 256-row
// entries are in gemm_fp8_grouped_big.hip. One launch for all groups: their
// tiles fill the chip together, where a launch per group would leave most CUs
// idle (64 groups of 8 rows, 4096 x 2048: 95 us in one, of which reading the
// 537 MB of weights takes 92 at the rate of a copy). With few rows per group the
// weights' bytes bound it; the 128x128 tile streams them best (forced: 32x32 165 us,
// 64x64 152, 256x256 132), although its rows are mostly empty there.

#include <hip/hip_runtime.h>

#include "gemm_fp8_nt.h"
#include "gemm_fp8_stream.h"
#include "gemm_fp8_tiled.h"

namespace dg {

namespace {

template <bool ROWA, int LAYOUT>
hipError_t launch(int id, const GemmArgs& p, const RowGroups& g, int64_t grid, hipStream_t stream) {
  switch (id) {
    case 0: return launch_tiled_groups<128, 128, 2, 2, 2, 128, ROWA, LAYOUT>(p, g, grid, stream);
    case 1: return launch_tiled_groups<128, 128, 2, 2, 2, 64, ROWA, LAYOUT>(p, g, grid, stream);
    case 2: return launch_tiled_groups<64, 64, 2, 2, 8, 128, ROWA, LAYOUT>(p, g, grid, stream);
    case 3: return launch_tiled_groups<64, 64, 2, 2, 8, 64, ROWA, LAYOUT>(p, g, grid, stream);
    case 6: return stream::launch_groups<128, ROWA, LAYOUT>(p, g, grid, stream);
    case 7: return stream::launch_groups<64, ROWA, LAYOUT>(p, g, grid, stream);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace

hipError_t launch_grouped(int id, const GemmArgs& p, const RowGroups& g, int64_t grid, hipStream_t stream) {
  if (id == 4 || id == 5 || id == 9 || id == 10) return launch_grouped_big(id, p, g, grid, stream);
  if (p.rowa) return p.layout ? launch<true, 1>(id, p, g, grid, stream) : launch<true, 0>(id, p, g, grid, stream);
  return p.layout ? launch<false, 1>(id, p, g, grid, stream) : launch<false, 0>(id, p, g, grid, stream);
}

}  // namespace dg

// The products of groups of rows on the 256-row tiles of gemm_fp8_big.h. Its
// own translation unit, so these instances compile beside the others. What
// bounds them is the plain tile's operand traffic and matrix work, plus the part
// tiles at the groups' ends and the tail of the last round: 32768 rows in 32
// unequal groups, 8192 x 2048, g x g factors, 680 us (1.62 PFLOP/s), 772 with GELU,
// 825 with GELU and the pre-activation kept (0.54 GB more); on 256x128 tiles 1086,
// on 128x128 998. Workgroups that take several tiles in turn were 12 to 30% slower:
// the loop's state spills scalar registers.

#include <hip/hip_runtime.h>

#include "gemm_fp8_big.h"
#include "gemm_fp8_nt.h"

namespace dg {

namespace {

template <bool ROWA, int LAYOUT>
hipError_t launch(int id, const GemmArgs& p, const RowGroups& g, int64_t grid, hipStream_t stream) {
  switch (id) {
    case 4: return big::launch_groups<128, 256, 2, ROWA, LAYOUT>(p, g, grid, stream);
    case 5: return big::launch_groups<64, 256, 2, ROWA, LAYOUT>(p, g, grid, stream);
    case 9: return big::launch_groups<128, 128, 4, ROWA, LAYOUT>(p, g, grid, stream);
    case 10: return big::launch_groups<64, 128, 4, ROWA, LAYOUT>(p, g, grid, stream);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace

hipError_t launch_grouped_big(int id, const GemmArgs& p, const RowGroups& g, int64_t grid, hipStream_t stream) {
  if (p.rowa) return p.layout ? launch<true, 1>(id, p, g, grid, stream) : launch<true, 0>(id, p, g, grid, stream);
  return p.layout ? launch<false, 1>(id, p, g, grid, stream) : launch<false, 0>(id, p, g, grid, stream);
}

}  // namespace dg

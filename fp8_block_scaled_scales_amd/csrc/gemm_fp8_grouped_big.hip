// The products of groups of rows on the 256-row tiles of gemm_fp8_big.h. Its
// own translation unit, so these instances compile beside the others.

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

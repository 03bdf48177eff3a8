// The gradient of the groups' weights, out_e = (A rows of group e)^T (B rows of
// group e): both operands as they are stored, row by row, which is the [K,M] and
// [K,N] layout of the product with the group's rows as K (gemm_groups.h). Bound by
// the plain TN tile's rate and, since K is short, by every tile's first loads and
// its store: 32768 rows in 32 groups, 8192 x 2048, 701 us (1.57 PFLOP/s; 734 to 756
// with ordinary stores of the 1.07 GB that no cache holds, 934 on 128x128 tiles).

#include <hip/hip_runtime.h>

#include "gemm_fp8_big.h"
#include "gemm_fp8_nt.h"
#include "gemm_fp8_tiled.h"

namespace dg {

hipError_t launch_grouped_wgrad(int id, const GemmArgs& p, const DepthGroups& g, int64_t grid, hipStream_t stream) {
  switch (id) {
    case 0: return launch_tiled_groups<128, 128, 2, 2, 2, 128, false, 3>(p, g, grid, stream);
    case 1: return launch_tiled_groups<128, 128, 2, 2, 2, 64, false, 3>(p, g, grid, stream);
    case 4: return big::launch_groups<128, 256, 2, false, 3>(p, g, grid, stream);
    case 5: return big::launch_groups<64, 256, 2, false, 3>(p, g, grid, stream);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace dg

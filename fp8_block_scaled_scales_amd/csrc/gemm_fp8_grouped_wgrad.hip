// The gradient of the groups' weights, out_e = (A rows of group e)^T (B rows of
// group e): both operands as they are stored, row by row, which is the [K,M] and
// [K,N] layout of the product with the group's rows as K (gemm_groups.h).

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

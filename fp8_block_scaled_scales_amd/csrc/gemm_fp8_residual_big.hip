// The product with a residual in its epilogue (gemm_epilogue.h) on the 256-row
// tiles of gemm_fp8_big.h, every layout, g x g factors. Its own
// translation unit, so these instances compile beside the others.

#include <hip/hip_runtime.h>

#include "gemm_fp8_big.h"
#include "gemm_fp8_nt.h"

namespace dg {

hipError_t launch_residual_big(int id, const GemmArgs& p, hipStream_t stream) {
  switch (id) {
    case 4: return big::launch_res<128, 256, 2, 1>(p, stream);
    case 5: return big::launch_res<64, 256, 2, 1>(p, stream);
    case 9: return big::launch_res<128, 128, 4, 1>(p, stream);
    case 10: return big::launch_res<64, 128, 4, 1>(p, stream);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace dg

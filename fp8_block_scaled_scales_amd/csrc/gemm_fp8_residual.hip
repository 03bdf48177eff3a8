// The product with a residual in its epilogue (gemm_epilogue.h): the streaming,
// tiled and 64x64 entries, every layout and factor form; the 256-row entries
// are in gemm_fp8_residual_big.hip and gemm_fp8_residual_big_rowa.hip.

#include <hip/hip_runtime.h>

#include "gemm_fp8_nt.h"
#include "gemm_fp8_stream.h"
#include "gemm_fp8_tiled.h"

namespace dg {

hipError_t launch_residual(int id, const GemmArgs& p, hipStream_t stream) {
  switch (id) {
    case 0: return launch_tiled_res<128, 128, 2, 2, 2, 128, 4, false>(p, stream);
    case 1: return launch_tiled_res<128, 128, 2, 2, 2, 64, 4, false>(p, stream);
    case 2: return launch_tiled_res<64, 64, 2, 2, 8, 128, 4, true>(p, stream);
    case 3: return launch_tiled_res<64, 64, 2, 2, 8, 64, 4, true>(p, stream);
    case 6: return stream::launch<128, true>(p, stream);
    case 7: return stream::launch<64, true>(p, stream);
    default: return p.rowa ? launch_residual_big_rowa(id, p, stream) : launch_residual_big(id, p, stream);
  }
}

}  // namespace dg

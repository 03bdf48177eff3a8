// The streaming table entries (gemm_fp8_stream.h), every layout.

#include <hip/hip_runtime.h>

#include "gemm_fp8_nt.h"
#include "gemm_fp8_stream.h"

namespace dg {

// Every layout: the NT table entries (6, 7) and their transposed forms.
hipError_t launch_stream_g128(const GemmArgs& p, hipStream_t s) { return stream::launch<128>(p, s); }
hipError_t launch_stream_g64(const GemmArgs& p, hipStream_t s) { return stream::launch<64>(p, s); }

}  // namespace dg

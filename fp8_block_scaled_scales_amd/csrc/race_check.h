// The waits and barriers of the race check build.
#pragma once

#include <hip/hip_runtime.h>

// Race check build (compiled with -DDG_EXTRA_SYNC into libdg_sync.so): every
// pipeline step ends with all of the wave's memory operations drained (every
// copy in flight landed, every LDS read done) and, in the kernels whose waves
// share the LDS ring, a workgroup barrier (the extra barrier per buffer switch
// of the template article, §5.5). The ring's own waits and barriers are meant
// to make these redundant, so this build must give the release build's bits:
// a difference means a slot was read before its copy landed or refilled
// while still being read. DG_STEP_SYNC_WAVE is for the per-wave rings, whose
// waves run different step counts and so cannot meet at extra barriers. The
// kernels that add or compare through LDS (quant_common.h, norm_fp8.hip,
// epilogue_bwd.hip) meet once more before LDS is written and after it is read.
#ifdef DG_EXTRA_SYNC
#define DG_STEP_SYNC_WG()            \
  do {                               \
    __builtin_amdgcn_s_waitcnt(0);   \
    __syncthreads();                 \
  } while (0)
#define DG_STEP_SYNC_WAVE() __builtin_amdgcn_s_waitcnt(0)
#else
#define DG_STEP_SYNC_WG() \
  do {                    \
  } while (0)
#define DG_STEP_SYNC_WAVE() \
  do {                      \
  } while (0)
#endif

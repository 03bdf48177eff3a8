// The launches that the calls around the product make at their largest sizes,
// on the CPU: this program defines the HIP calls that the library makes (its
// own symbols come before the runtime's), so nothing is launched; every launch
// is checked against the limits of a grid (2^31 - 1 workgroups, less than 2^32
// threads) and recorded. Built and run by tests/test_launch_limits.py.
//
// Usage: launch_checks norm_bwd ROWS COLS | norm ROWS COLS | epi ROWS COLS G BLOCK_ROWS | gemm M N K
// prints one line per launch (workgroups, threads, and for the norm's kernels
// the first row), then "status S"; exit status 1 if a launch passes a limit.

#include <hip/hip_runtime.h>

#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <cstring>

#include "../../fp8_block_scaled_scales_amd/csrc/layer_ops.h"
#include "../../include/dg.h"

namespace {

bool g_passed = true;
enum { kNorm, kNormBwd, kOther } g_call = kOther;

void* addr(int i) { return reinterpret_cast<void*>((uintptr_t)(i + 1) << 52); }
float* faddr(int i) { return static_cast<float*>(addr(i)); }

}  // namespace

extern "C" {

hipError_t hipGetDevice(int* dev) {
  *dev = 0;
  return hipSuccess;
}

hipError_t hipGetDevicePropertiesR0600(hipDeviceProp_tR0600* p, int) {
  std::memset(p, 0, sizeof *p);
  std::strcpy(p->gcnArchName, "gfx950");
  return hipSuccess;
}

hipError_t hipGetLastError(void) { return hipSuccess; }

// A launch statement pushes its sizes, and the kernel's host stub pops them.
static dim3 g_grid, g_block;
static size_t g_shared;
static hipStream_t g_stream;

hipError_t __hipPushCallConfiguration(dim3 grid, dim3 block, size_t shared, hipStream_t stream) {
  g_grid = grid;
  g_block = block;
  g_shared = shared;
  g_stream = stream;
  return hipSuccess;
}

hipError_t __hipPopCallConfiguration(dim3* grid, dim3* block, size_t* shared, hipStream_t* stream) {
  *grid = g_grid;
  *block = g_block;
  *shared = g_shared;
  *stream = g_stream;
  return hipSuccess;
}

hipError_t hipLaunchKernel(const void* kernel, dim3 grid, dim3 block, void** args, size_t, hipStream_t) {
  const uint64_t wgs = grid.x, threads = wgs * block.x;
  if (wgs == 0 || wgs > 0x7fffffff || threads > 0xffffffff || grid.y != 1 || grid.z != 1) g_passed = false;
  long long row0 = -1;
  if (g_call == kNorm) row0 = static_cast<const dg::NormArgs*>(args[0])->row0;
  // the norm's backward kernel of a workgroup per row: known by its first, many launch
  static const void* by_row = nullptr;
  if (g_call == kNormBwd && block.x == 1024 && wgs > 65536) by_row = kernel;
  if (kernel == by_row) row0 = static_cast<const dg::NormBwdArgs*>(args[0])->row0;
  std::printf("%llu %u %lld\n", (unsigned long long)wgs, block.x, row0);
  return hipSuccess;
}

}  // extern "C"

int main(int argc, char** argv) {
  if (argc < 4) return 2;
  int64_t n[4] = {0, 0, 0, 0};
  for (int i = 2; i < argc && i < 6; ++i) n[i - 2] = std::strtoll(argv[i], nullptr, 10);
  int rc = 1;
  const int64_t ws = (int64_t)1 << 50;
  if (!std::strcmp(argv[1], "norm")) {
    g_call = kNorm;
    rc = dg_rmsnorm_quantize_fp8(addr(0), DG_IN_BF16, n[1], nullptr, 0, 0, faddr(1), 1e-6f, n[0], n[1], 64, DG_FMT_E4M3, nullptr,
                                 nullptr, nullptr, addr(2), faddr(3), nullptr);
  } else if (!std::strcmp(argv[1], "norm_bwd")) {
    g_call = kNormBwd;
    rc = dg_rmsnorm_backward(addr(0), DG_IN_BF16, n[1], addr(1), DG_IN_BF16, n[1], faddr(2), faddr(3), nullptr, 0, n[0], n[1], addr(4),
                             faddr(5), addr(6), ws, nullptr);
  } else if (!std::strcmp(argv[1], "epi")) {
    rc = dg_epilogue_backward_fp8(addr(0), DG_IN_BF16, n[1], addr(1), n[1], DG_ACT_GELU, n[0], n[1], (int)n[2], (int)n[3], DG_FMT_E5M2,
                                  nullptr, faddr(2), addr(3), faddr(4), addr(5), ws, nullptr);
  } else if (!std::strcmp(argv[1], "gemm")) {
    rc = dg_gemm_fp8_residual(addr(0), addr(1), faddr(2), faddr(3), addr(4), n[0], n[1], n[2], 128, DG_LAYOUT_NT, 128, DG_FMT_E4M3,
                              DG_FMT_E4M3, nullptr, DG_ACT_GELU, addr(5), DG_IN_BF16, n[1], nullptr, nullptr, 0, nullptr);
  }
  std::printf("status %d\n", rc);
  return g_passed ? 0 : 1;
}

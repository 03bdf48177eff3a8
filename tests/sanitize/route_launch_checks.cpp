// The launches that the calls of experts and adapters make, on the CPU, as
// launch_checks.cpp does it for the calls around the product: HIP calls that
// launch nothing, every launch checked against the limits of a grid (2^31 - 1
// workgroups, less than 2^32 threads). Built and run by
// tests/test_route_launch_limits.py.
//
// Usage: route_launch_checks sort TOKENS K GROUPS ALIGN | rows TOKENS K COLS G BLOCK_ROWS TYPE ROWS |
//   combine TOKENS K COLS TYPE | weights TOKENS K COLS TYPE | grouped ROWS GROUPS N K G LAYOUT SA_ROWS |
//   wgrad ROWS GROUPS M N G | lora TOKENS GROUPS N K RANK OUT_TYPE
// prints "workgroups threads" per launch, then "status S"; exit status 1 if a
// launch passes a limit.

#include <hip/hip_runtime.h>

#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <cstring>

#include "../../include/dg.h"

namespace {

bool g_passed = true;

void* addr(int i) { return reinterpret_cast<void*>((uintptr_t)(i + 1) << 52); }
float* faddr(int i) { return static_cast<float*>(addr(i)); }
int32_t* iaddr(int i) { return static_cast<int32_t*>(addr(i)); }

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

hipError_t hipLaunchKernel(const void*, dim3 grid, dim3 block, void**, size_t, hipStream_t) {
  const uint64_t wgs = grid.x, threads = wgs * block.x;
  if (wgs == 0 || wgs > 0x7fffffff || threads > 0xffffffff || grid.y != 1 || grid.z != 1) g_passed = false;
  std::printf("%llu %u\n", (unsigned long long)wgs, block.x);
  return hipSuccess;
}

}  // extern "C"

int main(int argc, char** argv) {
  if (argc < 2) return 2;
  int64_t n[8] = {0};
  for (int i = 2; i < argc && i < 10; ++i) n[i - 2] = std::strtoll(argv[i], nullptr, 10);
  const char* what = argv[1];
  const int64_t ws = (int64_t)1 << 50;
  int rc = 1;
  if (!std::strcmp(what, "sort"))
    rc = dg_route_sort(addr(0), 8, n[0], (int)n[1], (int)n[2], (int)n[3], iaddr(1), iaddr(2), iaddr(3),
                       dg_route_rows(n[0], (int)n[1], (int)n[2], (int)n[3]), addr(4), ws, nullptr);
  else if (!std::strcmp(what, "rows"))
    rc = dg_route_quantize_fp8(addr(0), (int)n[5], n[2], n[0], n[2], (int)n[1], iaddr(1), iaddr(2), n[6], faddr(3), (int)n[3],
                               (int)n[4], DG_FMT_E5M2, addr(4), faddr(5), addr(6), ws, nullptr);
  else if (!std::strcmp(what, "combine"))
    rc = dg_route_combine(addr(0), (int)n[3], n[2], n[0] * n[1], n[0], n[2], (int)n[1], iaddr(1), faddr(2), nullptr, 0, addr(3),
                          DG_IN_BF16, nullptr);
  else if (!std::strcmp(what, "weights"))
    rc = dg_route_weight_grad(addr(0), DG_IN_BF16, n[2], addr(1), (int)n[3], n[2], n[0] * n[1], n[0], n[2], (int)n[1], iaddr(2),
                              faddr(3), nullptr);
  else if (!std::strcmp(what, "grouped"))
    rc = dg_gemm_fp8_grouped(addr(0), addr(1), faddr(2), faddr(3), iaddr(4), (int)n[1], addr(5), n[0], n[2], n[3], (int)n[4],
                             (int)n[5], (int)n[6], DG_FMT_E4M3, DG_FMT_E4M3, DG_ACT_NONE, nullptr, nullptr);
  else if (!std::strcmp(what, "wgrad"))
    rc = dg_gemm_fp8_grouped_wgrad(addr(0), addr(1), faddr(2), faddr(3), iaddr(4), (int)n[1], addr(5), n[0], n[2], n[3], (int)n[4],
                                   DG_FMT_E5M2, DG_FMT_E4M3, nullptr);
  else if (!std::strcmp(what, "lora"))
    rc = dg_lora(addr(0), DG_IN_BF16, n[3], n[0], n[3], addr(1), addr(2), nullptr, n[2], (int)n[4], (int)n[1], iaddr(3), iaddr(4),
                 iaddr(5), addr(6), n[2], addr(7), (int)n[5], addr(8), ws, nullptr);
  std::printf("status %d\n", rc);
  return g_passed ? 0 : 1;
}

// Internal interface of the operators around the product: the norm that
// feeds it (norm_fp8.hip) and the gradient through its epilogue
// (epilogue_bwd.hip). Element kinds: 0 FP32, 1 BF16, 2 FP16, 3 absent.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace dg {

constexpr int kAbsent = 3;

struct NormArgs {
  const void* x;  // [rows][cols], row pitch ldx elements, kind xk
  const void* res;  // kind rk (kAbsent: none), row pitch ldres
  const float* w;
  void* h;       // kind rk, [rows][cols]; may be res itself (written where it was read)
  void* y;       // kind xk, or null
  float* rstd;   // [rows], or null
  uint8_t* q;
  float* scales;  // [rows][cols/gran]
  int64_t rows, cols, ldx, ldres;
  float eps;
  int gran, fmt, xk, rk;
  int gshift, segs;  // log2(gran), cols / gran
  int64_t row0;      // a launch's first row
};

struct NormBwdArgs {
  const void* dy;  // kind dk, pitch lddy
  const void* h;   // kind hk, pitch ldh
  const float* rstd;
  const float* w;
  const void* dh;  // kind hk, pitch lddh, or null
  void* dx;        // kind hk, [rows][cols]; may be dh itself
  float* dw;
  float* ws;       // partial column sums (norm_bwd_workspace bytes)
  int64_t rows, cols, lddy, ldh, lddh;
  int dk, hk;
  int64_t row0;  // a launch's first row, where rows take several
};

struct EpiBwdArgs {
  const void* dout;     // kind dk, pitch lddout
  const uint16_t* pre;  // BF16, pitch ldpre; null without an activation
  void* dz;             // kind dk, or null
  float* dbias;         // [cols], or null
  uint8_t* q;
  float* scales;  // [ceil(rows/block_rows)][cols/gran]
  float* ws;      // partial column sums (epi_bwd_workspace bytes), used with dbias
  int64_t rows, cols, lddout, ldpre;
  int gran, block_rows, fmt, dk, act;
};

hipError_t launch_norm(const NormArgs& p, hipStream_t stream);
int64_t norm_bwd_workspace(int64_t rows, int64_t cols);  // bytes; no HIP call
hipError_t launch_norm_bwd(const NormBwdArgs& p, hipStream_t stream);
int64_t epi_bwd_workspace(int64_t rows, int64_t cols, int gran, int block_rows);
hipError_t launch_epi_bwd(const EpiBwdArgs& p, hipStream_t stream);

// out[c] = sum over p of part[p][c], p = 0 .. n-1, cols a multiple of 64.
hipError_t launch_column_sum(const float* part, int64_t n, int64_t cols, float* out, hipStream_t stream);

}  // namespace dg

// Internal interface of the operators of layers whose weights each row chooses:
// the sort of rows by group and what moves rows there and back (route.hip), and
// the low-rank adapters (lora.hip). Element kinds as in layer_ops.h.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace dg {

struct SortArgs {
  const void* ids;  // [n], int32 or int64
  int wide;         // int64
  int64_t n;
  int groups, align;
  int* offsets;   // [groups + 1]
  int* position;  // [n]
  int* slot;      // [rows]
  int64_t rows;
  int* hist;      // [chunks][groups] (sort_workspace bytes)
  int chunks;     // 0 in a call of one workgroup
  int per;        // slots of a chunk
};

struct RouteQuantArgs {
  const void* x;  // kind xk, pitch ldx
  int64_t ldx, tokens, cols;
  int k;
  const int* position;   // [tokens][k]
  const int* slot;       // [rows]
  const float* weights;  // [tokens][k], or null
  int64_t rows;
  uint8_t* q;
  float* scales;
  float* ws;  // g x g blocks by tokens: their segment maxima, then the blocks' reciprocal factors (route_quant_workspace bytes)
  int gran, block_rows, fmt, xk;
};

struct CombineArgs {
  const void* y;  // kind yk, pitch ldy, rows of them
  int64_t ldy, rows, tokens, cols;
  int k;
  const int* position;
  const float* weights;  // or null
  const void* res;       // kind ok, pitch ldres, or null
  int64_t ldres;
  void* out;  // kind ok
  int yk, ok;
};

struct WeightGradArgs {
  const void* x;  // kind xk, pitch ldx
  const void* y;  // kind yk, pitch ldy
  int64_t ldx, ldy, rows, tokens, cols;
  int k;
  const int* position;
  float* dw;
  int xk, yk;
};

struct LoraArgs {
  const void* x;  // kind xk, pitch ldx
  const void* a;  // [groups][rank][K]
  const void* b;  // [groups][N][rank]
  const float* scale;  // [groups], or null
  const int* offsets;
  const int* position;
  const int* slot;
  const void* base;  // kind ok, pitch ldbase, or null
  void* out;         // kind ok, [tokens][N]; may be base
  float* ws;         // [splits][tokens][rank]
  int64_t ldx, ldbase, tokens, N, K;
  int rank, groups, xk, ok;
  int splits;
};

int64_t sort_workspace(int64_t n, int groups);  // bytes; no HIP call
hipError_t launch_sort(const SortArgs& p, hipStream_t stream);
int64_t route_quant_workspace(int64_t tokens, int64_t cols, int64_t rows, int gran, int block_rows);
hipError_t launch_route_quant(const RouteQuantArgs& p, hipStream_t stream);
hipError_t launch_combine(const CombineArgs& p, hipStream_t stream);
hipError_t launch_weight_grad(const WeightGradArgs& p, hipStream_t stream);
int lora_splits(int64_t tokens, int64_t K, int groups);
hipError_t launch_lora(const LoraArgs& p, hipStream_t stream);

}  // namespace dg

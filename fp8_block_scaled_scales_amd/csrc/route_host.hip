// Host side of the calls of layers whose weights each row chooses (experts,
// adapters): argument checks, tile choice of the grouped products and launch.

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdio>

#include "../../include/dg.h"
#include "gemm_fp8_nt.h"
#include "gemm_groups.h"
#include "host_checks.h"
#include "layer_ops.h"
#include "route_ops.h"

using namespace dg;

namespace {

bool good_fmt(int f) { return f == DG_FMT_E4M3 || f == DG_FMT_E5M2; }
bool good_groups(int groups) { return groups > 0 && groups <= DG_MAX_GROUPS; }
bool good_rows(int64_t rows) { return rows > 0 && rows <= DG_MAX_DIM; }
bool good_slots(int64_t tokens, int k) { return tokens > 0 && k > 0 && tokens <= DG_MAX_DIM && tokens * k <= DG_MAX_DIM; }

int done(hipError_t err) {
  t_last_hip = err;
  return err == hipSuccess ? DG_OK : DG_ELAUNCH;
}

int64_t sorted_rows(int64_t tokens, int k, int groups, int align) {
  if (!good_slots(tokens, k) || !good_groups(groups) || align < 1 || align > DG_MAX_DIM) return DG_EINVAL;
  const int64_t n = tokens * k, most = n + std::min<int64_t>(groups, n) * (align - 1);
  const int64_t rows = most / align * align;
  return rows <= DG_MAX_DIM ? rows : (int64_t)DG_EINVAL;
}

int64_t sort_bytes(int64_t tokens, int k, int groups) {
  return good_slots(tokens, k) && good_groups(groups) ? sort_workspace(tokens * k, groups) : (int64_t)DG_EINVAL;
}

int sort(const void* ids, int id_bytes, int64_t tokens, int k, int groups, int align, int32_t* offsets, int32_t* position,
         int32_t* slot, int64_t rows, void* ws, int64_t ws_bytes, void* stream) {
  if (!ids || !offsets || !position || !slot || (id_bytes != 4 && id_bytes != 8)) return DG_EINVAL;
  const int64_t least = sorted_rows(tokens, k, groups, align);
  if (least < 0 || !good_rows(rows) || rows < least) return DG_EINVAL;
  const int64_t need = sort_bytes(tokens, k, groups);
  if (ws_bytes < need || (need > 0 && !ws)) return DG_EINVAL;
  if (misaligned(ids, id_bytes) || misaligned(offsets, 4) || misaligned(position, 4) || misaligned(slot, 4) || misaligned(ws, 16))
    return DG_EALIGN;
  {
    const uint64_t n = (uint64_t)(tokens * k);
    const Range outs[] = {{offsets, 4ull * (groups + 1)}, {position, 4 * n}, {slot, 4ull * rows}, {need ? ws : nullptr, (uint64_t)need}};
    const Range ins[] = {{ids, n * id_bytes}};
    if (clash(outs, ins)) return DG_EINVAL;
  }
  const int rc = device_ready();
  if (rc != DG_OK) return rc;
  SortArgs p{};
  p.ids = ids;
  p.wide = id_bytes == 8;
  p.n = tokens * k;
  p.groups = groups;
  p.align = align;
  p.offsets = offsets;
  p.position = position;
  p.slot = slot;
  p.rows = rows;
  p.hist = static_cast<int*>(ws);
  if (log_enabled())
    std::fprintf(stderr, "dg_route_sort tokens=%lld k=%d groups=%d align=%d rows=%lld workspace %lld\n", (long long)tokens, k,
                 groups, align, (long long)rows, (long long)need);
  return done(launch_sort(p, static_cast<hipStream_t>(stream)));
}

// Blocks of a call with gran x gran factors: a workgroup of up to 1024 threads each in a grid of less than 2^32 threads.
bool good_route_blocks(int64_t rows, int64_t cols, int gran, int block_rows) {
  return block_rows == 1 || ((rows + gran - 1) / gran) * (cols / gran) <= 0x3fffff;
}

int64_t quantize_bytes(int64_t tokens, int64_t cols, int k, int64_t rows, int gran, int block_rows) {
  if (!good_slots(tokens, k) || !good_dims(tokens, cols) || !good_rows(rows) || !good_gran(gran, cols) ||
      (block_rows != gran && block_rows != 1) || !good_route_blocks(rows, cols, gran, block_rows))
    return DG_EINVAL;
  return route_quant_workspace(tokens, cols, rows, gran, block_rows);
}

int quantize_rows(const void* x, int x_type, int64_t ldx, int64_t tokens, int64_t cols, int k, const int32_t* position,
                  const int32_t* slot, int64_t rows, const float* weights, int gran, int block_rows, int fmt, void* q,
                  float* scales, void* ws, int64_t ws_bytes, void* stream) {
  if (!x || !position || !slot || !q || !scales || !known_kind(x_type) || !good_fmt(fmt)) return DG_EINVAL;
  const int64_t need = quantize_bytes(tokens, cols, k, rows, gran, block_rows);
  if (need < 0 || !good_pitch(ldx, cols)) return DG_EINVAL;
  if (ws_bytes < need || (need > 0 && !ws)) return DG_EINVAL;
  const uint64_t xs = kind_size(x_type);
  if (misaligned_rows(x, ldx, xs) || misaligned(position, 4) || misaligned(slot, 4) || misaligned(weights, 4) ||
      misaligned(q, 16) || misaligned(scales, 4) || misaligned(ws, 16))
    return DG_EALIGN;
  {
    const uint64_t n = 4ull * (uint64_t)(tokens * k);
    const Range outs[] = {{q, (uint64_t)rows * (uint64_t)cols},
                          {scales, 4ull * ((rows + block_rows - 1) / block_rows) * (cols / gran)},
                          {need ? ws : nullptr, (uint64_t)need}};
    const Range ins[] = {{x, extent(tokens, cols, ldx, xs)}, {position, n}, {slot, 4ull * rows}, {weights, n}};
    if (clash(outs, ins)) return DG_EINVAL;
  }
  const int rc = device_ready();
  if (rc != DG_OK) return rc;
  RouteQuantArgs p{};
  p.x = x;
  p.ldx = ldx;
  p.tokens = tokens;
  p.cols = cols;
  p.k = k;
  p.position = position;
  p.slot = slot;
  p.weights = weights;
  p.rows = rows;
  p.q = static_cast<uint8_t*>(q);
  p.scales = scales;
  p.ws = static_cast<float*>(ws);
  p.gran = gran;
  p.block_rows = block_rows;
  p.fmt = fmt;
  p.xk = x_type;
  if (log_enabled())
    std::fprintf(stderr, "dg_route_quantize_fp8 tokens=%lld k=%d cols=%lld rows=%lld block %dx%d fmt=%d x=%d weights=%d\n",
                 (long long)tokens, k, (long long)cols, (long long)rows, block_rows, gran, fmt, x_type, weights ? 1 : 0);
  return done(launch_route_quant(p, static_cast<hipStream_t>(stream)));
}

int combine(const void* y, int y_type, int64_t ldy, int64_t rows, int64_t tokens, int64_t cols, int k,
            const int32_t* position, const float* weights, const void* res, int64_t ldres, void* out, int out_type,
            void* stream) {
  if (!y || !position || !out || !known_kind(y_type) || !known_kind(out_type)) return DG_EINVAL;
  if (!good_slots(tokens, k) || !good_dims(tokens, cols) || !good_rows(rows) || cols % 8) return DG_EINVAL;
  if (!good_pitch(ldy, cols) || (res && !good_pitch(ldres, cols))) return DG_EINVAL;
  const uint64_t ys = kind_size(y_type), os = kind_size(out_type);
  if (misaligned_rows(y, ldy, ys) || misaligned_rows(res, ldres, os) || misaligned(out, 16) || misaligned(position, 4) ||
      misaligned(weights, 4))
    return DG_EALIGN;
  {
    const uint64_t n = 4ull * (uint64_t)(tokens * k);
    const Range outs[] = {{out, os * (uint64_t)tokens * (uint64_t)cols}};
    const Range ins[] = {{res, res ? extent(tokens, cols, ldres, os) : 0}, {y, extent(rows, cols, ldy, ys)}, {position, n}, {weights, n}};
    const bool in_place = res == out && ldres == cols;  // every element is read by the thread that then writes it
    if (clash(outs, ins, in_place ? 0 : -1, 0)) return DG_EINVAL;
  }
  const int rc = device_ready();
  if (rc != DG_OK) return rc;
  CombineArgs p{};
  p.y = y;
  p.ldy = ldy;
  p.rows = rows;
  p.tokens = tokens;
  p.cols = cols;
  p.k = k;
  p.position = position;
  p.weights = weights;
  p.res = res;
  p.ldres = ldres;
  p.out = out;
  p.yk = y_type;
  p.ok = out_type;
  if (log_enabled())
    std::fprintf(stderr, "dg_route_combine tokens=%lld k=%d cols=%lld rows=%lld y=%d out=%d weights=%d res=%d\n", (long long)tokens, k,
                 (long long)cols, (long long)rows, y_type, out_type, weights ? 1 : 0, res ? 1 : 0);
  return done(launch_combine(p, static_cast<hipStream_t>(stream)));
}

int weight_grad(const void* dout, int dout_type, int64_t lddout, const void* y, int y_type, int64_t ldy, int64_t rows,
                int64_t tokens, int64_t cols, int k, const int32_t* position, float* dweights, void* stream) {
  if (!dout || !y || !position || !dweights || !known_kind(dout_type) || !known_kind(y_type)) return DG_EINVAL;
  if (!good_slots(tokens, k) || !good_dims(tokens, cols) || !good_rows(rows) || cols % 8) return DG_EINVAL;
  if (!good_pitch(lddout, cols) || !good_pitch(ldy, cols)) return DG_EINVAL;
  const uint64_t ds = kind_size(dout_type), ys = kind_size(y_type);
  if (misaligned_rows(dout, lddout, ds) || misaligned_rows(y, ldy, ys) || misaligned(position, 4) || misaligned(dweights, 4))
    return DG_EALIGN;
  {
    const uint64_t n = 4ull * (uint64_t)(tokens * k);
    const Range outs[] = {{dweights, n}};
    const Range ins[] = {{dout, extent(tokens, cols, lddout, ds)}, {y, extent(rows, cols, ldy, ys)}, {position, n}};
    if (clash(outs, ins)) return DG_EINVAL;
  }
  const int rc = device_ready();
  if (rc != DG_OK) return rc;
  WeightGradArgs p{};
  p.x = dout;
  p.y = y;
  p.ldx = lddout;
  p.ldy = ldy;
  p.rows = rows;
  p.tokens = tokens;
  p.cols = cols;
  p.k = k;
  p.position = position;
  p.dw = dweights;
  p.xk = dout_type;
  p.yk = y_type;
  if (log_enabled())
    std::fprintf(stderr, "dg_route_weight_grad tokens=%lld k=%d cols=%lld rows=%lld dout=%d y=%d\n", (long long)tokens, k,
                 (long long)cols, (long long)rows, dout_type, y_type);
  return done(launch_weight_grad(p, static_cast<hipStream_t>(stream)));
}

// ---- the grouped products -----------------------------------------------------

int kernel_gran(int gran) { return gran > 128 ? 128 : gran; }

struct GroupPlan {
  const KernelEntry* e;
  int64_t grid;
};

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Workgroups that any lengths of the groups could need.
int64_t row_grid(const KernelEntry* e, int64_t rows, int groups, int64_t N) {
  return (rows / e->bm + std::min<int64_t>(groups, rows)) * cdiv(N, e->bn);
}

// Estimated time as the plain products' (estimate_us in dg_host.hip), for lengths
// that the host does not know: rows that each fall to any group leave so many of
// them live, and a live group is taken to be longer than n rows with the chance
// exp(-n / mean), which gives it 1 / (1 - exp(-bm / mean)) tile rows; and half a
// round more where there is more than one, since not all workgroups end
// together. A live group's weights come from HBM (5.3 TB/s) at least once: of the
// entries that this holds back alike the table's first, 128x128, is taken (200
// rows in 16 groups, 8192 x 8192: 193 us, 32x32 tiles 231; but 8 rows in 8 groups,
// 4096 x 7168: 56 and 34, the estimate's choice). On 23 shapes, 16 to 8192 tokens
// with 2 to 8 rows each in 8 to 64 groups, N and K 1024 to 8192, the entry of the
// least estimate took 1.7% longer than the fastest on average and 12% at most; with
// every group of the mean length and whole rounds 4.8% and 55%.
double estimate_groups(const KernelEntry* e, int64_t rows, int groups, int64_t N, int64_t K) {
  const double live = -groups * std::expm1((double)rows * std::log1p(-1.0 / groups));
  const double tiles = live / -std::expm1(-e->bm * live / (double)rows) * (double)cdiv(N, e->bn);
  const double rounds = tiles <= 256.0 ? 1.0 : tiles / 256.0 + 0.5;
  const double bytes = (double)(e->bm + e->bn) * (double)K;
  const double flop = 2.0 * e->bm * e->bn * (double)K;
  const double tiled = e->launch_us + rounds * (e->round_us + std::max(bytes / (e->cu_gbps * 1e3), flop / (e->cu_tflops * 1e6)));
  return std::max(tiled, live * (double)N * (double)K / 5.3e6);
}

// Threads of a launch of e: grids are limited to less than 2^32 of them.
bool runs(const KernelEntry* e, int64_t grid) { return e && grid <= 0x7fffffff && grid * 64 * e->waves <= 0xffffffffll; }

GroupPlan plan_rows(int64_t rows, int groups, int64_t N, int64_t K, int sgran) {
  const int gran = kernel_gran(sgran), force = forced_tile();
  GroupPlan p{nullptr, 0};
  double best = 0.0;
  for (int i = 0; i < kTableSize; ++i) {
    const KernelEntry* e = &kTable[i];
    if (e->gran != gran) continue;
    const double t = e->id == force ? -1.0 : estimate_groups(e, rows, groups, N, K);
    if (!p.e || t < best) {
      best = t;
      p.e = e;
    }
  }
  p.grid = row_grid(p.e, rows, groups, N);
  return p;
}

int grouped(const void* a, const void* b, const float* sa, const float* sb, const int32_t* offsets, int groups, void* out,
            int64_t rows, int64_t N, int64_t K, int gran, int layout, int sa_rows, int fmt_a, int fmt_b, int act, void* pre,
            void* stream) {
  if (!a || !b || !sa || !sb || !offsets || !out || !good_groups(groups)) return DG_EINVAL;
  if (!good_dims(rows, N) || !good_rows(K) || !good_gran(gran, K)) return DG_EINVAL;
  if (layout != DG_LAYOUT_NT && layout != DG_LAYOUT_NN) return DG_EINVAL;
  if ((sa_rows != gran && sa_rows != 1) || !good_fmt(fmt_a) || !good_fmt(fmt_b)) return DG_EINVAL;
  if (act < DG_ACT_NONE || act > DG_ACT_GELU_TANH) return DG_EINVAL;
  if (misaligned(a, 16) || misaligned(b, 16) || misaligned(sa, 4) || misaligned(sb, 4) || misaligned(offsets, 4) ||
      misaligned(out, 2) || misaligned(pre, 2))
    return DG_EALIGN;
  const GroupPlan pl = plan_rows(rows, groups, N, K, gran);
  if (!runs(pl.e, pl.grid)) return DG_EINVAL;
  {
    const uint64_t nks = (uint64_t)(K / gran), ob = 2ull * rows * N;
    const Range outs[] = {{out, ob}, {pre, ob}};
    const Range ins[] = {{a, (uint64_t)rows * K},
                         {b, (uint64_t)groups * N * K},
                         {sa, 4ull * cdiv(rows, sa_rows) * nks},
                         {sb, 4ull * groups * cdiv(N, gran) * nks},
                         {offsets, 4ull * (groups + 1)}};
    if (clash(outs, ins)) return DG_EINVAL;
  }
  const int rc = device_ready();
  if (rc != DG_OK) return rc;
  GemmArgs p{};
  p.a = static_cast<const uint8_t*>(a);
  p.b = static_cast<const uint8_t*>(b);
  p.sa = sa;
  p.sb = sb;
  p.out = static_cast<uint16_t*>(out);
  p.M = rows;
  p.N = N;
  p.K = K;
  p.gran = kernel_gran(gran);
  p.sshift = gran == 256 ? 1 : 0;
  p.fmt = (fmt_a == DG_FMT_E5M2 ? 1 : 0) | (fmt_b == DG_FMT_E5M2 ? 2 : 0);
  p.rowa = sa_rows == 1 ? 1 : 0;
  p.layout = layout;
  p.ksplit = 1;
  p.act = act;
  p.epi.out = static_cast<uint16_t*>(out);
  p.epi.pre = static_cast<uint16_t*>(pre);
  p.epi.res_kind = kAbsent;
  p.epi.act = act;
  if (log_enabled())
    std::fprintf(stderr, "dg_gemm_fp8_grouped rows=%lld groups=%d N=%lld K=%lld g=%d layout=%d sa_rows=%d fmt=%d,%d act=%d -> kernel %d "
                 "(%dx%d) grid %lld\n", (long long)rows, groups, (long long)N, (long long)K, gran, layout, sa_rows, fmt_a, fmt_b, act,
                 pl.e->id, pl.e->bm, pl.e->bn, (long long)pl.grid);
  return done(launch_grouped(pl.e->id, p, RowGroups{offsets, groups, (int)rows}, pl.grid, static_cast<hipStream_t>(stream)));
}

// 256x256 tiles where every CU gets two of them, else 128x128. 256 / 128, in us: 8
// groups of 2000 x 2 rows, 1024 x 512 (64 tiles of 256) 21.7 / 14.5, 2048 x 1024 (256)
// 23.8 / 27.4, 4096 x 2048 (1024) 69 / 98; 64 groups of 8192 x 2 rows, 512 x 512 (256)
// 36.3 / 26.7, 768 x 512 (384) 38 / 32, 1024 x 512 (512) 40.2 / 39.7; 8 groups of 500 x
// 2 rows, 4096 x 2048 43.7 / 55.8.
GroupPlan plan_depth(int64_t M, int64_t N, int groups, int sgran) {
  const int gran = kernel_gran(sgran), force = forced_tile();
  GroupPlan p{nullptr, 0};
  const int want = cdiv(M, 256) * cdiv(N, 256) * groups >= 512 ? (gran == 128 ? 4 : 5) : (gran == 128 ? 0 : 1);
  for (int i = 0; i < kTableSize; ++i) {
    const KernelEntry* e = &kTable[i];
    if (e->gran != gran || (e->id != 0 && e->id != 1 && e->id != 4 && e->id != 5)) continue;
    if (e->id == force || (e->id == want && (!p.e || p.e->id != force))) p.e = e;
  }
  p.grid = 8 * depth_tiles_per_xcd(cdiv(M, p.e->bm) * cdiv(N, p.e->bn)) * groups;
  return p;
}

int grouped_wgrad(const void* a, const void* b, const float* sa, const float* sb, const int32_t* offsets, int groups, void* out,
                  int64_t rows, int64_t M, int64_t N, int gran, int fmt_a, int fmt_b, void* stream) {
  if (!a || !b || !sa || !sb || !offsets || !out || !good_groups(groups)) return DG_EINVAL;
  if (!good_dims(rows, M) || !good_rows(N) || !good_gran(gran, rows) || M % gran || N % gran) return DG_EINVAL;
  if (!good_fmt(fmt_a) || !good_fmt(fmt_b)) return DG_EINVAL;
  if (misaligned(a, 16) || misaligned(b, 16) || misaligned(sa, 4) || misaligned(sb, 4) || misaligned(offsets, 4) || misaligned(out, 2))
    return DG_EALIGN;
  const GroupPlan pl = plan_depth(M, N, groups, gran);
  if (!runs(pl.e, pl.grid)) return DG_EINVAL;
  {
    const Range outs[] = {{out, 2ull * groups * M * N}};
    const Range ins[] = {{a, (uint64_t)rows * M},
                         {b, (uint64_t)rows * N},
                         {sa, 4ull * (rows / gran) * (M / gran)},
                         {sb, 4ull * (rows / gran) * (N / gran)},
                         {offsets, 4ull * (groups + 1)}};
    if (clash(outs, ins)) return DG_EINVAL;
  }
  const int rc = device_ready();
  if (rc != DG_OK) return rc;
  GemmArgs p{};
  p.a = static_cast<const uint8_t*>(a);
  p.b = static_cast<const uint8_t*>(b);
  p.sa = sa;
  p.sb = sb;
  p.out = static_cast<uint16_t*>(out);
  p.M = M;
  p.N = N;
  p.K = rows;
  p.gran = kernel_gran(gran);
  p.sshift = gran == 256 ? 1 : 0;
  p.fmt = (fmt_a == DG_FMT_E5M2 ? 1 : 0) | (fmt_b == DG_FMT_E5M2 ? 2 : 0);
  p.layout = DG_LAYOUT_TN;
  p.vec_store = ((uintptr_t)out & 15) == 0 ? 1 : 0;
  p.ksplit = 1;
  if (log_enabled())
    std::fprintf(stderr, "dg_gemm_fp8_grouped_wgrad rows=%lld groups=%d M=%lld N=%lld g=%d fmt=%d,%d -> kernel %d (%dx%d) grid %lld\n",
                 (long long)rows, groups, (long long)M, (long long)N, gran, fmt_a, fmt_b, pl.e->id, pl.e->bm, pl.e->bn, (long long)pl.grid);
  return done(launch_grouped_wgrad(pl.e->id, p, DepthGroups{offsets, groups, (int)rows}, pl.grid, static_cast<hipStream_t>(stream)));
}

// ---- the adapters -------------------------------------------------------------

int64_t lora_bytes(int64_t tokens, int64_t K, int64_t N, int rank, int groups) {
  if (!good_dims(tokens, N) || !good_rows(K) || K % 8 || rank <= 0 || rank > 128 || rank % 8 || !good_groups(groups)) return DG_EINVAL;
  // at most 2^32 - 1 threads: 256 for each 16 rows by 256 columns
  if ((tokens / 16 + std::min<int64_t>(groups, tokens)) * cdiv(N, 256) + (1 << 16) > 0xffffff) return DG_EINVAL;
  return 4ll * lora_splits(tokens, K, groups) * tokens * rank;
}

int lora(const void* x, int type, int64_t ldx, int64_t tokens, int64_t K, const void* a, const void* b, const float* scale,
         int64_t N, int rank, int groups, const int32_t* offsets, const int32_t* position, const int32_t* slot, const void* base,
         int64_t ldbase, void* out, int out_type, void* ws, int64_t ws_bytes, void* stream) {
  if (!x || !a || !b || !offsets || !position || !slot || !out || !ws) return DG_EINVAL;
  if ((type != DG_IN_BF16 && type != DG_IN_F16) || !known_kind(out_type)) return DG_EINVAL;
  const int64_t need = lora_bytes(tokens, K, N, rank, groups);
  if (need < 0 || ws_bytes < need || !good_pitch(ldx, K) || (base && !good_pitch(ldbase, N))) return DG_EINVAL;
  const uint64_t os = kind_size(out_type);
  if (misaligned_rows(x, ldx, 2) || misaligned(a, 16) || misaligned(b, 16) || misaligned(scale, 4) || misaligned(offsets, 4) ||
      misaligned(position, 4) || misaligned(slot, 4) || misaligned(base, os) || misaligned(out, os) || misaligned(ws, 16))
    return DG_EALIGN;
  {
    const Range outs[] = {{out, os * (uint64_t)tokens * (uint64_t)N}, {ws, (uint64_t)need}};
    const Range ins[] = {{base, base ? extent(tokens, N, ldbase, os) : 0},
                         {x, extent(tokens, K, ldx, 2)},
                         {a, 2ull * groups * rank * K},
                         {b, 2ull * groups * rank * N},
                         {scale, 4ull * groups},
                         {offsets, 4ull * (groups + 1)},
                         {position, 4ull * tokens},
                         {slot, 4ull * tokens}};
    const bool in_place = base == out && ldbase == N;  // every element is read by the thread that then writes it
    if (clash(outs, ins, in_place ? 0 : -1, 0)) return DG_EINVAL;
  }
  const int rc = device_ready();
  if (rc != DG_OK) return rc;
  LoraArgs p{};
  p.x = x;
  p.a = a;
  p.b = b;
  p.scale = scale;
  p.offsets = offsets;
  p.position = position;
  p.slot = slot;
  p.base = base;
  p.out = out;
  p.ws = static_cast<float*>(ws);
  p.ldx = ldx;
  p.ldbase = ldbase;
  p.tokens = tokens;
  p.N = N;
  p.K = K;
  p.rank = rank;
  p.groups = groups;
  p.xk = type;
  p.ok = out_type;
  p.splits = lora_splits(tokens, K, groups);
  if (log_enabled())
    std::fprintf(stderr, "dg_lora tokens=%lld K=%lld N=%lld rank=%d groups=%d x=%d out=%d base=%d splits %d\n", (long long)tokens,
                 (long long)K, (long long)N, rank, groups, type, out_type, base ? (base == out ? 2 : 1) : 0, p.splits);
  return done(launch_lora(p, static_cast<hipStream_t>(stream)));
}

}  // namespace

extern "C" {

int dg_route_sort(const void* ids, int id_bytes, int64_t tokens, int k, int groups, int align, int32_t* offsets,
                  int32_t* position, int32_t* slot, int64_t rows, void* workspace, int64_t workspace_bytes, void* stream) {
  return sort(ids, id_bytes, tokens, k, groups, align, offsets, position, slot, rows, workspace, workspace_bytes, stream);
}

int64_t dg_route_rows(int64_t tokens, int k, int groups, int align) { return sorted_rows(tokens, k, groups, align); }

int64_t dg_route_sort_workspace(int64_t tokens, int k, int groups) { return sort_bytes(tokens, k, groups); }

int dg_route_quantize_fp8(const void* x, int x_type, int64_t ldx, int64_t tokens, int64_t cols, int k,
                          const int32_t* position, const int32_t* slot, int64_t rows, const float* weights, int gran,
                          int block_rows, int fmt, void* q, float* scales, void* workspace, int64_t workspace_bytes,
                          void* stream) {
  return quantize_rows(x, x_type, ldx, tokens, cols, k, position, slot, rows, weights, gran, block_rows, fmt, q, scales,
                       workspace, workspace_bytes, stream);
}

int64_t dg_route_quantize_workspace(int64_t tokens, int64_t cols, int k, int64_t rows, int gran, int block_rows) {
  return quantize_bytes(tokens, cols, k, rows, gran, block_rows);
}

int dg_route_combine(const void* y, int y_type, int64_t ldy, int64_t rows, int64_t tokens, int64_t cols, int k,
                     const int32_t* position, const float* weights, const void* res, int64_t ldres, void* out, int out_type,
                     void* stream) {
  return combine(y, y_type, ldy, rows, tokens, cols, k, position, weights, res, ldres, out, out_type, stream);
}

int dg_route_weight_grad(const void* dout, int dout_type, int64_t lddout, const void* y, int y_type, int64_t ldy,
                         int64_t rows, int64_t tokens, int64_t cols, int k, const int32_t* position, float* dweights,
                         void* stream) {
  return weight_grad(dout, dout_type, lddout, y, y_type, ldy, rows, tokens, cols, k, position, dweights, stream);
}

int dg_gemm_fp8_grouped(const void* a, const void* b, const float* sa, const float* sb, const int32_t* offsets,
                        int groups, void* out, int64_t rows, int64_t N, int64_t K, int gran, int layout, int sa_rows,
                        int fmt_a, int fmt_b, int act, void* pre, void* stream) {
  return grouped(a, b, sa, sb, offsets, groups, out, rows, N, K, gran, layout, sa_rows, fmt_a, fmt_b, act, pre, stream);
}

int dg_gemm_fp8_grouped_wgrad(const void* a, const void* b, const float* sa, const float* sb, const int32_t* offsets,
                              int groups, void* out, int64_t rows, int64_t M, int64_t N, int gran, int fmt_a, int fmt_b,
                              void* stream) {
  return grouped_wgrad(a, b, sa, sb, offsets, groups, out, rows, M, N, gran, fmt_a, fmt_b, stream);
}

int dg_lora(const void* x, int type, int64_t ldx, int64_t tokens, int64_t K, const void* a, const void* b,
            const float* scale, int64_t N, int rank, int groups, const int32_t* offsets, const int32_t* position,
            const int32_t* slot, const void* base, int64_t ldbase, void* out, int out_type, void* workspace,
            int64_t workspace_bytes, void* stream) {
  return lora(x, type, ldx, tokens, K, a, b, scale, N, rank, groups, offsets, position, slot, base, ldbase, out, out_type,
              workspace, workspace_bytes, stream);
}

int64_t dg_lora_workspace(int64_t tokens, int64_t K, int64_t N, int rank, int groups) {
  return lora_bytes(tokens, K, N, rank, groups);
}

}  // extern "C"

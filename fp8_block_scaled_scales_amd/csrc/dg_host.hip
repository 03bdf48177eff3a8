// Host side of the C ABI declared in include/dg.h: argument checks, the
// one-time per-device architecture check, tile-table selection and launch.
//
// Tile selection replaces a runtime JIT with a small precompiled table
// (the pages describe compiling per shape at first use, DeepGEMM实战 §2.1, and
// precompiling common shapes, the DeepGEMM-style template article §2.3/§5.3;
// this library only does the latter).

#include <hip/hip_runtime.h>

#include <cstdio>
#include <cstdlib>
#include <algorithm>
#include <cstring>
#include <mutex>

#include "../../include/dg.h"
#include "gemm_fp8_nt.h"
#include "host_checks.h"
#include "layer_ops.h"
#include "quant_fp8.h"

using namespace dg;

namespace {

constexpr int kMaxDevices = 64;
std::once_flag g_dev_once[kMaxDevices];
int g_dev_status[kMaxDevices];  // DG_OK or DG_EUNSUPPORTED, set once per device

// Split-K plans (dg_gemm_fp8_ws only) are capped at this many FP32 partial
// floats, which bounds the workspace a caller provides.
constexpr int64_t kWsFloats = 4ll << 20;  // 16 MB of partial tiles

// When a workspace plan splits K. A split costs about 2 us beyond the
// streaming kernel's time for the same K range (the FP32 partials' trip
// through memory and the second kernel), and its 64x64 tiles move fewer
// bytes per CU only when there are few of them, so it pays where it cuts a
// long K range several times: at least kSplitMinSteps 128-byte K steps and
// at least kSplitMin splits (at most 32 tiles of 64x64, whatever M). Graph-timed
// on small M (8, 64, 128 rows, N 256 to 4096, g = 128, K 1024 to 32768):
// K >= 16384 with 8 to 16 splits took 0.46 to 0.81 of the streaming time,
// and with M 192 to 2048 (N 64 to 640, K 16384 to 65536, g 64 and 128) 0.46
// to 0.90 of the planned entry's; K = 7168 with 8 to 14 splits 0.91 to
// 1.15; K <= 4096 1.05 to 1.6; 4 splits 0.95 to 1.57 at any K; 2 splits
// (M = 128, N = 4096, whose streaming tiles take two rounds) 0.87 to 1.10.
// kMaxSplit bounds the second kernel's sum per output.
constexpr int64_t kSplitMinSteps = 128;
constexpr int64_t kSplitMin = 8;

// kSplitMinSteps for the residual epilogue's form. With a transposed operand the
// streaming tiles take its K rows in 32-byte pieces at about half the rate, the
// 64x64 tiles in 64-byte ones, so a split wins earlier: 19x51x12352 TN 25.2 ->
// 11.9 us, 565x68x10240 TT 19.9 -> 13.5, 47x19x6656 TT 11.0 -> 9.9; 2x453x3840
// NN 9.5 -> 9.9. NT: 8x300x8192 9.7 -> 8.2, 64x512x8192 10.4 -> 9.2. The plain
// calls keep one plan for every layout, so that every layout gives the same
// bits.
constexpr int64_t kSplitMinStepsT = 48, kSplitMinStepsR = 64;

int64_t residual_split_steps(int layout) { return layout != DG_LAYOUT_NT ? kSplitMinStepsT : kSplitMinStepsR; }
constexpr int64_t kMaxSplit = 16;

// Workspace layout of a split-K plan: the FP32 partial tiles,
// [tile][split][bm][bn], row-major inside a tile.

// The workspace of dg_gemm_fp8_noalloc, for callers that cannot allocate
// device memory: a fixed array in the library's code object, one copy per GPU
// the library runs on, held until the process ends. Its host-side name is a
// stand-in, not a device address: the device address is looked up once per
// device (hipGetSymbolAddress, with that device current) and only that
// address is passed to kernels. A split-K call writes every partial it
// reads, so the array's contents never matter.
constexpr int64_t kScratchBytes = 4ll << 20;
static __device__ __align__(256) unsigned char scratch[kScratchBytes];
std::once_flag g_scratch_once[kMaxDevices];
void* g_scratch[kMaxDevices];
hipError_t g_scratch_err[kMaxDevices];

void find_scratch(int dev) {
  void* p = nullptr;
  g_scratch_err[dev] = hipGetSymbolAddress(&p, HIP_SYMBOL(scratch));
  g_scratch[dev] = g_scratch_err[dev] == hipSuccess ? p : nullptr;
}

thread_local char t_msg[256];

void check_device(int dev) {
  hipDeviceProp_t prop;
  if (hipGetDeviceProperties(&prop, dev) != hipSuccess) {
    g_dev_status[dev] = DG_EUNSUPPORTED;
    return;
  }
  g_dev_status[dev] = std::strncmp(prop.gcnArchName, "gfx950", 6) == 0 ? DG_OK : DG_EUNSUPPORTED;
}

// Argument checks shared by the GEMM and the tile query. No HIP call.
int validate(int64_t M, int64_t N, int64_t K, int gran) {
  if (M <= 0 || N <= 0 || K <= 0) return DG_EINVAL;
  if (M > DG_MAX_DIM || N > DG_MAX_DIM || K > DG_MAX_DIM) return DG_EINVAL;
  if (gran != 64 && gran != 128 && gran != 256) return DG_EINVAL;
  if (K % gran != 0) return DG_EINVAL;
  return DG_OK;
}

// K segment the kernels contract before each promotion: g itself for 64 and
// 128; g = 256 runs the 128 kernels with one scale factor per two segments.
int kernel_gran(int gran) { return gran > 128 ? 128 : gran; }

const dg::KernelEntry* find(int cls, int gran) {
  for (int i = 0; i < dg::kTableSize; ++i)
    if (dg::kTable[i].gran == gran && dg::kTable[i].cls == cls) return &dg::kTable[i];
  return nullptr;
}

struct Plan {
  const dg::KernelEntry* e;
  int ksplit;
  int64_t tiles;
};

// Tile-table choice (pure host arithmetic, no HIP call).
// Every shape takes the table entry of the call's granularity with the least
// estimated time (estimate_us), the whole K per workgroup: the 32x32
// streaming tiles (whose waves split K inside the workgroup), 64x64,
// 128x128, or the 256-row tiles 128 or 256 wide. With a workspace, a long K
// (kSplitMinSteps) that gives at least kSplitMin splits instead splits the
// K range of each 64x64 tile over several workgroups, until about
// one workgroup per CU (256) runs, at most kMaxSplit per tile and at least 4
// pipeline steps per split.
// DG_FORCE_TILE=<kernel id>, read at every call, replaces the choice when
// that entry has the call's granularity (tuning, benchmarking and tests; a
// split-K entry then runs with one split unless the call has a workspace).
int64_t splits_for(const dg::KernelEntry* e, int64_t tiles, int64_t nsteps) {
  int64_t ks = (256 + tiles / 2) / tiles;
  ks = std::min<int64_t>(std::min<int64_t>(ks, kMaxSplit), nsteps / 4);
  while (ks > 1 && tiles * ks * e->bm * e->bn > kWsFloats) --ks;
  return std::max<int64_t>(ks, 1);
}

int64_t tiles_of(const dg::KernelEntry* e, int64_t M, int64_t N) {
  return ((M + e->bm - 1) / e->bm) * ((N + e->bn - 1) / e->bn);
}

// Estimated microseconds of one launch of e on M x N x K (whole K per
// workgroup). Every class is held back by how fast one CU pulls its tile's
// operand rows from L2 (the workgroups of one CU share that rate) or by its
// arithmetic, so a launch takes the entry's fixed cost plus, per round of
// one tile per CU, a fixed cost and the larger of moving bm + bn rows of K
// bytes and 2 bm bn K FLOP at the entry's per-CU rates. The constants were
// fitted by least squares in log time to graph-timed launches of every
// entry on 166 shapes (M 32 to 4096, N 1024 to 28672, K 2048 to 8192,
// g 64 and 128); the least estimate picked an entry within 3% of the
// fastest on every one of them.
double estimate_us(const dg::KernelEntry* e, int64_t M, int64_t N, int64_t K) {
  const int64_t rounds = (tiles_of(e, M, N) + 255) / 256;
  const double bytes = (double)(e->bm + e->bn) * (double)K;
  const double flop = 2.0 * e->bm * e->bn * (double)K;
  return e->launch_us +
         (double)rounds * (e->round_us + std::max(bytes / (e->cu_gbps * 1e3), flop / (e->cu_tflops * 1e6)));
}

Plan plan(int64_t M, int64_t N, int64_t K, int sgran, bool split_ok, int64_t split_steps = kSplitMinSteps) {
  Plan p{nullptr, 1, 0};
  const int gran = kernel_gran(sgran);
  const int64_t nsteps = (K + 127) / 128;
  auto split_k = [&]() {
    p.e = find(dg::kClassSplitK, gran);
    p.tiles = tiles_of(p.e, M, N);
    p.ksplit = split_ok ? (int)splits_for(p.e, p.tiles, nsteps) : 1;
    return p;
  };
  const int force = forced_tile();
  if (force >= 0) {
    for (int i = 0; i < dg::kTableSize; ++i)
      if (dg::kTable[i].id == force && dg::kTable[i].gran == gran) p.e = &dg::kTable[i];
    if (p.e) {
      p.tiles = tiles_of(p.e, M, N);
      if (p.e->cls == dg::kClassSplitK && split_ok) p.ksplit = (int)splits_for(p.e, p.tiles, nsteps);
      return p;
    }
  }
  if (split_ok && nsteps >= split_steps && split_k().ksplit >= kSplitMin) return p;
  // The entry with the least estimated time: small tiles where there are few
  // of them (fewer bytes per CU, more CUs busy), large ones where the
  // arithmetic dominates.
  p = Plan{nullptr, 1, 0};
  double best = 0.0;
  for (int i = 0; i < dg::kTableSize; ++i) {
    const dg::KernelEntry* e = &dg::kTable[i];
    if (e->gran != gran) continue;
    const double t = estimate_us(e, M, N, K);
    if (!p.e || t < best) {
      best = t;
      p.e = e;
    }
  }
  p.tiles = tiles_of(p.e, M, N);
  p.ksplit = 1;
  return p;
}

// Whether a plan has an entry and a grid that a launch takes.
bool runs(const Plan& p) { return p.e && p.tiles * p.ksplit <= 0x7fffffff; }

// Workspace bytes of a plan: none without a K split.
int64_t workspace_bytes(const Plan& p) {
  if (p.ksplit <= 1) return 0;
  return p.tiles * p.ksplit * p.e->bm * p.e->bn * (int64_t)sizeof(float);
}

}  // namespace

namespace dg {

thread_local hipError_t t_last_hip = hipSuccess;

bool log_enabled() {
  static const bool on = [] {
    const char* e = std::getenv("DG_LOG");
    return e && e[0] == '1';
  }();
  return on;
}

int forced_tile() {
  const char* e = std::getenv("DG_FORCE_TILE");
  return e ? std::atoi(e) : -1;
}

// One-time per-device check; returns DG_OK, DG_EUNSUPPORTED or DG_ELAUNCH.
int device_ready(int* dev_out) {
  int dev = 0;
  if ((t_last_hip = hipGetDevice(&dev)) != hipSuccess) return DG_ELAUNCH;
  if (dev < 0 || dev >= kMaxDevices) return DG_EUNSUPPORTED;
  std::call_once(g_dev_once[dev], check_device, dev);
  if (dev_out) *dev_out = dev;
  return g_dev_status[dev];
}

}  // namespace dg

namespace {

// Layout check shared by the GEMM and the tile query: a known code. A
// transposed operand's stored rows (M bytes for A [K,M], N for B [K,N]) may
// have any length: its tiles are copied in 16-byte pieces along those rows
// whatever their alignment, and the bytes a piece takes past a row's end
// belong to rows of A or B past M or N, whose outputs are never stored.
int validate_layout(int64_t M, int64_t N, int layout) {
  (void)M;
  (void)N;
  if (layout < DG_LAYOUT_NT || layout > DG_LAYOUT_TN) return DG_EINVAL;
  return DG_OK;
}

// The residual epilogue's own arguments (dg_gemm_fp8_residual).
struct Residual {
  const void* res;
  int res_type;
  int64_t ldres;
  void* pre;
};

// split_ok: few-tile long-K shapes may split K over workgroups, through ws (the
// caller's, ws_bytes long; none when ws_bytes is 0) or, with use_scratch,
// through the library's static scratch array. rs: the residual epilogue (null:
// none), which takes every activation.
int gemm(const void* a, const void* b, const float* sa, const float* sb, void* out, int64_t M, int64_t N, int64_t K,
         int gran, int layout, int sa_rows, int fmt_a, int fmt_b, const float* bias, int act, void* stream,
         bool split_ok = false, void* ws = nullptr, int64_t ws_bytes = 0, bool use_scratch = false,
         const Residual* rs = nullptr) {
  if (!a || !b || !sa || !sb || !out) return DG_EINVAL;
  if (sa_rows != gran && sa_rows != 1) return DG_EINVAL;
  if (validate_layout(M, N, layout) != DG_OK) return DG_EINVAL;
  if ((fmt_a != DG_FMT_E4M3 && fmt_a != DG_FMT_E5M2) || (fmt_b != DG_FMT_E4M3 && fmt_b != DG_FMT_E5M2))
    return DG_EINVAL;
  if (act < DG_ACT_NONE || act > (rs ? DG_ACT_GELU_TANH : DG_ACT_GELU)) return DG_EINVAL;
  if (rs && rs->res && (!known_kind(rs->res_type) || !good_pitch(rs->ldres, N))) return DG_EINVAL;
  if ((uintptr_t)bias & 3) return DG_EALIGN;
  if (rs && (((uintptr_t)rs->pre & 1) || (rs->res && ((uintptr_t)rs->res & (kind_size(rs->res_type) - 1)))))
    return DG_EALIGN;
  if (ws_bytes < 0 || (ws_bytes > 0 && !ws) || (ws && ws_bytes == 0)) return DG_EINVAL;
  if ((uintptr_t)ws & 255) return DG_EALIGN;
  int rc = validate(M, N, K, gran);
  if (rc != DG_OK) return rc;
  if (((uintptr_t)a & 15) || ((uintptr_t)b & 15) || ((uintptr_t)sa & 3) || ((uintptr_t)sb & 3) ||
      ((uintptr_t)out & 1))
    return DG_EALIGN;
  // The residual epilogue's form; with nothing that the plain forms lack they
  // run, by their own plan (the same sums and roundings: the same bits).
  const bool form3 = rs && (rs->res || rs->pre || act > DG_ACT_GELU);
  // A workspace lets few-tile long-K shapes split K; without one nothing does.
  Plan pl = plan(M, N, K, gran, split_ok && (ws_bytes > 0 || use_scratch),
                 form3 ? residual_split_steps(layout) : kSplitMinSteps);
  if (!runs(pl)) return DG_EINVAL;
  const int64_t need = workspace_bytes(pl);
  if (ws_bytes > 0 && ws_bytes < need) return DG_EINVAL;
  if (use_scratch && need > kScratchBytes) return DG_ESCRATCH;
  {
    // out is written while the inputs are read: it may overlap none of them
    // (the inputs may overlap each other), nor the workspace. Sizes are the
    // logical ones, which every layout stores in the same number of bytes.
    const uint64_t nks = (uint64_t)(K / gran);
    const uint64_t sa_rows_n = sa_rows == 1 ? (uint64_t)M : (uint64_t)((M + gran - 1) / gran);
    const uint64_t ob = 2ull * (uint64_t)M * (uint64_t)N;
    const uint64_t ab = (uint64_t)M * (uint64_t)K, bb = (uint64_t)N * (uint64_t)K;
    const uint64_t sab = 4ull * sa_rows_n * nks, sbb = 4ull * (uint64_t)((N + gran - 1) / gran) * nks;
    const uint64_t biasb = bias ? 4ull * (uint64_t)N : 0, wsb = (uint64_t)ws_bytes;
    if (overlaps(out, ob, a, ab) || overlaps(out, ob, b, bb) || overlaps(out, ob, sa, sab) ||
        overlaps(out, ob, sb, sbb) || overlaps(out, ob, bias, biasb))
      return DG_EINVAL;
    if (overlaps(ws, wsb, a, ab) || overlaps(ws, wsb, b, bb) || overlaps(ws, wsb, sa, sab) ||
        overlaps(ws, wsb, sb, sbb) || overlaps(ws, wsb, bias, biasb) || overlaps(ws, wsb, out, ob))
      return DG_EINVAL;
    if (rs) {
      // pre is an output like out. The residual may be out itself (BF16,
      // pitch N): every element is read by the thread that then writes it.
      const uint64_t rb = rs->res ? extent(M, N, rs->ldres, kind_size(rs->res_type)) : 0, pb = rs->pre ? ob : 0;
      const bool in_place = rs->res == out && rs->res_type == DG_IN_BF16 && rs->ldres == N;
      if (!in_place && overlaps(out, ob, rs->res, rb)) return DG_EINVAL;
      if (overlaps(rs->pre, pb, out, ob) || overlaps(rs->pre, pb, rs->res, rb) || overlaps(rs->pre, pb, a, ab) ||
          overlaps(rs->pre, pb, b, bb) || overlaps(rs->pre, pb, sa, sab) || overlaps(rs->pre, pb, sb, sbb) ||
          overlaps(rs->pre, pb, bias, biasb) || overlaps(rs->pre, pb, ws, wsb) || overlaps(ws, wsb, rs->res, rb))
        return DG_EINVAL;
    }
  }

  int dev = 0;
  rc = device_ready(&dev);
  if (rc != DG_OK) return rc;
  const dg::KernelEntry* e = pl.e;
  if (use_scratch && pl.ksplit > 1) {
    std::call_once(g_scratch_once[dev], find_scratch, dev);
    if (!g_scratch[dev]) {
      t_last_hip = g_scratch_err[dev];
      return DG_ELAUNCH;
    }
    ws = g_scratch[dev];
  }

  dg::GemmArgs p;
  p.a = static_cast<const uint8_t*>(a);
  p.b = static_cast<const uint8_t*>(b);
  p.sa = sa;
  p.sb = sb;
  p.out = static_cast<uint16_t*>(out);
  p.M = M;
  p.N = N;
  p.K = K;
  p.gran = kernel_gran(gran);
  p.sshift = gran == 256 ? 1 : 0;
  p.fmt = (fmt_a == DG_FMT_E5M2 ? 1 : 0) | (fmt_b == DG_FMT_E5M2 ? 2 : 0);
  p.rowa = sa_rows == 1 ? 1 : 0;
  p.layout = layout;
  p.vec_store = (((uintptr_t)out & 15) == 0 && N % 8 == 0) ? 1 : 0;
  p.ksplit = pl.ksplit;
  p.ws = pl.ksplit > 1 ? static_cast<float*>(ws) : nullptr;
  p.bias = bias;
  p.act = act;
  p.epi = {};
  if (form3) {
    p.epi.bias = bias;
    p.epi.res = rs->res;
    p.epi.out = static_cast<uint16_t*>(out);
    p.epi.pre = static_cast<uint16_t*>(rs->pre);
    p.epi.ldres = rs->ldres;
    p.epi.res_kind = rs->res ? rs->res_type : dg::kAbsent;
    p.epi.act = act;
  }
  if (log_enabled())
    std::fprintf(stderr,
                 "dg_gemm_fp8 M=%lld N=%lld K=%lld g=%d layout=%d sa_rows=%d fmt=%d,%d bias=%d act=%d -> kernel %d "
                 "(%dx%d, %d stages, %d waves) ksplit %d grid %lld workspace %lld\n",
                 (long long)M, (long long)N, (long long)K, gran, layout, sa_rows, fmt_a, fmt_b, bias ? 1 : 0, act, e->id,
                 e->bm, e->bn, e->stages, e->waves, pl.ksplit, (long long)(pl.tiles * pl.ksplit), (long long)need);
  // the streaming entries take every layout themselves
  t_last_hip = form3 ? dg::launch_residual(e->id, p, static_cast<hipStream_t>(stream))
               : layout == DG_LAYOUT_NT || e->cls == dg::kClassStream
                   ? e->launch(p, static_cast<hipStream_t>(stream))
                   : dg::launch_layout(e->id, p, static_cast<hipStream_t>(stream));
  return t_last_hip == hipSuccess ? DG_OK : DG_ELAUNCH;
}

// block_rows: rows per block, gran (g x g blocks) or 1 (1 x g blocks); in:
// DG_IN_F32, DG_IN_BF16 or DG_IN_F16.
int quantize(const void* x, int in, int64_t rows, int64_t cols, int gran, int block_rows, int fmt, void* q,
             float* scales, void* stream) {
  if (!x || !q || !scales) return DG_EINVAL;
  if (fmt != DG_FMT_E4M3 && fmt != DG_FMT_E5M2) return DG_EINVAL;
  if (in != DG_IN_F32 && in != DG_IN_BF16 && in != DG_IN_F16) return DG_EINVAL;
  const uint64_t esize = in == DG_IN_F32 ? 4 : 2;
  if (rows <= 0 || cols <= 0 || rows > DG_MAX_DIM || cols > DG_MAX_DIM) return DG_EINVAL;
  if ((gran != 64 && gran != 128 && gran != 256) || cols % gran != 0) return DG_EINVAL;
  if (block_rows != gran && block_rows != 1) return DG_EINVAL;
  if (((rows + block_rows - 1) / block_rows) * (cols / gran) > 0x7fffffff) return DG_EINVAL;
  // a lane writes one code per element of its 16-byte load: 4 bytes, or 8 for 16-bit input
  if (((uintptr_t)x & 15) || ((uintptr_t)q & (16 / esize - 1)) || ((uintptr_t)scales & 3)) return DG_EALIGN;
  {
    const uint64_t xb = esize * (uint64_t)rows * (uint64_t)cols, qb = (uint64_t)rows * (uint64_t)cols;
    const uint64_t sbytes = 4ull * (uint64_t)((rows + block_rows - 1) / block_rows) * (uint64_t)(cols / gran);
    if (overlaps(x, xb, q, qb) || overlaps(x, xb, scales, sbytes) || overlaps(q, qb, scales, sbytes)) return DG_EINVAL;
  }
  const int rc = device_ready();
  if (rc != DG_OK) return rc;
  dg::QuantArgs p;
  p.x = x;
  p.q = static_cast<uint8_t*>(q);
  p.scales = scales;
  p.rows = rows;
  p.cols = cols;
  p.gran = gran;
  p.fmt = fmt;
  p.in = in;
  if (log_enabled())
    std::fprintf(stderr, "dg_quantize_fp8 rows=%lld cols=%lld block %dx%d fmt=%d in=%d\n", (long long)rows,
                 (long long)cols, block_rows, gran, fmt, in);
  t_last_hip = block_rows == 1 ? dg::launch_quant_rows(p, static_cast<hipStream_t>(stream))
                               : dg::launch_quant(p, static_cast<hipStream_t>(stream));
  return t_last_hip == hipSuccess ? DG_OK : DG_ELAUNCH;
}

// The gradient's g x g blocks: a workgroup of up to 1024 threads each (256 at g = 64) in a grid of less than 2^32 threads.
bool good_blocks(int64_t rows, int64_t cols, int gran, int block_rows) {
  return block_rows == 1 || ((rows + gran - 1) / gran) * (cols / gran) <= (gran == 64 ? 0xffffff : 0x3fffff);
}

int rmsnorm_quantize(const void* x, int x_type, int64_t ldx, const void* res, int res_type, int64_t ldres,
                     const float* w, float eps, int64_t rows, int64_t cols, int gran, int fmt, void* h, void* y,
                     float* rstd, void* q, float* scales, void* stream) {
  if (!x || !w || !q || !scales || (!res != !h)) return DG_EINVAL;
  if (!known_kind(x_type) || (res && !known_kind(res_type))) return DG_EINVAL;
  if (fmt != DG_FMT_E4M3 && fmt != DG_FMT_E5M2) return DG_EINVAL;
  if (!good_dims(rows, cols) || !good_gran(gran, cols) || !good_pitch(ldx, cols) || (res && !good_pitch(ldres, cols)))
    return DG_EINVAL;
  if (!(eps >= 0.0f) || eps > 1e30f) return DG_EINVAL;
  const uint64_t xs = kind_size(x_type), rs = res ? kind_size(res_type) : 0;
  if (misaligned_rows(x, ldx, xs) || misaligned_rows(res, ldres, rs) || misaligned(w, 16) || misaligned(h, 16) ||
      misaligned(y, 16) || misaligned(q, 8) || misaligned(rstd, 4) || misaligned(scales, 4))
    return DG_EALIGN;
  {
    const uint64_t n = (uint64_t)rows * (uint64_t)cols;
    const Range outs[] = {{h, n * rs}, {y, n * xs}, {rstd, 4ull * rows}, {q, n}, {scales, 4ull * rows * (cols / gran)}};
    const Range ins[] = {{x, extent(rows, cols, ldx, xs)}, {res, res ? extent(rows, cols, ldres, rs) : 0}, {w, 4ull * cols}};
    const bool in_place = h && h == res && ldres == cols;  // a row is read whole before it is written
    if (clash(outs, ins, in_place ? 0 : -1, 1)) return DG_EINVAL;
  }
  const int rc = device_ready();
  if (rc != DG_OK) return rc;
  dg::NormArgs p;
  p.x = x;
  p.res = res;
  p.w = w;
  p.h = h;
  p.y = y;
  p.rstd = rstd;
  p.q = static_cast<uint8_t*>(q);
  p.scales = scales;
  p.rows = rows;
  p.cols = cols;
  p.ldx = ldx;
  p.ldres = ldres;
  p.eps = eps;
  p.gran = gran;
  p.fmt = fmt;
  p.xk = x_type;
  p.rk = res ? res_type : dg::kAbsent;
  p.gshift = gran == 64 ? 6 : gran == 128 ? 7 : 8;
  p.segs = (int)(cols / gran);
  if (log_enabled())
    std::fprintf(stderr, "dg_rmsnorm_quantize_fp8 rows=%lld cols=%lld g=%d fmt=%d x=%d res=%d y=%d\n", (long long)rows,
                 (long long)cols, gran, fmt, x_type, p.rk, y ? 1 : 0);
  t_last_hip = dg::launch_norm(p, static_cast<hipStream_t>(stream));
  return t_last_hip == hipSuccess ? DG_OK : DG_ELAUNCH;
}

int rmsnorm_backward(const void* dy, int dy_type, int64_t lddy, const void* h, int h_type, int64_t ldh,
                     const float* rstd, const float* w, const void* dh, int64_t lddh, int64_t rows, int64_t cols,
                     void* dx, float* dw, void* ws, int64_t ws_bytes, void* stream) {
  if (!dy || !h || !rstd || !w || !dx || !dw) return DG_EINVAL;
  if (!known_kind(dy_type) || !known_kind(h_type)) return DG_EINVAL;
  if (!good_dims(rows, cols) || cols % 64 != 0) return DG_EINVAL;
  if (!good_pitch(lddy, cols) || !good_pitch(ldh, cols) || (dh && !good_pitch(lddh, cols))) return DG_EINVAL;
  const int64_t need = dg::norm_bwd_workspace(rows, cols);
  if (ws_bytes < need || (need > 0 && !ws)) return DG_EINVAL;
  const uint64_t ds = kind_size(dy_type), hs = kind_size(h_type);
  if (misaligned_rows(dy, lddy, ds) || misaligned_rows(h, ldh, hs) || misaligned_rows(dh, lddh, hs) ||
      misaligned(w, 16) || misaligned(dx, 16) || misaligned(dw, 4) || misaligned(rstd, 4) || misaligned(ws, 16))
    return DG_EALIGN;
  {
    const Range outs[] = {{dx, hs * rows * cols}, {dw, 4ull * cols}, {need ? ws : nullptr, (uint64_t)need}};
    const Range ins[] = {{dh, dh ? extent(rows, cols, lddh, hs) : 0},
                         {dy, extent(rows, cols, lddy, ds)},
                         {h, extent(rows, cols, ldh, hs)},
                         {rstd, 4ull * rows},
                         {w, 4ull * cols}};
    const bool in_place = dh == dx && lddh == cols;
    if (clash(outs, ins, in_place ? 0 : -1, 0)) return DG_EINVAL;
  }
  const int rc = device_ready();
  if (rc != DG_OK) return rc;
  dg::NormBwdArgs p;
  p.dy = dy;
  p.h = h;
  p.rstd = rstd;
  p.w = w;
  p.dh = dh;
  p.dx = dx;
  p.dw = dw;
  p.ws = static_cast<float*>(ws);
  p.rows = rows;
  p.cols = cols;
  p.lddy = lddy;
  p.ldh = ldh;
  p.lddh = lddh;
  p.dk = dy_type;
  p.hk = h_type;
  p.row0 = 0;
  if (log_enabled())
    std::fprintf(stderr, "dg_rmsnorm_backward rows=%lld cols=%lld dy=%d h=%d dh=%d workspace %lld\n", (long long)rows,
                 (long long)cols, dy_type, h_type, dh ? 1 : 0, (long long)need);
  t_last_hip = dg::launch_norm_bwd(p, static_cast<hipStream_t>(stream));
  return t_last_hip == hipSuccess ? DG_OK : DG_ELAUNCH;
}

int epilogue_backward(const void* dout, int dout_type, int64_t lddout, const void* pre, int64_t ldpre, int act,
                      int64_t rows, int64_t cols, int gran, int block_rows, int fmt, void* dz, float* dbias, void* q,
                      float* scales, void* ws, int64_t ws_bytes, void* stream) {
  if (!dout || !q || !scales) return DG_EINVAL;
  if (!known_kind(dout_type)) return DG_EINVAL;
  if (act < DG_ACT_NONE || act > DG_ACT_GELU_TANH || (act != DG_ACT_NONE) != (pre != nullptr)) return DG_EINVAL;
  if (fmt != DG_FMT_E4M3 && fmt != DG_FMT_E5M2) return DG_EINVAL;
  if (!good_dims(rows, cols) || !good_gran(gran, cols) || (block_rows != gran && block_rows != 1)) return DG_EINVAL;
  if (!good_pitch(lddout, cols) || (pre && !good_pitch(ldpre, cols))) return DG_EINVAL;
  if (!good_blocks(rows, cols, gran, block_rows)) return DG_EINVAL;
  const int64_t need = dbias ? dg::epi_bwd_workspace(rows, cols, gran, block_rows) : 0;
  if (ws_bytes < need || (need > 0 && !ws)) return DG_EINVAL;
  const uint64_t ds = kind_size(dout_type);
  if (misaligned_rows(dout, lddout, ds) || misaligned_rows(pre, ldpre, 2) || misaligned(dz, 16) || misaligned(q, 8) ||
      misaligned(dbias, 4) || misaligned(scales, 4) || misaligned(ws, 16))
    return DG_EALIGN;
  {
    const uint64_t n = (uint64_t)rows * (uint64_t)cols;
    const Range outs[] = {{dz, n * ds},
                          {dbias, 4ull * cols},
                          {q, n},
                          {scales, 4ull * ((rows + block_rows - 1) / block_rows) * (cols / gran)},
                          {need ? ws : nullptr, (uint64_t)need}};
    const Range ins[] = {{dout, extent(rows, cols, lddout, ds)}, {pre, pre ? extent(rows, cols, ldpre, 2) : 0}};
    const bool in_place = dz && dz == dout && lddout == cols;
    if (clash(outs, ins, in_place ? 0 : -1, 0)) return DG_EINVAL;
  }
  const int rc = device_ready();
  if (rc != DG_OK) return rc;
  dg::EpiBwdArgs p;
  p.dout = dout;
  p.pre = static_cast<const uint16_t*>(pre);
  p.dz = dz;
  p.dbias = dbias;
  p.q = static_cast<uint8_t*>(q);
  p.scales = scales;
  p.ws = static_cast<float*>(ws);
  p.rows = rows;
  p.cols = cols;
  p.lddout = lddout;
  p.ldpre = ldpre;
  p.gran = gran;
  p.block_rows = block_rows;
  p.fmt = fmt;
  p.dk = dout_type;
  p.act = act;
  if (log_enabled())
    std::fprintf(stderr, "dg_epilogue_backward_fp8 rows=%lld cols=%lld block %dx%d fmt=%d act=%d dout=%d workspace %lld\n",
                 (long long)rows, (long long)cols, block_rows, gran, fmt, act, dout_type, (long long)need);
  t_last_hip = dg::launch_epi_bwd(p, static_cast<hipStream_t>(stream));
  return t_last_hip == hipSuccess ? DG_OK : DG_ELAUNCH;
}

}  // namespace

extern "C" {

int dg_version(void) { return DG_VERSION; }

const char* dg_strerror(int code) {
  switch (code) {
    case DG_OK: return "success";
    case DG_EINVAL:
      return "invalid argument (null pointer, bad dimension, K not a multiple of gran, gran not 64/128/256, "
             "sa_rows neither gran nor 1, a format code other than DG_FMT_E4M3/DG_FMT_E5M2, an unknown "
             "activation, layout or element type, a row pitch shorter than its row, an "
             "output or workspace that overlaps another argument, or a workspace smaller than the plan needs)";
    case DG_EALIGN:
      return "misaligned pointer or row pitch (a, b need 16 bytes; sa, sb, bias 4 bytes; out 2 bytes; workspace 256 "
             "bytes; the norm's and the gradients' matrices and row pitches 16 bytes)";
    case DG_EUNSUPPORTED: return "unsupported device (gfx950 required)";
    case DG_ESCRATCH:
      return "the call's K split needs more workspace than dg_gemm_fp8_noalloc's fixed scratch "
             "(dg_noalloc_scratch_bytes()); use dg_gemm_fp8_ws with a workspace of dg_query_tile_ws's size";
    case DG_ELAUNCH:
      std::snprintf(t_msg, sizeof t_msg, "HIP error %d: %s", (int)t_last_hip, hipGetErrorString(t_last_hip));
      return t_msg;
    default: return "unknown status";
  }
}

}  // extern "C"

namespace {

int query(int64_t M, int64_t N, int64_t K, int gran, int layout, bool split_ok, dg_tile_info* info) {
  if (!info) return DG_EINVAL;
  int rc = validate(M, N, K, gran);
  if (rc != DG_OK) return rc;
  if ((rc = validate_layout(M, N, layout)) != DG_OK) return rc;
  const Plan p = plan(M, N, K, gran, split_ok);
  if (!runs(p)) return DG_EINVAL;
  info->kernel_id = p.e->id;
  info->bm = p.e->bm;
  info->bn = p.e->bn;
  info->bk = 128;
  info->stages = p.e->stages;
  info->waves = p.e->waves;
  info->ksplit = p.ksplit;
  info->grid = p.tiles * p.ksplit;
  info->workspace_bytes = workspace_bytes(p);
  return DG_OK;
}

}  // namespace

extern "C" {

int dg_query_tile_layout(int64_t M, int64_t N, int64_t K, int gran, int layout, dg_tile_info* info) {
  return query(M, N, K, gran, layout, false, info);
}

int dg_query_tile_ws(int64_t M, int64_t N, int64_t K, int gran, int layout, dg_tile_info* info) {
  return query(M, N, K, gran, layout, true, info);
}

int dg_gemm_fp8_noalloc(const void* a, const void* b, const float* sa, const float* sb, void* out, int64_t M,
                        int64_t N, int64_t K, int gran, int layout, int sa_rows, int fmt_a, int fmt_b,
                        const float* bias, int act, void* stream) {
  return gemm(a, b, sa, sb, out, M, N, K, gran, layout, sa_rows, fmt_a, fmt_b, bias, act, stream, true, nullptr, 0,
              true);
}

int64_t dg_noalloc_scratch_bytes(void) { return kScratchBytes; }

int dg_query_tile(int64_t M, int64_t N, int64_t K, int gran, dg_tile_info* info) {
  return dg_query_tile_layout(M, N, K, gran, DG_LAYOUT_NT, info);
}

int dg_gemm_fp8_ws(const void* a, const void* b, const float* sa, const float* sb, void* out, int64_t M, int64_t N,
                   int64_t K, int gran, int layout, int sa_rows, int fmt_a, int fmt_b, const float* bias, int act,
                   void* workspace, int64_t workspace_bytes, void* stream) {
  return gemm(a, b, sa, sb, out, M, N, K, gran, layout, sa_rows, fmt_a, fmt_b, bias, act, stream, true, workspace,
              workspace_bytes);
}

int dg_gemm_fp8_nt(const void* a, const void* b, const float* sa, const float* sb, void* out, int64_t M,
                   int64_t N, int64_t K, int gran, void* stream) {
  return gemm(a, b, sa, sb, out, M, N, K, gran, DG_LAYOUT_NT, gran, DG_FMT_E4M3, DG_FMT_E4M3, nullptr, DG_ACT_NONE,
              stream);
}

int dg_gemm_fp8_nt_fmt(const void* a, const void* b, const float* sa, const float* sb, void* out, int64_t M,
                       int64_t N, int64_t K, int gran, int fmt_a, int fmt_b, void* stream) {
  return gemm(a, b, sa, sb, out, M, N, K, gran, DG_LAYOUT_NT, gran, fmt_a, fmt_b, nullptr, DG_ACT_NONE, stream);
}

int dg_gemm_fp8_nt_epi(const void* a, const void* b, const float* sa, const float* sb, void* out, int64_t M,
                       int64_t N, int64_t K, int gran, int fmt_a, int fmt_b, const float* bias, int act,
                       void* stream) {
  return gemm(a, b, sa, sb, out, M, N, K, gran, DG_LAYOUT_NT, gran, fmt_a, fmt_b, bias, act, stream);
}

int dg_gemm_fp8_nt_ex(const void* a, const void* b, const float* sa, const float* sb, void* out, int64_t M,
                      int64_t N, int64_t K, int gran, int sa_rows, int fmt_a, int fmt_b, const float* bias, int act,
                      void* stream) {
  return gemm(a, b, sa, sb, out, M, N, K, gran, DG_LAYOUT_NT, sa_rows, fmt_a, fmt_b, bias, act, stream);
}

int dg_gemm_fp8_layout(const void* a, const void* b, const float* sa, const float* sb, void* out, int64_t M,
                       int64_t N, int64_t K, int gran, int layout, int fmt_a, int fmt_b, const float* bias, int act,
                       void* stream) {
  return gemm(a, b, sa, sb, out, M, N, K, gran, layout, gran, fmt_a, fmt_b, bias, act, stream);
}

int dg_quantize_fp8_blocks(const float* x, int64_t rows, int64_t cols, int gran, int fmt, void* q, float* scales,
                           void* stream) {
  return quantize(x, DG_IN_F32, rows, cols, gran, gran, fmt, q, scales, stream);
}

int dg_quantize_fp8_rows(const float* x, int64_t rows, int64_t cols, int gran, int fmt, void* q, float* scales,
                         void* stream) {
  return quantize(x, DG_IN_F32, rows, cols, gran, 1, fmt, q, scales, stream);
}

int dg_quantize_e4m3_blocks(const float* x, int64_t rows, int64_t cols, int gran, void* q, float* scales,
                            void* stream) {
  return quantize(x, DG_IN_F32, rows, cols, gran, gran, DG_FMT_E4M3, q, scales, stream);
}

int dg_quantize_fp8_blocks_typed(const void* x, int in_type, int64_t rows, int64_t cols, int gran, int fmt, void* q,
                                 float* scales, void* stream) {
  return quantize(x, in_type, rows, cols, gran, gran, fmt, q, scales, stream);
}

int dg_quantize_fp8_rows_typed(const void* x, int in_type, int64_t rows, int64_t cols, int gran, int fmt, void* q,
                               float* scales, void* stream) {
  return quantize(x, in_type, rows, cols, gran, 1, fmt, q, scales, stream);
}

int dg_gemm_fp8_residual(const void* a, const void* b, const float* sa, const float* sb, void* out, int64_t M,
                         int64_t N, int64_t K, int gran, int layout, int sa_rows, int fmt_a, int fmt_b,
                         const float* bias, int act, const void* res, int res_type, int64_t ldres, void* pre,
                         void* workspace, int64_t workspace_bytes, void* stream) {
  const Residual rs{res, res_type, ldres, pre};
  return gemm(a, b, sa, sb, out, M, N, K, gran, layout, sa_rows, fmt_a, fmt_b, bias, act, stream, true, workspace,
              workspace_bytes, false, &rs);
}

int64_t dg_gemm_fp8_residual_workspace(int64_t M, int64_t N, int64_t K, int gran, int layout) {
  if (validate(M, N, K, gran) != DG_OK || validate_layout(M, N, layout) != DG_OK) return DG_EINVAL;
  const Plan p = plan(M, N, K, gran, true, residual_split_steps(layout));
  return runs(p) ? workspace_bytes(p) : (int64_t)DG_EINVAL;
}

int dg_rmsnorm_quantize_fp8(const void* x, int x_type, int64_t ldx, const void* res, int res_type, int64_t ldres,
                            const float* w, float eps, int64_t rows, int64_t cols, int gran, int fmt, void* h, void* y,
                            float* rstd, void* q, float* scales, void* stream) {
  return rmsnorm_quantize(x, x_type, ldx, res, res_type, ldres, w, eps, rows, cols, gran, fmt, h, y, rstd, q, scales,
                          stream);
}

int64_t dg_rmsnorm_backward_workspace(int64_t rows, int64_t cols) {
  return good_dims(rows, cols) && cols % 64 == 0 ? dg::norm_bwd_workspace(rows, cols) : (int64_t)DG_EINVAL;
}

int dg_rmsnorm_backward(const void* dy, int dy_type, int64_t lddy, const void* h, int h_type, int64_t ldh,
                        const float* rstd, const float* w, const void* dh, int64_t lddh, int64_t rows, int64_t cols,
                        void* dx, float* dw, void* workspace, int64_t workspace_bytes, void* stream) {
  return rmsnorm_backward(dy, dy_type, lddy, h, h_type, ldh, rstd, w, dh, lddh, rows, cols, dx, dw, workspace,
                          workspace_bytes, stream);
}

int64_t dg_epilogue_backward_workspace(int64_t rows, int64_t cols, int gran, int block_rows) {
  return good_dims(rows, cols) && good_gran(gran, cols) && (block_rows == gran || block_rows == 1) &&
                 good_blocks(rows, cols, gran, block_rows)
             ? dg::epi_bwd_workspace(rows, cols, gran, block_rows)
             : (int64_t)DG_EINVAL;
}

int dg_epilogue_backward_fp8(const void* dout, int dout_type, int64_t lddout, const void* pre, int64_t ldpre, int act,
                             int64_t rows, int64_t cols, int gran, int block_rows, int fmt, void* dz, float* dbias,
                             void* q, float* scales, void* workspace, int64_t workspace_bytes, void* stream) {
  return epilogue_backward(dout, dout_type, lddout, pre, ldpre, act, rows, cols, gran, block_rows, fmt, dz, dbias, q,
                           scales, workspace, workspace_bytes, stream);
}

}  // extern "C"

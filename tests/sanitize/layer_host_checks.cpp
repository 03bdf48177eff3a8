// The calls around the product (norm, residual product, their gradients and
// workspace queries) under AddressSanitizer and UndefinedBehaviorSanitizer, as
// host_checks.cpp does it for the others: every call carries one argument
// error, so each returns before its first HIP call. Exit status 0 when every
// call returns what the header promises.

#include <cmath>
#include <cstddef>
#include <cstdint>
#include <cstdio>
#include <initializer_list>
#include <limits>

#include "dg.h"

// The sources are compiled without their device code: nothing to register.
extern "C" {
long layer_checks_no_device_code[8];
void** __hipRegisterFatBinary(const void*) { return reinterpret_cast<void**>(layer_checks_no_device_code); }
void __hipUnregisterFatBinary(void**) {}
void __hipRegisterFunction(void**, const void*, char*, const char*, unsigned, void*, void*, void*, void*, int*) {}
void __hipRegisterVar(void**, void*, char*, char*, int, size_t, int, int) {}
}

namespace {

int g_failures = 0;

void expect(int64_t got, int64_t want, const char* what, long long a = 0, long long b = 0) {
  if (got != want) {
    ++g_failures;
    std::fprintf(stderr, "FAILED: %s (%lld, %lld): got %lld, want %lld\n", what, a, b, (long long)got, (long long)want);
  }
}

void* addr(int i) { return reinterpret_cast<void*>((uintptr_t)(i + 1) << 52); }
float* faddr(int i) { return static_cast<float*>(addr(i)); }
template <class T>
T* shift(T* p, uintptr_t by) {
  return reinterpret_cast<T*>(reinterpret_cast<uintptr_t>(p) + by);
}

struct Norm {
  const void* x = addr(0);
  int xk = DG_IN_BF16;
  int64_t ldx = 256;
  const void* res = addr(1);
  int rk = DG_IN_F32;
  int64_t ldres = 256;
  const float* w = faddr(2);
  float eps = 1e-6f;
  int64_t rows = 8, cols = 256;
  int gran = 128, fmt = DG_FMT_E4M3;
  void *h = addr(3), *y = addr(4);
  float* rstd = faddr(5);
  void* q = addr(6);
  float* s = faddr(7);
  int operator()() const {
    return dg_rmsnorm_quantize_fp8(x, xk, ldx, res, rk, ldres, w, eps, rows, cols, gran, fmt, h, y, rstd, q, s, nullptr);
  }
};

struct NormBwd {
  const void* dy = addr(0);
  int dk = DG_IN_BF16;
  int64_t lddy = 256;
  const void* h = addr(1);
  int hk = DG_IN_F32;
  int64_t ldh = 256;
  const float *rstd = faddr(2), *w = faddr(3);
  const void* dh = addr(4);
  int64_t lddh = 256, rows = 64, cols = 256;
  void* dx = addr(5);
  float* dw = faddr(6);
  void* ws = addr(7);
  int64_t nb = (int64_t)1 << 40;
  int operator()() const {
    return dg_rmsnorm_backward(dy, dk, lddy, h, hk, ldh, rstd, w, dh, lddh, rows, cols, dx, dw, ws, nb, nullptr);
  }
};

struct Epi {
  const void* dout = addr(0);
  int dk = DG_IN_BF16;
  int64_t lddout = 256;
  const void* pre = addr(1);
  int64_t ldpre = 256;
  int act = DG_ACT_GELU;
  int64_t rows = 300, cols = 256;
  int gran = 128, br = 128, fmt = DG_FMT_E5M2;
  void* dz = addr(2);
  float* db = faddr(3);
  void* q = addr(4);
  float* s = faddr(5);
  void* ws = addr(6);
  int64_t nb = (int64_t)1 << 40;
  int operator()() const {
    return dg_epilogue_backward_fp8(dout, dk, lddout, pre, ldpre, act, rows, cols, gran, br, fmt, dz, db, q, s, ws, nb, nullptr);
  }
};

struct Gemm {
  const void *a = addr(0), *b = addr(1);
  const float *sa = faddr(2), *sb = faddr(3);
  void* out = addr(4);
  int64_t M = 256, N = 256, K = 256;
  int gran = 128, layout = 0, sa_rows = 128, fa = 0, fb = 0;
  const float* bias = faddr(5);
  int act = DG_ACT_GELU;
  const void* res = addr(6);
  int rk = DG_IN_BF16;
  int64_t ldres = 256;
  void *pre = addr(7), *ws = nullptr;
  int64_t nb = 0;
  int operator()() const {
    return dg_gemm_fp8_residual(a, b, sa, sb, out, M, N, K, gran, layout, sa_rows, fa, fb, bias, act, res, rk, ldres, pre, ws, nb,
                                nullptr);
  }
};

// `call` with one member changed.
#define REJECT(TYPE, WANT, CHANGE)            \
  do {                                        \
    TYPE c;                                   \
    CHANGE;                                   \
    expect(c(), WANT, #TYPE ": " #CHANGE);    \
  } while (0)

const int64_t kDims[] = {std::numeric_limits<int64_t>::min(), -1, 0, DG_MAX_DIM + 1, (int64_t)1 << 40, std::numeric_limits<int64_t>::max()};

void norm() {
  for (int64_t d : kDims) {
    REJECT(Norm, DG_EINVAL, c.rows = d);
    REJECT(Norm, DG_EINVAL, c.cols = d);
    REJECT(Norm, DG_EINVAL, c.ldx = d);
    REJECT(Norm, DG_EINVAL, c.ldres = d);
  }
  REJECT(Norm, DG_EINVAL, c.x = nullptr);
  REJECT(Norm, DG_EINVAL, c.w = nullptr);
  REJECT(Norm, DG_EINVAL, c.q = nullptr);
  REJECT(Norm, DG_EINVAL, c.s = nullptr);
  REJECT(Norm, DG_EINVAL, c.h = nullptr);
  REJECT(Norm, DG_EINVAL, c.res = nullptr);
  REJECT(Norm, DG_EINVAL, c.xk = 3);
  REJECT(Norm, DG_EINVAL, c.rk = -1);
  REJECT(Norm, DG_EINVAL, c.fmt = 2);
  for (int g : {0, -128, 32, 96, 512, std::numeric_limits<int>::min()}) REJECT(Norm, DG_EINVAL, c.gran = g);
  for (float e : {-1e-6f, std::nanf(""), INFINITY, 1e31f}) REJECT(Norm, DG_EINVAL, c.eps = e);
  REJECT(Norm, DG_EALIGN, c.x = shift(addr(0), 8));
  REJECT(Norm, DG_EALIGN, c.ldx = 257);
  REJECT(Norm, DG_EALIGN, c.w = shift(faddr(2), 4));
  REJECT(Norm, DG_EALIGN, c.q = shift(addr(6), 4));
  REJECT(Norm, DG_EALIGN, c.rstd = shift(faddr(5), 2));
  REJECT(Norm, DG_EINVAL, c.h = addr(0));
  REJECT(Norm, DG_EINVAL, c.y = addr(3));
  REJECT(Norm, DG_EINVAL, (c.h = const_cast<void*>(c.res), c.ldres = 512));
  // the largest sizes and pitches, refused by an overlap alone
  REJECT(Norm, DG_EINVAL, (c.rows = DG_MAX_DIM, c.cols = DG_MAX_DIM, c.ldx = DG_MAX_DIM, c.ldres = DG_MAX_DIM, c.y = addr(6)));
}

void norm_bwd() {
  for (int64_t d : kDims) {
    REJECT(NormBwd, DG_EINVAL, c.rows = d);
    REJECT(NormBwd, DG_EINVAL, c.cols = d);
    REJECT(NormBwd, DG_EINVAL, c.lddy = d);
    REJECT(NormBwd, DG_EINVAL, c.ldh = d);
    REJECT(NormBwd, DG_EINVAL, c.lddh = d);
    expect(dg_rmsnorm_backward_workspace(d, 256), DG_EINVAL, "workspace rows", d);
    expect(dg_rmsnorm_backward_workspace(64, d), DG_EINVAL, "workspace cols", d);
  }
  REJECT(NormBwd, DG_EINVAL, c.dy = nullptr);
  REJECT(NormBwd, DG_EINVAL, c.dw = nullptr);
  REJECT(NormBwd, DG_EINVAL, c.dk = 7);
  REJECT(NormBwd, DG_EINVAL, c.cols = 200);
  REJECT(NormBwd, DG_EINVAL, c.nb = -1);
  REJECT(NormBwd, DG_EINVAL, (c.rows = 5000, c.nb = 64));
  REJECT(NormBwd, DG_EINVAL, (c.rows = 5000, c.ws = nullptr));
  REJECT(NormBwd, DG_EALIGN, c.dx = shift(addr(5), 8));
  REJECT(NormBwd, DG_EALIGN, c.ldh = 258);
  REJECT(NormBwd, DG_EINVAL, c.dx = addr(1));
  REJECT(NormBwd, DG_EINVAL, c.dx = shift(addr(4), 16));
  const int64_t rows[] = {1, 3, 64, 2048, 2049, 8192, (int64_t)1 << 22, DG_MAX_DIM};
  const int64_t cols[] = {64, 512, 576, 2048, 4096, 8192, 16384, 16448, 1 << 20, DG_MAX_DIM};
  for (int64_t r : rows)
    for (int64_t n : cols) {
      const int64_t b = dg_rmsnorm_backward_workspace(r, n);
      expect(b >= 0 && b % (4 * n) == 0 && b / (4 * n) <= r, 1, "workspace size", r, n);
    }
}

void epi() {
  for (int64_t d : kDims) {
    REJECT(Epi, DG_EINVAL, c.rows = d);
    REJECT(Epi, DG_EINVAL, c.cols = d);
    REJECT(Epi, DG_EINVAL, c.lddout = d);
    REJECT(Epi, DG_EINVAL, c.ldpre = d);
    expect(dg_epilogue_backward_workspace(d, 256, 128, 128), DG_EINVAL, "workspace rows", d);
    expect(dg_epilogue_backward_workspace(64, d, 128, 1), DG_EINVAL, "workspace cols", d);
  }
  for (int g : {0, -128, 32, 96, 512, std::numeric_limits<int>::min()}) {
    REJECT(Epi, DG_EINVAL, (c.gran = g, c.br = g));
    expect(dg_epilogue_backward_workspace(64, 256, g, g), DG_EINVAL, "workspace gran", g);
  }
  REJECT(Epi, DG_EINVAL, c.pre = nullptr);
  REJECT(Epi, DG_EINVAL, c.act = DG_ACT_NONE);
  REJECT(Epi, DG_EINVAL, c.act = 5);
  REJECT(Epi, DG_EINVAL, c.br = 2);
  REJECT(Epi, DG_EINVAL, (c.rows = 5000, c.nb = 16));
  REJECT(Epi, DG_EALIGN, c.ldpre = 260);
  REJECT(Epi, DG_EALIGN, c.db = shift(faddr(3), 2));
  REJECT(Epi, DG_EINVAL, c.dz = addr(1));
  REJECT(Epi, DG_EINVAL, (c.dz = addr(0), c.lddout = 512));
  REJECT(Epi, DG_EINVAL, (c.rows = DG_MAX_DIM, c.cols = DG_MAX_DIM, c.lddout = DG_MAX_DIM, c.ldpre = DG_MAX_DIM, c.gran = 256, c.br = 256));
  for (int64_t r : {(int64_t)1, (int64_t)1024, (int64_t)1025, (int64_t)DG_MAX_DIM})
    for (int64_t n : {(int64_t)256, (int64_t)4096, (int64_t)1 << 20})
      for (int g : {64, 128, 256})
        for (int br : {g, 1}) {
          const int64_t b = dg_epilogue_backward_workspace(r, n, g, br);
          const bool fits = br == 1 || ((r + g - 1) / g) * (n / g) <= (g == 64 ? 0xffffff : 0x3fffff);
          expect(fits ? b >= 0 && b % (4 * n) == 0 && b / (4 * n) <= r : b == DG_EINVAL, 1, "workspace size", r, n);
        }
}

void gemm() {
  for (int64_t d : kDims) {
    REJECT(Gemm, DG_EINVAL, c.M = d);
    REJECT(Gemm, DG_EINVAL, c.N = d);
    REJECT(Gemm, DG_EINVAL, c.K = d);
    REJECT(Gemm, DG_EINVAL, c.ldres = d);
    expect(dg_gemm_fp8_residual_workspace(d, 256, 256, 128, 0), DG_EINVAL, "workspace M", d);
    expect(dg_gemm_fp8_residual_workspace(256, 256, d, 128, 0), DG_EINVAL, "workspace K", d);
  }
  REJECT(Gemm, DG_EINVAL, c.out = nullptr);
  REJECT(Gemm, DG_EINVAL, c.act = 5);
  REJECT(Gemm, DG_EINVAL, c.rk = 3);
  REJECT(Gemm, DG_EINVAL, c.layout = 4);
  REJECT(Gemm, DG_EINVAL, c.pre = addr(6));
  REJECT(Gemm, DG_EINVAL, (c.res = addr(4), c.rk = DG_IN_F16));
  REJECT(Gemm, DG_EINVAL, (c.ws = addr(8), c.nb = 0));
  REJECT(Gemm, DG_EINVAL, (c.M = 64, c.N = 64, c.K = 8192, c.ldres = 64, c.ws = addr(8), c.nb = 64));
  REJECT(Gemm, DG_EALIGN, c.pre = shift(addr(7), 1));
  REJECT(Gemm, DG_EALIGN, c.res = shift(addr(6), 1));
  REJECT(Gemm, DG_EINVAL, (c.M = c.N = c.ldres = DG_MAX_DIM));
  for (int layout = -1; layout <= 4; ++layout)
    for (int64_t m : {(int64_t)1, (int64_t)64, (int64_t)4096, (int64_t)DG_MAX_DIM})
      for (int64_t k : {(int64_t)256, (int64_t)6144, (int64_t)8192, (int64_t)DG_MAX_DIM}) {
        const int64_t b = dg_gemm_fp8_residual_workspace(m, 512, k, 128, layout);
        expect(layout < 0 || layout > 3 ? b == DG_EINVAL : b >= 0 && b % (4 * 64 * 64) == 0, 1, "workspace size", m, k);
      }
}

}  // namespace

int main() {
  norm();
  norm_bwd();
  epi();
  gemm();
  if (g_failures) {
    std::fprintf(stderr, "%d checks failed\n", g_failures);
    return 1;
  }
  std::printf("layer host checks passed\n");
  return 0;
}

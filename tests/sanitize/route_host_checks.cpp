// The calls of experts and adapters under AddressSanitizer and
// UndefinedBehaviorSanitizer, as host_checks.cpp does it for the others: every
// call carries one argument error, so each returns before its first HIP call,
// and the size queries take extreme sizes. Exit status 0 when every call
// returns what the header promises.

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

void expect(int64_t got, int64_t want, const char* what, long long a = 0) {
  if (got != want) {
    ++g_failures;
    std::fprintf(stderr, "FAILED: %s (%lld): got %lld, want %lld\n", what, a, (long long)got, (long long)want);
  }
}

void* addr(int i) { return reinterpret_cast<void*>((uintptr_t)(i + 1) << 52); }
template <class T>
T* at(int i, uintptr_t by = 0) {
  return reinterpret_cast<T*>(((uintptr_t)(i + 1) << 52) + by);
}

struct Sort {
  const void* ids = addr(0);
  int bytes = 8;
  int64_t tokens = 5000;
  int k = 2, groups = 8, align = 16;
  int32_t *off = at<int32_t>(1), *pos = at<int32_t>(2), *slot = at<int32_t>(3);
  int64_t rows = 20000;
  void* ws = addr(4);
  int64_t nb = 1 << 20;
  int operator()() const { return dg_route_sort(ids, bytes, tokens, k, groups, align, off, pos, slot, rows, ws, nb, nullptr); }
};

struct Rows {
  const void* x = addr(0);
  int xk = DG_IN_BF16;
  int64_t ldx = 256, tokens = 100, cols = 256;
  int k = 2;
  const int32_t *pos = at<int32_t>(1), *slot = at<int32_t>(2);
  int64_t rows = 512;
  const float* w = at<float>(3);
  int gran = 128, br = 128, fmt = DG_FMT_E5M2;
  void* q = addr(4);
  float* s = at<float>(5);
  void* ws = addr(6);
  int64_t nb = (int64_t)1 << 40;
  int operator()() const { return dg_route_quantize_fp8(x, xk, ldx, tokens, cols, k, pos, slot, rows, w, gran, br, fmt, q, s, ws, nb, nullptr); }
};

struct Combine {
  const void* y = addr(0);
  int yk = DG_IN_F16;
  int64_t ldy = 256, rows = 512, tokens = 100, cols = 256;
  int k = 2;
  const int32_t* pos = at<int32_t>(1);
  const float* w = at<float>(2);
  const void* res = addr(3);
  int64_t ldres = 256;
  void* out = addr(4);
  int ok = DG_IN_F32;
  int operator()() const { return dg_route_combine(y, yk, ldy, rows, tokens, cols, k, pos, w, res, ldres, out, ok, nullptr); }
};

struct Weights {
  const void *x = addr(0), *y = addr(1);
  int xk = DG_IN_F32, yk = DG_IN_BF16;
  int64_t ldx = 256, ldy = 256, rows = 512, tokens = 100, cols = 256;
  int k = 2;
  const int32_t* pos = at<int32_t>(2);
  float* dw = at<float>(3);
  int operator()() const { return dg_route_weight_grad(x, xk, ldx, y, yk, ldy, rows, tokens, cols, k, pos, dw, nullptr); }
};

struct Grouped {
  const void *a = addr(0), *b = addr(1);
  const float *sa = at<float>(2), *sb = at<float>(3);
  const int32_t* off = at<int32_t>(4);
  int groups = 8;
  void* out = addr(5);
  int64_t rows = 512, N = 96, K = 256;
  int gran = 128, layout = DG_LAYOUT_NN, sr = 1, fa = 0, fb = 1, act = DG_ACT_GELU;
  void* pre = addr(6);
  int operator()() const { return dg_gemm_fp8_grouped(a, b, sa, sb, off, groups, out, rows, N, K, gran, layout, sr, fa, fb, act, pre, nullptr); }
};

struct Wgrad {
  const void *a = addr(0), *b = addr(1);
  const float *sa = at<float>(2), *sb = at<float>(3);
  const int32_t* off = at<int32_t>(4);
  int groups = 8;
  void* out = addr(5);
  int64_t rows = 512, M = 256, N = 384;
  int gran = 128, fa = 1, fb = 0;
  int operator()() const { return dg_gemm_fp8_grouped_wgrad(a, b, sa, sb, off, groups, out, rows, M, N, gran, fa, fb, nullptr); }
};

struct Lora {
  const void *x = addr(0), *a = addr(1), *b = addr(2);
  int kind = DG_IN_BF16;
  int64_t ldx = 512, tokens = 64, K = 512;
  const float* scale = at<float>(3);
  int64_t N = 100;
  int rank = 16, groups = 8;
  const int32_t *off = at<int32_t>(4), *pos = at<int32_t>(5), *slot = at<int32_t>(6);
  const void* base = addr(7);
  int64_t ldbase = 100;
  void* out = addr(8);
  int ok = DG_IN_F32;
  void* ws = addr(9);
  int64_t nb = (int64_t)1 << 40;
  int operator()() const {
    return dg_lora(x, kind, ldx, tokens, K, a, b, scale, N, rank, groups, off, pos, slot, base, ldbase, out, ok, ws, nb, nullptr);
  }
};

// Each value of a field in turn, with the rest as they are.
template <class Call, class T>
void bad(const char* what, T Call::*field, std::initializer_list<T> values, int want = DG_EINVAL) {
  for (T v : values) {
    Call c;
    c.*field = v;
    expect(c(), want, what);
  }
}

constexpr int64_t kHuge = std::numeric_limits<int64_t>::max(), kLow = std::numeric_limits<int64_t>::min();
constexpr int kMaxInt = std::numeric_limits<int>::max(), kMinInt = std::numeric_limits<int>::min();

}  // namespace

int main() {
  const std::initializer_list<int64_t> sizes = {0, -1, kHuge, kLow, (int64_t)1 << 62, (int64_t)1 << 24};
  const std::initializer_list<int> ints = {0, -1, kMinInt};

  bad("sort tokens", &Sort::tokens, sizes);
  bad("sort rows", &Sort::rows, sizes);
  bad("sort k", &Sort::k, {0, -1, kMinInt, kMaxInt});
  bad("sort groups", &Sort::groups, {0, -1, kMinInt, kMaxInt, DG_MAX_GROUPS + 1});
  bad("sort align", &Sort::align, {0, -1, kMinInt, kMaxInt});
  bad("sort bytes", &Sort::bytes, {0, 2, 16, kMinInt});
  bad("sort workspace", &Sort::nb, {(int64_t)0, (int64_t)-1, kLow});
  bad("sort ids", &Sort::ids, {(const void*)nullptr});
  bad("sort ids address", &Sort::ids, {(const void*)at<char>(0, 4)}, DG_EALIGN);

  bad("rows tokens", &Rows::tokens, sizes);
  bad("rows cols", &Rows::cols, sizes);
  bad("rows rows", &Rows::rows, sizes);
  bad("rows ldx", &Rows::ldx, {(int64_t)0, (int64_t)-1, kHuge, kLow, (int64_t)255});
  bad("rows k", &Rows::k, {0, -1, kMinInt, kMaxInt});
  bad("rows gran", &Rows::gran, {0, -1, 1, 96, 512, kMinInt, kMaxInt});
  bad("rows block rows", &Rows::br, {0, -1, 64, 256, kMinInt, kMaxInt});
  bad("rows format", &Rows::fmt, {-1, 2, kMinInt, kMaxInt});
  bad("rows type", &Rows::xk, {-1, 3, kMinInt, kMaxInt});
  bad("rows workspace", &Rows::nb, {(int64_t)-1, kLow});
  bad("rows q in x", &Rows::q, {addr(0)});

  bad("combine tokens", &Combine::tokens, sizes);
  bad("combine rows", &Combine::rows, sizes);
  bad("combine cols", &Combine::cols, sizes);
  bad("combine ldy", &Combine::ldy, {(int64_t)0, (int64_t)-8, kHuge, kLow});
  bad("combine ldres", &Combine::ldres, {(int64_t)0, (int64_t)-8, kHuge, kLow});
  bad("combine k", &Combine::k, ints);
  bad("combine type", &Combine::yk, {-1, 3, kMaxInt});
  bad("combine out type", &Combine::ok, {-1, 3, kMaxInt});

  bad("weights tokens", &Weights::tokens, sizes);
  bad("weights rows", &Weights::rows, sizes);
  bad("weights cols", &Weights::cols, sizes);
  bad("weights ldx", &Weights::ldx, {(int64_t)0, (int64_t)-8, kHuge, kLow});
  bad("weights ldy", &Weights::ldy, {(int64_t)0, (int64_t)-8, kHuge, kLow});
  bad("weights k", &Weights::k, ints);

  bad("grouped rows", &Grouped::rows, sizes);
  bad("grouped N", &Grouped::N, sizes);
  bad("grouped K", &Grouped::K, sizes);
  bad("grouped groups", &Grouped::groups, {0, -1, kMinInt, kMaxInt, DG_MAX_GROUPS + 1});
  bad("grouped gran", &Grouped::gran, {0, -1, 32, kMinInt, kMaxInt});
  bad("grouped layout", &Grouped::layout, {-1, 2, 3, kMinInt, kMaxInt});
  bad("grouped rows of factors", &Grouped::sr, {0, -1, 64, kMinInt, kMaxInt});
  bad("grouped activation", &Grouped::act, {-1, 5, kMinInt, kMaxInt});

  bad("wgrad rows", &Wgrad::rows, sizes);
  bad("wgrad M", &Wgrad::M, sizes);
  bad("wgrad N", &Wgrad::N, sizes);
  bad("wgrad groups", &Wgrad::groups, {0, -1, kMinInt, kMaxInt, DG_MAX_GROUPS + 1});
  bad("wgrad gran", &Wgrad::gran, {0, -1, 32, kMinInt, kMaxInt});

  bad("lora tokens", &Lora::tokens, sizes);
  bad("lora K", &Lora::K, sizes);
  bad("lora N", &Lora::N, sizes);
  bad("lora rank", &Lora::rank, {0, -1, 4, 136, kMinInt, kMaxInt});
  bad("lora groups", &Lora::groups, {0, -1, kMinInt, kMaxInt, DG_MAX_GROUPS + 1});
  bad("lora ldx", &Lora::ldx, {(int64_t)0, (int64_t)-8, kHuge, kLow});
  bad("lora ldbase", &Lora::ldbase, {(int64_t)0, (int64_t)-8, kHuge, kLow});
  bad("lora workspace", &Lora::nb, {(int64_t)0, (int64_t)-1, kLow});
  bad("lora type", &Lora::kind, {0, -1, 3, kMaxInt});
  bad("lora out type", &Lora::ok, {-1, 3, kMaxInt});

  for (int64_t n : sizes) {
    expect(dg_route_rows(n, 2, 8, 16), DG_EINVAL, "rows query", n);
    expect(dg_route_sort_workspace(n, 2, 8), DG_EINVAL, "sort query", n);
    expect(dg_route_quantize_workspace(n, 256, 2, 512, 128, 128), DG_EINVAL, "rows workspace, tokens", n);
    expect(dg_route_quantize_workspace(100, n, 2, 512, 128, 128), DG_EINVAL, "rows workspace, cols", n);
    expect(dg_route_quantize_workspace(100, 256, 2, n, 128, 128), DG_EINVAL, "rows workspace, rows", n);
    expect(dg_lora_workspace(n, 512, 100, 16, 8), DG_EINVAL, "lora workspace, tokens", n);
    expect(dg_lora_workspace(64, n, 100, 16, 8), DG_EINVAL, "lora workspace, K", n);
    expect(dg_lora_workspace(64, 512, n, 16, 8), DG_EINVAL, "lora workspace, N", n);
  }
  for (int n : {0, -1, kMinInt, kMaxInt}) {
    expect(dg_route_rows(100, n, 8, 16), DG_EINVAL, "rows query, k", n);
    expect(dg_route_rows(100, 2, n, 16), DG_EINVAL, "rows query, groups", n);
    expect(dg_route_rows(100, 2, 8, n), DG_EINVAL, "rows query, align", n);
    expect(dg_route_sort_workspace(100, n, 8), DG_EINVAL, "sort query, k", n);
    expect(dg_route_sort_workspace(100, 2, n), DG_EINVAL, "sort query, groups", n);
    expect(dg_lora_workspace(64, 512, 100, n, 8), DG_EINVAL, "lora workspace, rank", n);
    expect(dg_lora_workspace(64, 512, 100, 16, n), DG_EINVAL, "lora workspace, groups", n);
  }
  if (g_failures) return 1;
  std::printf("route host checks passed\n");
  return 0;
}

// The short way from PyTorch tensors to the C ABI for the calls that serve a
// few tokens (the norm, the product with a residual, their gradients): a call
// whose arguments are plainly right is checked and launched here, in about
// 0.5 us beside the 3.4 us of the launch, where the checks in Python take
// four. Anything else (an argument that is missing or wrong, a tensor
// subclass, a given stream, another current device) is left to the Python
// functions, which allocate, find what is wrong and raise; nothing is refused
// here.
//
// Every function returns the C ABI's status, or None where it leaves the call
// to Python. The C ABI's entry points come from the library that the package
// has open (bind).

#include <torch/csrc/autograd/python_variable.h>

#include <ATen/ATen.h>
#include <Python.h>
#include <c10/hip/HIPFunctions.h>
#include <c10/hip/HIPStream.h>

#include <cstdint>

#include "../../include/dg.h"

namespace {

decltype(&dg_rmsnorm_quantize_fp8) g_norm;
decltype(&dg_rmsnorm_backward) g_norm_bwd;
decltype(&dg_rmsnorm_backward_workspace) g_norm_bwd_ws;
decltype(&dg_epilogue_backward_fp8) g_epi_bwd;
decltype(&dg_epilogue_backward_workspace) g_epi_bwd_ws;
decltype(&dg_gemm_fp8_residual) g_gemm;
decltype(&dg_gemm_fp8_residual_workspace) g_gemm_ws;
decltype(&dg_route_sort) g_sort;
decltype(&dg_route_sort_workspace) g_sort_ws;
decltype(&dg_route_quantize_fp8) g_rows;
decltype(&dg_route_quantize_workspace) g_rows_ws;
decltype(&dg_route_combine) g_combine;
decltype(&dg_route_weight_grad) g_weight_grad;
decltype(&dg_gemm_fp8_grouped) g_grouped;
decltype(&dg_gemm_fp8_grouped_wgrad) g_wgrad;
decltype(&dg_lora) g_lora;
decltype(&dg_lora_workspace) g_lora_ws;

// What one call's arguments are checked against: dev is the first tensor's
// device; ok turns false at the first argument that is not plainly right.
struct Call {
  bool ok = true;
  c10::Device dev{c10::DeviceType::CPU};

  const at::Tensor* tensor(PyObject* o) {
    if (!ok || !THPVariable_CheckExact(o)) return fail();
    const at::Tensor& t = THPVariable_Unpack(o);
    if (!t.defined() || t.layout() != c10::kStrided) return fail();
    return &t;
  }

  const at::Tensor* fail() {
    ok = false;
    return nullptr;
  }

  // The tensor that sets the device: 2-D, on the current GPU.
  const at::Tensor* first(PyObject* o) {
    const at::Tensor* t = tensor(o);
    if (!t) return nullptr;
    dev = t->device();
    if (t->dim() != 2 || !t->is_cuda() || dev.index() != c10::hip::current_device()) return fail();
    return t;
  }

  static bool fp8(c10::ScalarType t, int fmt) {
    return t == c10::ScalarType::Byte ||
           t == (fmt == DG_FMT_E5M2 ? c10::ScalarType::Float8_e5m2 : c10::ScalarType::Float8_e4m3fn);
  }

  static int kind(c10::ScalarType t) {
    return t == c10::ScalarType::Float      ? DG_IN_F32
           : t == c10::ScalarType::BFloat16 ? DG_IN_BF16
           : t == c10::ScalarType::Half     ? DG_IN_F16
                                            : -1;
  }

  // An input matrix of one of the three kinds, its rows contiguous.
  struct Rows {
    void* p = nullptr;
    int kind = 0;
    int64_t pitch = 0;
  };
  Rows rows(PyObject* o, int64_t r, int64_t c, int want = -1) {
    Rows m;
    const at::Tensor* t = tensor(o);
    if (!t) return m;
    m.kind = kind(t->scalar_type());
    if (m.kind < 0 || (want >= 0 && m.kind != want) || t->dim() != 2 || t->size(0) != r || t->size(1) != c ||
        t->device() != dev)
      return fail(), m;
    if (t->is_contiguous()) {
      m.pitch = c;
    } else {
      if ((t->stride(1) != 1 && c > 1) || (t->stride(0) < c && r > 1)) return fail(), m;
      m.pitch = r > 1 ? t->stride(0) : c;
    }
    m.p = t->data_ptr();
    return m;
  }
  Rows rows_or_none(PyObject* o, int64_t r, int64_t c, int want = -1) {
    return o == Py_None ? Rows{} : rows(o, r, c, want);
  }

  void* take(const at::Tensor* t, bool type_ok) {
    if (!t || !type_ok || !t->is_contiguous() || t->device() != dev) return fail(), nullptr;
    return t->data_ptr();
  }
  // A contiguous matrix or vector of a given type.
  void* mat(PyObject* o, c10::ScalarType type, int64_t r, int64_t c) {
    const at::Tensor* t = tensor(o);
    return take(t, t && t->scalar_type() == type && t->dim() == 2 && t->size(0) == r && t->size(1) == c);
  }
  void* vec(PyObject* o, int64_t n) {
    const at::Tensor* t = tensor(o);
    return take(t, t && t->scalar_type() == c10::ScalarType::Float && t->dim() == 1 && t->size(0) == n);
  }
  void* codes(PyObject* o, int fmt, int64_t r, int64_t c) {
    const at::Tensor* t = tensor(o);
    return take(t, t && fp8(t->scalar_type(), fmt) && t->dim() == 2 && t->size(0) == r && t->size(1) == c);
  }
  // A contiguous [n][r][c] of codes (fmt >= 0) or of a given type.
  void* cube(PyObject* o, int fmt, c10::ScalarType type, int64_t n, int64_t r, int64_t c) {
    const at::Tensor* t = tensor(o);
    return take(t, t && (fmt >= 0 ? fp8(t->scalar_type(), fmt) : t->scalar_type() == type) && t->dim() == 3 && t->size(0) == n &&
                       t->size(1) == r && t->size(2) == c);
  }
  // A contiguous int32 vector: its length (0 where it is none).
  int64_t indices(PyObject* o, void** p) {
    const at::Tensor* t = tensor(o);
    *p = take(t, t && t->scalar_type() == c10::ScalarType::Int && t->dim() == 1);
    return ok ? t->size(0) : 0;
  }
  void* mat_or_none(PyObject* o, c10::ScalarType type, int64_t r, int64_t c) {
    return o == Py_None ? nullptr : mat(o, type, r, c);
  }
  void* vec_or_none(PyObject* o, int64_t n) { return o == Py_None ? nullptr : vec(o, n); }

  int64_t integer(PyObject* o) {
    if (!ok || !PyLong_CheckExact(o)) return fail(), 0;
    int over = 0;
    const long long v = PyLong_AsLongLongAndOverflow(o, &over);
    if (over) ok = false;
    return v;
  }
  double real(PyObject* o) {
    if (!ok || !PyFloat_CheckExact(o)) return fail(), 0.0;
    return PyFloat_AS_DOUBLE(o);
  }

  void* stream() const { return (void*)c10::hip::getCurrentHIPStream(dev.index()).stream(); }

  // The caller's workspace, or one of `need` bytes from torch's allocator on
  // the current stream, which the tensor frees in that stream's order.
  at::Tensor workspace(PyObject* o, int64_t need) {
    if (o != Py_None) {
      const at::Tensor* t = tensor(o);
      if (!take(t, t && t->scalar_type() == c10::ScalarType::Byte && t->dim() == 1) && ok) ok = false;
      return ok ? *t : at::Tensor();
    }
    return at::empty({need}, at::TensorOptions().dtype(c10::ScalarType::Byte).device(dev));
  }
};

bool good_gran(int64_t g, int64_t cols) { return (g == 64 || g == 128 || g == 256) && cols % g == 0; }
bool good_fmt(int64_t f) { return f == DG_FMT_E4M3 || f == DG_FMT_E5M2; }
bool good_act(int64_t a) { return a >= DG_ACT_NONE && a <= DG_ACT_GELU_TANH; }

PyObject* status(int rc) { return PyLong_FromLong(rc); }

// A C++ exception (torch's allocator, say) leaves the call to Python, where the same one is raised as usual.
template <class F>
PyObject* guarded(F f) {
  try {
    return f();
  } catch (...) {
    Py_RETURN_NONE;
  }
}

// x, res, weight, eps, gran, fmt, h, y, rstd, q, scales
PyObject* rmsnorm_quantize(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Call k;
    const at::Tensor* x = n == 11 ? k.first(a[0]) : nullptr;
    if (!x) Py_RETURN_NONE;
    const int64_t r = x->size(0), c = x->size(1);
    const auto in = k.rows(a[0], r, c), res = k.rows_or_none(a[1], r, c);
    void* w = k.vec(a[2], c);
    const double eps = k.real(a[3]);
    const int64_t g = k.integer(a[4]), fmt = k.integer(a[5]);
    if (!k.ok || !good_gran(g, c) || !good_fmt(fmt) || (a[1] == Py_None) != (a[6] == Py_None)) Py_RETURN_NONE;
    const auto type = x->scalar_type();
    void* h = res.p ? k.mat(a[6], THPVariable_Unpack(a[1]).scalar_type(), r, c) : nullptr;
    void* y = k.mat_or_none(a[7], type, r, c);
    void* rstd = k.vec_or_none(a[8], r);
    void* q = k.codes(a[9], (int)fmt, r, c);
    void* s = k.mat(a[10], c10::ScalarType::Float, r, c / g);
    if (!k.ok) Py_RETURN_NONE;
    return status(g_norm(in.p, in.kind, in.pitch, res.p, res.kind, res.pitch, (const float*)w, (float)eps, r, c, (int)g,
                         (int)fmt, h, y, (float*)rstd, q, (float*)s, k.stream()));
  });
}

// dy, h, rstd, weight, dh, dx, dweight, workspace
PyObject* rmsnorm_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Call k;
    const at::Tensor* dy = n == 8 ? k.first(a[0]) : nullptr;
    if (!dy) Py_RETURN_NONE;
    const int64_t r = dy->size(0), c = dy->size(1);
    const auto g = k.rows(a[0], r, c), h = k.rows(a[1], r, c);
    void* rstd = k.vec(a[2], r);
    void* w = k.vec(a[3], c);
    if (!k.ok) Py_RETURN_NONE;
    const auto dh = k.rows_or_none(a[4], r, c, h.kind);
    void* dx = k.mat(a[5], THPVariable_Unpack(a[1]).scalar_type(), r, c);
    void* dw = k.vec(a[6], c);
    const int64_t need = g_norm_bwd_ws(r, c);
    if (!k.ok || need < 0) Py_RETURN_NONE;
    at::Tensor ws;
    if (need) ws = k.workspace(a[7], need);
    if (!k.ok) Py_RETURN_NONE;
    return status(g_norm_bwd(g.p, g.kind, g.pitch, h.p, h.kind, h.pitch, (const float*)rstd, (const float*)w, dh.p, dh.pitch,
                             r, c, dx, (float*)dw, need ? ws.data_ptr() : nullptr, need ? ws.numel() : 0, k.stream()));
  });
}

// dout, pre, act, gran, block_rows, fmt, dz, dbias, q, scales, workspace
PyObject* epilogue_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Call k;
    const at::Tensor* d = n == 11 ? k.first(a[0]) : nullptr;
    if (!d) Py_RETURN_NONE;
    const int64_t r = d->size(0), c = d->size(1);
    const auto in = k.rows(a[0], r, c), pre = k.rows_or_none(a[1], r, c, DG_IN_BF16);
    const int64_t act = k.integer(a[2]), g = k.integer(a[3]), br = k.integer(a[4]), fmt = k.integer(a[5]);
    if (!k.ok || !good_gran(g, c) || !good_fmt(fmt) || !good_act(act) || (br != g && br != 1) ||
        (act == DG_ACT_NONE) != (pre.p == nullptr))
      Py_RETURN_NONE;
    void* dz = k.mat_or_none(a[6], d->scalar_type(), r, c);
    void* db = k.vec_or_none(a[7], c);
    void* q = k.codes(a[8], (int)fmt, r, c);
    void* s = k.mat(a[9], c10::ScalarType::Float, (r + br - 1) / br, c / g);
    if (!k.ok) Py_RETURN_NONE;
    const int64_t need = db ? g_epi_bwd_ws(r, c, (int)g, (int)br) : 0;
    if (need < 0) Py_RETURN_NONE;
    at::Tensor ws;
    if (need) ws = k.workspace(a[10], need);
    if (!k.ok) Py_RETURN_NONE;
    return status(g_epi_bwd(in.p, in.kind, in.pitch, pre.p, pre.pitch, (int)act, r, c, (int)g, (int)br, (int)fmt, dz,
                            (float*)db, q, (float*)s, need ? ws.data_ptr() : nullptr, need ? ws.numel() : 0, k.stream()));
  });
}

// a, b, sa, sb, res, out, gran, layout, sa_rows, fmt_a, fmt_b, bias, act, pre, workspace
PyObject* gemm_residual(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Call k;
    const at::Tensor* A = n == 15 ? k.first(a[0]) : nullptr;
    const at::Tensor* B = A ? k.tensor(a[1]) : nullptr;
    if (!B || B->dim() != 2) Py_RETURN_NONE;
    const int64_t g = k.integer(a[6]), layout = k.integer(a[7]), sr = k.integer(a[8]), fa = k.integer(a[9]),
                  fb = k.integer(a[10]), act = k.integer(a[12]);
    if (!k.ok || layout < DG_LAYOUT_NT || layout > DG_LAYOUT_TN || !good_fmt(fa) || !good_fmt(fb) || !good_act(act))
      Py_RETURN_NONE;
    const bool ta = layout & 2, tb = layout & 1;
    const int64_t M = A->size(ta ? 1 : 0), K = A->size(ta ? 0 : 1), N = B->size(tb ? 1 : 0);
    if (!good_gran(g, K) || (sr != g && sr != 1)) Py_RETURN_NONE;
    void* pa = k.codes(a[0], (int)fa, ta ? K : M, ta ? M : K);
    void* pb = k.codes(a[1], (int)fb, tb ? K : N, tb ? N : K);
    void* sa = k.mat(a[2], c10::ScalarType::Float, (M + sr - 1) / sr, K / g);
    void* sb = k.mat(a[3], c10::ScalarType::Float, (N + g - 1) / g, K / g);
    const auto res = k.rows_or_none(a[4], M, N);
    void* out = k.mat(a[5], c10::ScalarType::BFloat16, M, N);
    void* bias = k.vec_or_none(a[11], N);
    void* pre = k.mat_or_none(a[13], c10::ScalarType::BFloat16, M, N);
    if (!k.ok) Py_RETURN_NONE;
    const int64_t need = g_gemm_ws(M, N, K, (int)g, (int)layout);
    if (need < 0) Py_RETURN_NONE;
    at::Tensor ws;
    if (need) ws = k.workspace(a[14], need);
    if (!k.ok) Py_RETURN_NONE;
    return status(g_gemm(pa, pb, (const float*)sa, (const float*)sb, out, M, N, K, (int)g, (int)layout, (int)sr, (int)fa,
                         (int)fb, (const float*)bias, (int)act, res.p, res.kind, res.pitch, pre,
                         need ? ws.data_ptr() : nullptr, need ? ws.numel() : 0, k.stream()));
  });
}

constexpr auto kInt = c10::ScalarType::Int;

// ids, groups, align, offsets, position, slot, workspace
PyObject* route_sort(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Call k;
    const at::Tensor* ids = n == 7 ? k.first(a[0]) : nullptr;
    if (!ids) Py_RETURN_NONE;
    const auto type = ids->scalar_type();
    if (type != kInt && type != c10::ScalarType::Long) Py_RETURN_NONE;
    const int64_t r = ids->size(0), c = ids->size(1), groups = k.integer(a[1]), align = k.integer(a[2]);
    void* id = k.take(ids, true);
    void *off, *slot;
    const int64_t no = k.indices(a[3], &off);
    void* pos = k.mat(a[4], kInt, r, c);
    const int64_t rows = k.indices(a[5], &slot);
    if (!k.ok || groups < 1 || groups > DG_MAX_GROUPS || align < 1 || align > DG_MAX_DIM || no != groups + 1 || c > DG_MAX_DIM)
      Py_RETURN_NONE;
    const int64_t need = g_sort_ws(r, (int)c, (int)groups);
    if (need < 0) Py_RETURN_NONE;
    at::Tensor ws;
    if (need) ws = k.workspace(a[6], need);
    if (!k.ok) Py_RETURN_NONE;
    return status(g_sort(id, type == kInt ? 4 : 8, r, (int)c, (int)groups, (int)align, (int32_t*)off, (int32_t*)pos, (int32_t*)slot,
                         rows, need ? ws.data_ptr() : nullptr, need ? ws.numel() : 0, k.stream()));
  });
}

// x, position, slot, weights, gran, block_rows, fmt, q, scales, workspace
PyObject* route_quantize(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Call k;
    const at::Tensor* x = n == 10 ? k.first(a[0]) : nullptr;
    const at::Tensor* pt = x ? k.tensor(a[1]) : nullptr;
    if (!pt || pt->dim() != 2) Py_RETURN_NONE;
    const int64_t r = x->size(0), c = x->size(1), kk = pt->size(1);
    const auto in = k.rows(a[0], r, c);
    void* pos = k.mat(a[1], kInt, r, kk);
    void* slot;
    const int64_t rows = k.indices(a[2], &slot);
    void* w = k.mat_or_none(a[3], c10::ScalarType::Float, r, kk);
    const int64_t g = k.integer(a[4]), br = k.integer(a[5]), fmt = k.integer(a[6]);
    if (!k.ok || !good_gran(g, c) || !good_fmt(fmt) || (br != g && br != 1) || kk > DG_MAX_DIM) Py_RETURN_NONE;
    void* q = k.codes(a[7], (int)fmt, rows, c);
    void* s = k.mat(a[8], c10::ScalarType::Float, (rows + br - 1) / br, c / g);
    if (!k.ok) Py_RETURN_NONE;
    const int64_t need = g_rows_ws(r, c, (int)kk, rows, (int)g, (int)br);
    if (need < 0) Py_RETURN_NONE;
    at::Tensor ws;
    if (need) ws = k.workspace(a[9], need);
    if (!k.ok) Py_RETURN_NONE;
    return status(g_rows(in.p, in.kind, in.pitch, r, c, (int)kk, (const int32_t*)pos, (const int32_t*)slot, rows, (const float*)w,
                         (int)g, (int)br, (int)fmt, q, (float*)s, need ? ws.data_ptr() : nullptr, need ? ws.numel() : 0, k.stream()));
  });
}

// y, position, weights, res, out
PyObject* route_combine(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Call k;
    const at::Tensor* y = n == 5 ? k.first(a[0]) : nullptr;
    const at::Tensor* pt = y ? k.tensor(a[1]) : nullptr;
    const at::Tensor* ot = pt ? k.tensor(a[4]) : nullptr;
    if (!ot || pt->dim() != 2) Py_RETURN_NONE;
    const int64_t rows = y->size(0), c = y->size(1), r = pt->size(0), kk = pt->size(1);
    const auto in = k.rows(a[0], rows, c);
    void* pos = k.mat(a[1], kInt, r, kk);
    void* w = k.mat_or_none(a[2], c10::ScalarType::Float, r, kk);
    const int ok = Call::kind(ot->scalar_type());
    if (!k.ok || ok < 0 || kk > DG_MAX_DIM) Py_RETURN_NONE;
    const auto res = k.rows_or_none(a[3], r, c, ok);
    void* out = k.mat(a[4], ot->scalar_type(), r, c);
    if (!k.ok) Py_RETURN_NONE;
    return status(g_combine(in.p, in.kind, in.pitch, rows, r, c, (int)kk, (const int32_t*)pos, (const float*)w, res.p, res.pitch, out,
                            ok, k.stream()));
  });
}

// dout, y, position, dweights
PyObject* route_weight_grad(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Call k;
    const at::Tensor* d = n == 4 ? k.first(a[0]) : nullptr;
    const at::Tensor* yt = d ? k.tensor(a[1]) : nullptr;
    const at::Tensor* pt = yt ? k.tensor(a[2]) : nullptr;
    if (!pt || pt->dim() != 2 || yt->dim() != 2) Py_RETURN_NONE;
    const int64_t r = d->size(0), c = d->size(1), rows = yt->size(0), kk = pt->size(1);
    const auto in = k.rows(a[0], r, c), y = k.rows(a[1], rows, c);
    void* pos = k.mat(a[2], kInt, r, kk);
    void* dw = k.mat(a[3], c10::ScalarType::Float, r, kk);
    if (!k.ok || kk > DG_MAX_DIM) Py_RETURN_NONE;
    return status(g_weight_grad(in.p, in.kind, in.pitch, y.p, y.kind, y.pitch, rows, r, c, (int)kk, (const int32_t*)pos, (float*)dw,
                                k.stream()));
  });
}

// a, b, sa, sb, offsets, out, gran, layout, sa_rows, fmt_a, fmt_b, act, pre
PyObject* gemm_grouped(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Call k;
    const at::Tensor* A = n == 13 ? k.first(a[0]) : nullptr;
    const at::Tensor* B = A ? k.tensor(a[1]) : nullptr;
    if (!B || B->dim() != 3) Py_RETURN_NONE;
    const int64_t g = k.integer(a[6]), layout = k.integer(a[7]), sr = k.integer(a[8]), fa = k.integer(a[9]), fb = k.integer(a[10]),
                  act = k.integer(a[11]);
    if (!k.ok || (layout != DG_LAYOUT_NT && layout != DG_LAYOUT_NN) || !good_fmt(fa) || !good_fmt(fb) || !good_act(act))
      Py_RETURN_NONE;
    const int64_t R = A->size(0), K = A->size(1), E = B->size(0), N = B->size(layout ? 2 : 1);
    if (!good_gran(g, K) || (sr != g && sr != 1) || E > DG_MAX_GROUPS) Py_RETURN_NONE;
    void* pa = k.codes(a[0], (int)fa, R, K);
    void* pb = k.cube(a[1], (int)fb, kInt, E, layout ? K : N, layout ? N : K);
    void* sa = k.mat(a[2], c10::ScalarType::Float, (R + sr - 1) / sr, K / g);
    void* sb = k.cube(a[3], -1, c10::ScalarType::Float, E, (N + g - 1) / g, K / g);
    void* off;
    const int64_t no = k.indices(a[4], &off);
    void* out = k.mat(a[5], c10::ScalarType::BFloat16, R, N);
    void* pre = k.mat_or_none(a[12], c10::ScalarType::BFloat16, R, N);
    if (!k.ok || no != E + 1) Py_RETURN_NONE;
    return status(g_grouped(pa, pb, (const float*)sa, (const float*)sb, (const int32_t*)off, (int)E, out, R, N, K, (int)g, (int)layout,
                            (int)sr, (int)fa, (int)fb, (int)act, pre, k.stream()));
  });
}

// a, b, sa, sb, offsets, out, gran, fmt_a, fmt_b
PyObject* grouped_wgrad(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Call k;
    const at::Tensor* A = n == 9 ? k.first(a[0]) : nullptr;
    const at::Tensor* B = A ? k.tensor(a[1]) : nullptr;
    if (!B || B->dim() != 2) Py_RETURN_NONE;
    const int64_t g = k.integer(a[6]), fa = k.integer(a[7]), fb = k.integer(a[8]);
    const int64_t R = A->size(0), M = A->size(1), N = B->size(1);
    if (!k.ok || !good_gran(g, R) || M % g || N % g || !good_fmt(fa) || !good_fmt(fb)) Py_RETURN_NONE;
    void* pa = k.codes(a[0], (int)fa, R, M);
    void* pb = k.codes(a[1], (int)fb, R, N);
    void* sa = k.mat(a[2], c10::ScalarType::Float, R / g, M / g);
    void* sb = k.mat(a[3], c10::ScalarType::Float, R / g, N / g);
    void* off;
    const int64_t E = k.indices(a[4], &off) - 1;
    if (!k.ok || E < 1 || E > DG_MAX_GROUPS) Py_RETURN_NONE;
    void* out = k.cube(a[5], -1, c10::ScalarType::BFloat16, E, M, N);
    if (!k.ok) Py_RETURN_NONE;
    return status(g_wgrad(pa, pb, (const float*)sa, (const float*)sb, (const int32_t*)off, (int)E, out, R, M, N, (int)g, (int)fa, (int)fb,
                          k.stream()));
  });
}

// x, a, b, offsets, position, slot, scale, base, out, workspace
PyObject* lora(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Call k;
    const at::Tensor* x = n == 10 ? k.first(a[0]) : nullptr;
    const at::Tensor* at_ = x ? k.tensor(a[1]) : nullptr;
    const at::Tensor* bt = at_ ? k.tensor(a[2]) : nullptr;
    const at::Tensor* ot = bt ? k.tensor(a[8]) : nullptr;
    if (!ot || at_->dim() != 3 || bt->dim() != 3) Py_RETURN_NONE;
    const int64_t T = x->size(0), K = x->size(1), E = at_->size(0), rank = at_->size(1), N = bt->size(1);
    const auto in = k.rows(a[0], T, K);
    if (!k.ok || (in.kind != DG_IN_BF16 && in.kind != DG_IN_F16) || E > DG_MAX_GROUPS || rank > 128) Py_RETURN_NONE;
    void* pa = k.cube(a[1], -1, x->scalar_type(), E, rank, K);
    void* pb = k.cube(a[2], -1, x->scalar_type(), E, N, rank);
    void *off, *slot;
    const int64_t no = k.indices(a[3], &off);
    void* pos = k.mat(a[4], kInt, T, 1);
    const int64_t rows = k.indices(a[5], &slot);
    void* scale = k.vec_or_none(a[6], E);
    const int ok = Call::kind(ot->scalar_type());
    if (!k.ok || ok < 0 || no != E + 1 || rows != T) Py_RETURN_NONE;
    const auto base = k.rows_or_none(a[7], T, N, ok);
    void* out = k.mat(a[8], ot->scalar_type(), T, N);
    if (!k.ok) Py_RETURN_NONE;
    const int64_t need = g_lora_ws(T, K, N, (int)rank, (int)E);
    if (need < 0) Py_RETURN_NONE;
    at::Tensor ws = k.workspace(a[9], need);
    if (!k.ok) Py_RETURN_NONE;
    return status(g_lora(in.p, in.kind, in.pitch, T, K, pa, pb, (const float*)scale, N, (int)rank, (int)E, (const int32_t*)off,
                         (const int32_t*)pos, (const int32_t*)slot, base.p, base.pitch, out, ok, ws.data_ptr(), ws.numel(), k.stream()));
  });
}

// The addresses of the entry points for experts and adapters, in the order below.
PyObject* bind_route(PyObject*, PyObject* args) {
  unsigned long long p[10];
  if (!PyArg_ParseTuple(args, "KKKKKKKKKK", &p[0], &p[1], &p[2], &p[3], &p[4], &p[5], &p[6], &p[7], &p[8], &p[9])) return nullptr;
  g_sort = (decltype(g_sort))p[0];
  g_sort_ws = (decltype(g_sort_ws))p[1];
  g_rows = (decltype(g_rows))p[2];
  g_rows_ws = (decltype(g_rows_ws))p[3];
  g_combine = (decltype(g_combine))p[4];
  g_weight_grad = (decltype(g_weight_grad))p[5];
  g_grouped = (decltype(g_grouped))p[6];
  g_wgrad = (decltype(g_wgrad))p[7];
  g_lora = (decltype(g_lora))p[8];
  g_lora_ws = (decltype(g_lora_ws))p[9];
  Py_RETURN_NONE;
}

// The addresses of the library's entry points, in the order below.
PyObject* bind(PyObject*, PyObject* args) {
  unsigned long long p[7];
  if (!PyArg_ParseTuple(args, "KKKKKKK", &p[0], &p[1], &p[2], &p[3], &p[4], &p[5], &p[6])) return nullptr;
  g_norm = (decltype(g_norm))p[0];
  g_norm_bwd = (decltype(g_norm_bwd))p[1];
  g_norm_bwd_ws = (decltype(g_norm_bwd_ws))p[2];
  g_epi_bwd = (decltype(g_epi_bwd))p[3];
  g_epi_bwd_ws = (decltype(g_epi_bwd_ws))p[4];
  g_gemm = (decltype(g_gemm))p[5];
  g_gemm_ws = (decltype(g_gemm_ws))p[6];
  Py_RETURN_NONE;
}

PyMethodDef kMethods[] = {
    {"rmsnorm_quantize", (PyCFunction)(void (*)(void))rmsnorm_quantize, METH_FASTCALL, nullptr},
    {"rmsnorm_backward", (PyCFunction)(void (*)(void))rmsnorm_backward, METH_FASTCALL, nullptr},
    {"epilogue_backward", (PyCFunction)(void (*)(void))epilogue_backward, METH_FASTCALL, nullptr},
    {"gemm_residual", (PyCFunction)(void (*)(void))gemm_residual, METH_FASTCALL, nullptr},
    {"route_sort", (PyCFunction)(void (*)(void))route_sort, METH_FASTCALL, nullptr},
    {"route_quantize", (PyCFunction)(void (*)(void))route_quantize, METH_FASTCALL, nullptr},
    {"route_combine", (PyCFunction)(void (*)(void))route_combine, METH_FASTCALL, nullptr},
    {"route_weight_grad", (PyCFunction)(void (*)(void))route_weight_grad, METH_FASTCALL, nullptr},
    {"gemm_grouped", (PyCFunction)(void (*)(void))gemm_grouped, METH_FASTCALL, nullptr},
    {"grouped_wgrad", (PyCFunction)(void (*)(void))grouped_wgrad, METH_FASTCALL, nullptr},
    {"lora", (PyCFunction)(void (*)(void))lora, METH_FASTCALL, nullptr},
    {"bind", bind, METH_VARARGS, nullptr},
    {"bind_route", bind_route, METH_VARARGS, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&kModule); }

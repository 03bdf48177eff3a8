"""Block-scaled FP8 GEMM for AMD MI355X (gfx950): Python binding of libdg.so.

Argument marshalling only. Every step of the GEMM runs in the HIP kernels of
``libdg.so`` (C ABI in ``include/dg.h``); this module checks tensor dtypes,
shapes and devices, passes raw device pointers and the current HIP stream, and
turns status codes into exceptions. There is no fallback: if the library is
missing or fails to load, importing this package raises.

The operation (DeepGEMM实战 §2.2, §3.2, §4.2):
  out[i,j] = bf16( sum_kb sa[i/g,kb] * sb[j/g,kb] * sum_{k in kb} A[i,k] * B[j,k] )
with A [M,K], B [N,K] in E4M3FN or E5M2 (NT layout), FP32 scales per g x g
block (g = 64, 128 or 256) and FP32 accumulation within and across K segments.
"""

from __future__ import annotations

import ctypes
import os
import warnings

import torch  # loads the HIP runtime libdg.so binds to

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libdg.so")
# The same sources built with an extra full wait and workgroup barrier after
# every pipeline step (race check build; see load_library).
SYNC_LIB_PATH = os.path.join(_HERE, "libdg_sync.so")

DG_OK = 0
DG_EINVAL = -1
DG_EALIGN = -2
DG_EUNSUPPORTED = -3
DG_ELAUNCH = -4
DG_ESCRATCH = -5
DG_FMT_E4M3 = 0
DG_FMT_E5M2 = 1
DG_IN_F32 = 0
DG_IN_BF16 = 1
DG_IN_F16 = 2
DG_ACT_NONE = 0
DG_ACT_RELU = 1
DG_ACT_GELU = 2
DG_ACT_SILU = 3
DG_ACT_GELU_TANH = 4
DG_MAX_GROUPS = 1024  # experts or adapters of one call
DG_MAX_DIM = (1 << 24) - 256  # largest M, N or K (and quantiser rows, cols) the library accepts


class dg_tile_info(ctypes.Structure):
    _fields_ = [("kernel_id", ctypes.c_int), ("bm", ctypes.c_int), ("bn", ctypes.c_int),
                ("bk", ctypes.c_int), ("stages", ctypes.c_int), ("waves", ctypes.c_int),
                ("ksplit", ctypes.c_int), ("grid", ctypes.c_int64), ("workspace_bytes", ctypes.c_int64)]


def load_library(path: str):
    """Open a build of the C ABI at ``path`` (ctypes handle with every
    signature declared). The package itself uses libdg.so; the race check
    build libdg_sync.so is opened this way beside it (its own symbols, bound
    within itself) to compare the two builds' results."""
    if not os.path.exists(path):
        raise ImportError("%s is not built (run fp8_block_scaled_scales_amd.build.build()); "
                          "there is no non-HIP fallback" % os.path.basename(path))
    lib = ctypes.CDLL(path)
    vp, i64 = ctypes.c_void_p, ctypes.c_int64
    lib.dg_gemm_fp8_nt.restype = ctypes.c_int
    lib.dg_gemm_fp8_nt.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, ctypes.c_int, vp]
    lib.dg_query_tile.restype = ctypes.c_int
    lib.dg_query_tile.argtypes = [i64, i64, i64, ctypes.c_int, ctypes.POINTER(dg_tile_info)]
    lib.dg_gemm_fp8_nt_fmt.restype = ctypes.c_int
    lib.dg_gemm_fp8_nt_fmt.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, ctypes.c_int, ctypes.c_int, ctypes.c_int,
                                       vp]
    lib.dg_gemm_fp8_nt_epi.restype = ctypes.c_int
    lib.dg_gemm_fp8_nt_epi.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, ctypes.c_int, ctypes.c_int, ctypes.c_int,
                                       vp, ctypes.c_int, vp]
    lib.dg_gemm_fp8_nt_ex.restype = ctypes.c_int
    lib.dg_gemm_fp8_nt_ex.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, ctypes.c_int, ctypes.c_int, ctypes.c_int,
                                      ctypes.c_int, vp, ctypes.c_int, vp]
    lib.dg_gemm_fp8_layout.restype = ctypes.c_int
    lib.dg_gemm_fp8_layout.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, ctypes.c_int, ctypes.c_int, ctypes.c_int,
                                       ctypes.c_int, vp, ctypes.c_int, vp]
    lib.dg_query_tile_layout.restype = ctypes.c_int
    lib.dg_query_tile_layout.argtypes = [i64, i64, i64, ctypes.c_int, ctypes.c_int, ctypes.POINTER(dg_tile_info)]
    lib.dg_query_tile_ws.restype = ctypes.c_int
    lib.dg_query_tile_ws.argtypes = [i64, i64, i64, ctypes.c_int, ctypes.c_int, ctypes.POINTER(dg_tile_info)]
    lib.dg_gemm_fp8_ws.restype = ctypes.c_int
    lib.dg_gemm_fp8_ws.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, ctypes.c_int, ctypes.c_int, ctypes.c_int,
                                   ctypes.c_int, ctypes.c_int, vp, ctypes.c_int, vp, i64, vp]
    lib.dg_gemm_fp8_noalloc.restype = ctypes.c_int
    lib.dg_gemm_fp8_noalloc.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, ctypes.c_int, ctypes.c_int, ctypes.c_int,
                                        ctypes.c_int, ctypes.c_int, vp, ctypes.c_int, vp]
    lib.dg_noalloc_scratch_bytes.restype = ctypes.c_int64
    lib.dg_noalloc_scratch_bytes.argtypes = []
    lib.dg_quantize_fp8_rows.restype = ctypes.c_int
    lib.dg_quantize_fp8_rows.argtypes = [vp, i64, i64, ctypes.c_int, ctypes.c_int, vp, vp, vp]
    lib.dg_quantize_e4m3_blocks.restype = ctypes.c_int
    lib.dg_quantize_e4m3_blocks.argtypes = [vp, i64, i64, ctypes.c_int, vp, vp, vp]
    lib.dg_quantize_fp8_blocks.restype = ctypes.c_int
    lib.dg_quantize_fp8_blocks.argtypes = [vp, i64, i64, ctypes.c_int, ctypes.c_int, vp, vp, vp]
    for name in ("dg_quantize_fp8_blocks_typed", "dg_quantize_fp8_rows_typed"):
        fn = getattr(lib, name)
        fn.restype = ctypes.c_int
        fn.argtypes = [vp, ctypes.c_int, i64, i64, ctypes.c_int, ctypes.c_int, vp, vp, vp]
    fmt, act, kind, f32 = ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_float
    lib.dg_gemm_fp8_residual.restype = ctypes.c_int
    lib.dg_gemm_fp8_residual.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, ctypes.c_int, ctypes.c_int, ctypes.c_int,
                                         fmt, fmt, vp, act, vp, kind, i64, vp, vp, i64, vp]
    lib.dg_gemm_fp8_residual_workspace.restype = i64
    lib.dg_gemm_fp8_residual_workspace.argtypes = [i64, i64, i64, ctypes.c_int, ctypes.c_int]
    lib.dg_rmsnorm_quantize_fp8.restype = ctypes.c_int
    lib.dg_rmsnorm_quantize_fp8.argtypes = [vp, kind, i64, vp, kind, i64, vp, f32, i64, i64, ctypes.c_int, fmt, vp, vp,
                                            vp, vp, vp, vp]
    lib.dg_rmsnorm_backward.restype = ctypes.c_int
    lib.dg_rmsnorm_backward.argtypes = [vp, kind, i64, vp, kind, i64, vp, vp, vp, i64, i64, i64, vp, vp, vp, i64, vp]
    lib.dg_rmsnorm_backward_workspace.restype = i64
    lib.dg_rmsnorm_backward_workspace.argtypes = [i64, i64]
    lib.dg_epilogue_backward_fp8.restype = ctypes.c_int
    lib.dg_epilogue_backward_fp8.argtypes = [vp, kind, i64, vp, i64, act, i64, i64, ctypes.c_int, ctypes.c_int, fmt, vp,
                                             vp, vp, vp, vp, i64, vp]
    lib.dg_epilogue_backward_workspace.restype = i64
    lib.dg_epilogue_backward_workspace.argtypes = [i64, i64, ctypes.c_int, ctypes.c_int]
    i32 = ctypes.c_int
    lib.dg_route_sort.restype = i32
    lib.dg_route_sort.argtypes = [vp, i32, i64, i32, i32, i32, vp, vp, vp, i64, vp, i64, vp]
    lib.dg_route_rows.restype = i64
    lib.dg_route_rows.argtypes = [i64, i32, i32, i32]
    lib.dg_route_sort_workspace.restype = i64
    lib.dg_route_sort_workspace.argtypes = [i64, i32, i32]
    lib.dg_route_quantize_fp8.restype = i32
    lib.dg_route_quantize_fp8.argtypes = [vp, kind, i64, i64, i64, i32, vp, vp, i64, vp, i32, i32, fmt, vp, vp, vp, i64, vp]
    lib.dg_route_quantize_workspace.restype = i64
    lib.dg_route_quantize_workspace.argtypes = [i64, i64, i32, i64, i32, i32]
    lib.dg_route_combine.restype = i32
    lib.dg_route_combine.argtypes = [vp, kind, i64, i64, i64, i64, i32, vp, vp, vp, i64, vp, kind, vp]
    lib.dg_route_weight_grad.restype = i32
    lib.dg_route_weight_grad.argtypes = [vp, kind, i64, vp, kind, i64, i64, i64, i64, i32, vp, vp, vp]
    lib.dg_gemm_fp8_grouped.restype = i32
    lib.dg_gemm_fp8_grouped.argtypes = [vp, vp, vp, vp, vp, i32, vp, i64, i64, i64, i32, i32, i32, fmt, fmt, act, vp, vp]
    lib.dg_gemm_fp8_grouped_wgrad.restype = i32
    lib.dg_gemm_fp8_grouped_wgrad.argtypes = [vp, vp, vp, vp, vp, i32, vp, i64, i64, i64, i32, fmt, fmt, vp]
    lib.dg_lora.restype = i32
    lib.dg_lora.argtypes = [vp, kind, i64, i64, i64, vp, vp, vp, i64, i32, i32, vp, vp, vp, vp, i64, vp, kind, vp, i64, vp]
    lib.dg_lora_workspace.restype = i64
    lib.dg_lora_workspace.argtypes = [i64, i64, i64, i32, i32]
    lib.dg_strerror.restype = ctypes.c_char_p
    lib.dg_strerror.argtypes = [ctypes.c_int]
    lib.dg_version.restype = ctypes.c_int
    lib.dg_version.argtypes = []
    return lib


_lib = load_library(LIB_PATH)


class _NoBinding:
    """In place of a _binding that is not there: every call is left to the Python functions, which need libdg.so alone."""

    @staticmethod
    def _leave(*args):
        return None

    gemm_residual = rmsnorm_quantize = rmsnorm_backward = epilogue_backward = _leave
    route_sort = route_quantize = route_combine = route_weight_grad = gemm_grouped = grouped_wgrad = lora = _leave


try:
    from . import _binding  # the short way into the calls that serve a few tokens
except ImportError as e:
    warnings.warn("_binding.so is not built for this torch (run fp8_block_scaled_scales_amd.build.build()): calls of a few "
                  "tokens take some microseconds more (%s)" % e, RuntimeWarning)
    _binding = _NoBinding
else:
    _binding.bind(*(ctypes.cast(getattr(_lib, f), ctypes.c_void_p).value for f in (
        "dg_rmsnorm_quantize_fp8", "dg_rmsnorm_backward", "dg_rmsnorm_backward_workspace", "dg_epilogue_backward_fp8",
        "dg_epilogue_backward_workspace", "dg_gemm_fp8_residual", "dg_gemm_fp8_residual_workspace")))
    _binding.bind_route(*(ctypes.cast(getattr(_lib, f), ctypes.c_void_p).value for f in (
        "dg_route_sort", "dg_route_sort_workspace", "dg_route_quantize_fp8", "dg_route_quantize_workspace", "dg_route_combine",
        "dg_route_weight_grad", "dg_gemm_fp8_grouped", "dg_gemm_fp8_grouped_wgrad", "dg_lora", "dg_lora_workspace")))
lib = _lib  # raw ctypes handle, for tests that exercise the C ABI directly


class DGError(RuntimeError):
    def __init__(self, code: int, where: str):
        super().__init__("%s: %s (status %d)" % (where, dg_strerror(code), code))
        self.code = code


class DGArgumentError(DGError, ValueError):
    pass


def _raise(code: int, where: str):
    if code in (DG_EINVAL, DG_EALIGN):
        raise DGArgumentError(code, where)
    raise DGError(code, where)


def dg_strerror(code: int) -> str:
    return _lib.dg_strerror(int(code)).decode()


def dg_version() -> int:
    return _lib.dg_version()


def dg_query_tile(M: int, N: int, K: int, gran: int = 128, layout: int = 0, workspace: bool = False) -> dict:
    """The tile-table plan of a call: dg_gemm_fp8_layout's (workspace=False) or dg_gemm_fp8_ws's."""
    info = dg_tile_info()
    fn = _lib.dg_query_tile_ws if workspace else _lib.dg_query_tile_layout
    rc = fn(M, N, K, gran, layout, ctypes.byref(info))
    if rc != DG_OK:
        _raise(rc, "dg_query_tile")
    return {name: getattr(info, name) for name, _ in dg_tile_info._fields_}


_FP8 = (torch.float8_e4m3fn, torch.uint8)
_FP8_OF = {DG_FMT_E4M3: (torch.float8_e4m3fn, torch.uint8), DG_FMT_E5M2: (torch.float8_e5m2, torch.uint8)}
_GRANS = (64, 128, 256)
_IN_OF = {torch.float32: DG_IN_F32, torch.bfloat16: DG_IN_BF16, torch.float16: DG_IN_F16}


def _check(t, name, dtypes, shape, device):
    # one expression for a tensor that is right; what is wrong is found and named only then
    if (isinstance(t, torch.Tensor) and t.dtype in dtypes and t.shape == shape and t.is_contiguous() and
            t.device == device):
        return
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if t.dtype not in dtypes:
        raise ValueError("%s has dtype %s, expected one of %s" % (name, t.dtype, dtypes))
    if tuple(t.shape) != tuple(shape):
        raise ValueError("%s has shape %s, expected %s" % (name, tuple(t.shape), tuple(shape)))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    if t.device != device:
        raise ValueError("%s is on %s, expected %s" % (name, t.device, device))


def _gemm(a, b, sa, sb, out, gran, fmt_a, fmt_b, stream, where, bias=None, act=DG_ACT_NONE, sa_rows=None):
    if a.dim() != 2 or b.dim() != 2:
        raise ValueError("a and b must be 2-D")
    M, K = a.shape
    N = b.shape[0]
    dev = a.device
    if gran not in _GRANS or K % gran:
        raise ValueError("gran must be 64, 128 or 256 and divide K")
    if fmt_a not in _FP8_OF or fmt_b not in _FP8_OF:
        raise ValueError("formats must be DG_FMT_E4M3 or DG_FMT_E5M2")
    sa_rows = gran if sa_rows is None else sa_rows
    if sa_rows not in (gran, 1):
        raise ValueError("sa_rows must be gran (g x g blocks) or 1 (per-row factors)")
    _check(a, "a", _FP8_OF[fmt_a], (M, K), dev)
    _check(b, "b", _FP8_OF[fmt_b], (N, K), dev)
    _check(sa, "sa", (torch.float32,), ((M + sa_rows - 1) // sa_rows, K // gran), dev)
    _check(sb, "sb", (torch.float32,), ((N + gran - 1) // gran, K // gran), dev)
    if out is None:
        out = torch.empty((M, N), dtype=torch.bfloat16, device=dev)
    _check(out, "out", (torch.bfloat16,), (M, N), dev)
    if bias is not None:
        _check(bias, "bias", (torch.float32,), (N,), dev)
    if act not in (DG_ACT_NONE, DG_ACT_RELU, DG_ACT_GELU):
        raise ValueError("act must be DG_ACT_NONE, DG_ACT_RELU or DG_ACT_GELU")
    if dev.type != "cuda":
        raise ValueError("a must be a GPU tensor")
    s = stream if stream is not None else torch.cuda.current_stream(dev)
    with torch.cuda.device(dev):
        if where == "dg_gemm_fp8_nt_ex":
            rc = _lib.dg_gemm_fp8_nt_ex(a.data_ptr(), b.data_ptr(), sa.data_ptr(), sb.data_ptr(), out.data_ptr(),
                                        M, N, K, gran, sa_rows, fmt_a, fmt_b,
                                        None if bias is None else bias.data_ptr(), act, s.cuda_stream)
        elif where == "dg_gemm_fp8_nt_epi":
            rc = _lib.dg_gemm_fp8_nt_epi(a.data_ptr(), b.data_ptr(), sa.data_ptr(), sb.data_ptr(), out.data_ptr(),
                                         M, N, K, gran, fmt_a, fmt_b, None if bias is None else bias.data_ptr(),
                                         act, s.cuda_stream)
        elif fmt_a == DG_FMT_E4M3 and fmt_b == DG_FMT_E4M3 and where == "dg_gemm_fp8_nt":
            rc = _lib.dg_gemm_fp8_nt(a.data_ptr(), b.data_ptr(), sa.data_ptr(), sb.data_ptr(), out.data_ptr(),
                                     M, N, K, gran, s.cuda_stream)
        else:
            rc = _lib.dg_gemm_fp8_nt_fmt(a.data_ptr(), b.data_ptr(), sa.data_ptr(), sb.data_ptr(), out.data_ptr(),
                                         M, N, K, gran, fmt_a, fmt_b, s.cuda_stream)
    if rc != DG_OK:
        _raise(rc, where)
    return out


def dg_gemm_fp8_nt(a, b, sa, sb, out=None, gran: int = 128, stream=None):
    """out[M,N] (bf16) = A[M,K] * B[N,K]^T with gran x gran FP32 block scales.

    a: [M,K] float8_e4m3fn (or uint8 holding E4M3FN codes), b: [N,K] likewise,
    sa: [ceil(M/gran), K/gran] float32, sb: [ceil(N/gran), K/gran] float32,
    gran 64, 128 or 256, out: optional preallocated [M,N] bfloat16 (allocated
    when None). Enqueued on ``stream`` (a torch.cuda.Stream; default: the
    current stream).
    """
    return _gemm(a, b, sa, sb, out, gran, DG_FMT_E4M3, DG_FMT_E4M3, stream, "dg_gemm_fp8_nt")


def dg_gemm_fp8_nt_fmt(a, b, sa, sb, out=None, gran: int = 128, fmt_a: int = DG_FMT_E4M3,
                       fmt_b: int = DG_FMT_E4M3, stream=None):
    """dg_gemm_fp8_nt with each operand's FP8 format given (DG_FMT_E4M3 / DG_FMT_E5M2).

    An E5M2 operand is float8_e5m2 (or uint8 holding E5M2 codes).
    """
    return _gemm(a, b, sa, sb, out, gran, fmt_a, fmt_b, stream, "dg_gemm_fp8_nt_fmt")


def dg_gemm_fp8_nt_epi(a, b, sa, sb, out=None, gran: int = 128, fmt_a: int = DG_FMT_E4M3,
                       fmt_b: int = DG_FMT_E4M3, bias=None, act: int = DG_ACT_NONE, stream=None):
    """dg_gemm_fp8_nt_fmt with out = bf16(act(C + bias[None, :])) fused into the store.

    bias: optional [N] float32; act: DG_ACT_NONE, DG_ACT_RELU or DG_ACT_GELU (exact erf form).
    """
    return _gemm(a, b, sa, sb, out, gran, fmt_a, fmt_b, stream, "dg_gemm_fp8_nt_epi", bias, act)


def dg_gemm_fp8_nt_ex(a, b, sa, sb, out=None, gran: int = 128, sa_rows: int | None = None,
                      fmt_a: int = DG_FMT_E4M3, fmt_b: int = DG_FMT_E4M3, bias=None, act: int = DG_ACT_NONE,
                      stream=None):
    """dg_gemm_fp8_nt_epi with A's factor blocks chosen: sa_rows = gran (g x g, the default) or 1.

    With sa_rows = 1, sa is [M, K/gran] float32: one factor per row of A and K
    segment (per-row A scales); B keeps its g x g blocks.
    """
    return _gemm(a, b, sa, sb, out, gran, fmt_a, fmt_b, stream, "dg_gemm_fp8_nt_ex", bias, act, sa_rows)


# Operand layouts: bit 1 = A stored [K, M], bit 0 = B stored [K, N].
DG_LAYOUT_NT, DG_LAYOUT_NN, DG_LAYOUT_TT, DG_LAYOUT_TN = 0, 1, 2, 3


def dg_gemm_fp8_layout(a, b, sa, sb, out=None, gran: int = 128, layout: int = DG_LAYOUT_NT,
                       fmt_a: int = DG_FMT_E4M3, fmt_b: int = DG_FMT_E4M3, bias=None, act: int = DG_ACT_NONE,
                       stream=None):
    """dg_gemm_fp8_nt_epi with A stored [M,K] or [K,M] and B stored [N,K] or [K,N] per ``layout``.

    a: [M,K] (NT, NN) or [K,M] (TT, TN); b: [N,K] (NT, TT) or [K,N] (NN, TN); sa and
    sb keep their logical shapes [ceil(M/g), K/g] and [ceil(N/g), K/g]. M and N may
    be any length (ragged edges included) in every layout. Per-row A factors with
    a layout: dg_gemm_fp8_ws (workspace=None) takes both.
    """
    if layout not in (DG_LAYOUT_NT, DG_LAYOUT_NN, DG_LAYOUT_TT, DG_LAYOUT_TN):
        raise ValueError("layout must be DG_LAYOUT_NT, _NN, _TT or _TN")
    if a.dim() != 2 or b.dim() != 2:
        raise ValueError("a and b must be 2-D")
    K, M = a.shape if layout & 2 else a.shape[::-1]
    N = b.shape[1] if layout & 1 else b.shape[0]
    dev = a.device
    if gran not in _GRANS or K % gran:
        raise ValueError("gran must be 64, 128 or 256 and divide K")
    if fmt_a not in _FP8_OF or fmt_b not in _FP8_OF:
        raise ValueError("formats must be DG_FMT_E4M3 or DG_FMT_E5M2")
    _check(a, "a", _FP8_OF[fmt_a], (K, M) if layout & 2 else (M, K), dev)
    _check(b, "b", _FP8_OF[fmt_b], (K, N) if layout & 1 else (N, K), dev)
    _check(sa, "sa", (torch.float32,), ((M + gran - 1) // gran, K // gran), dev)
    _check(sb, "sb", (torch.float32,), ((N + gran - 1) // gran, K // gran), dev)
    if out is None:
        out = torch.empty((M, N), dtype=torch.bfloat16, device=dev)
    _check(out, "out", (torch.bfloat16,), (M, N), dev)
    if bias is not None:
        _check(bias, "bias", (torch.float32,), (N,), dev)
    if act not in (DG_ACT_NONE, DG_ACT_RELU, DG_ACT_GELU):
        raise ValueError("act must be DG_ACT_NONE, DG_ACT_RELU or DG_ACT_GELU")
    if dev.type != "cuda":
        raise ValueError("a must be a GPU tensor")
    s = stream if stream is not None else torch.cuda.current_stream(dev)
    with torch.cuda.device(dev):
        rc = _lib.dg_gemm_fp8_layout(a.data_ptr(), b.data_ptr(), sa.data_ptr(), sb.data_ptr(), out.data_ptr(),
                                     M, N, K, gran, layout, fmt_a, fmt_b, None if bias is None else bias.data_ptr(),
                                     act, s.cuda_stream)
    if rc != DG_OK:
        _raise(rc, "dg_gemm_fp8_layout")
    return out


def dg_workspace(M: int, N: int, K: int, gran: int = 128, layout: int = DG_LAYOUT_NT, device="cuda"):
    """A workspace for dg_gemm_fp8_ws of this shape (uint8 tensor), or None when its plan needs none."""
    n = dg_query_tile(M, N, K, gran, layout, workspace=True)["workspace_bytes"]
    return torch.empty(n, dtype=torch.uint8, device=device) if n else None


def _ws_args(a, b, sa, sb, out, gran, layout, sa_rows, fmt_a, fmt_b, bias, act, more=None):
    """Checks shared by the calls that take a layout with sa_rows; returns (M, N, K, sa_rows, dev).
    more(M, N, dev): a call's further checks."""
    if layout not in (DG_LAYOUT_NT, DG_LAYOUT_NN, DG_LAYOUT_TT, DG_LAYOUT_TN):
        raise ValueError("layout must be DG_LAYOUT_NT, _NN, _TT or _TN")
    if a.dim() != 2 or b.dim() != 2:
        raise ValueError("a and b must be 2-D")
    K, M = a.shape if layout & 2 else a.shape[::-1]
    N = b.shape[1] if layout & 1 else b.shape[0]
    dev = a.device
    if gran not in _GRANS or K % gran:
        raise ValueError("gran must be 64, 128 or 256 and divide K")
    if fmt_a not in _FP8_OF or fmt_b not in _FP8_OF:
        raise ValueError("formats must be DG_FMT_E4M3 or DG_FMT_E5M2")
    sa_rows = gran if sa_rows is None else sa_rows
    if sa_rows not in (gran, 1):
        raise ValueError("sa_rows must be gran (g x g blocks) or 1 (per-row factors)")
    _check(a, "a", _FP8_OF[fmt_a], (K, M) if layout & 2 else (M, K), dev)
    _check(b, "b", _FP8_OF[fmt_b], (K, N) if layout & 1 else (N, K), dev)
    _check(sa, "sa", (torch.float32,), ((M + sa_rows - 1) // sa_rows, K // gran), dev)
    _check(sb, "sb", (torch.float32,), ((N + gran - 1) // gran, K // gran), dev)
    if out is not None:
        _check(out, "out", (torch.bfloat16,), (M, N), dev)
    if bias is not None:
        _check(bias, "bias", (torch.float32,), (N,), dev)
    if act not in (DG_ACT_NONE, DG_ACT_RELU, DG_ACT_GELU):
        raise ValueError("act must be DG_ACT_NONE, DG_ACT_RELU or DG_ACT_GELU")
    if more is not None:
        more(M, N, dev)
    if dev.type != "cuda":
        raise ValueError("a must be a GPU tensor")
    return M, N, K, sa_rows, dev


def dg_gemm_fp8_ws(a, b, sa, sb, out=None, gran: int = 128, layout: int = DG_LAYOUT_NT, sa_rows: int | None = None,
                   fmt_a: int = DG_FMT_E4M3, fmt_b: int = DG_FMT_E4M3, bias=None, act: int = DG_ACT_NONE,
                   workspace=None, stream=None):
    """dg_gemm_fp8_layout (with dg_gemm_fp8_nt_ex's sa_rows) plus a caller-owned workspace.

    With a workspace (a contiguous uint8 GPU tensor of at least
    dg_query_tile(..., workspace=True)["workspace_bytes"] bytes, 256-byte
    aligned; see ``dg_workspace``) shapes with few output tiles and a long K
    (16384 and up, cut at least 8 ways) split K over several
    workgroups; every other shape runs what the call without a workspace
    runs. Concurrent calls need distinct workspaces.
    """
    M, N, K, sa_rows, dev = _ws_args(a, b, sa, sb, out, gran, layout, sa_rows, fmt_a, fmt_b, bias, act)
    if out is None:
        out = torch.empty((M, N), dtype=torch.bfloat16, device=dev)
    ws_ptr, ws_bytes = None, 0
    if workspace is not None:
        _check(workspace, "workspace", (torch.uint8,), (workspace.numel(),), dev)
        ws_ptr, ws_bytes = workspace.data_ptr(), workspace.numel()
    s = stream if stream is not None else torch.cuda.current_stream(dev)
    with torch.cuda.device(dev):
        rc = _lib.dg_gemm_fp8_ws(a.data_ptr(), b.data_ptr(), sa.data_ptr(), sb.data_ptr(), out.data_ptr(),
                                 M, N, K, gran, layout, sa_rows, fmt_a, fmt_b,
                                 None if bias is None else bias.data_ptr(), act, ws_ptr, ws_bytes, s.cuda_stream)
    if rc != DG_OK:
        _raise(rc, "dg_gemm_fp8_ws")
    return out


def dg_gemm_fp8_noalloc(a, b, sa, sb, out, gran: int = 128, layout: int = DG_LAYOUT_NT, sa_rows: int | None = None,
                        fmt_a: int = DG_FMT_E4M3, fmt_b: int = DG_FMT_E4M3, bias=None, act: int = DG_ACT_NONE,
                        stream=None):
    """dg_gemm_fp8_ws with the library's fixed scratch array as the workspace: nothing is allocated.

    ``out`` must be given (this wrapper allocates nothing either). Calls that
    may overlap in time on one GPU race on the shared scratch; a plan that
    needs more than dg_noalloc_scratch_bytes() raises (DG_ESCRATCH).
    """
    if out is None:
        raise ValueError("dg_gemm_fp8_noalloc needs a preallocated out")
    M, N, K, sa_rows, dev = _ws_args(a, b, sa, sb, out, gran, layout, sa_rows, fmt_a, fmt_b, bias, act)
    s = stream if stream is not None else torch.cuda.current_stream(dev)
    with torch.cuda.device(dev):
        rc = _lib.dg_gemm_fp8_noalloc(a.data_ptr(), b.data_ptr(), sa.data_ptr(), sb.data_ptr(), out.data_ptr(),
                                      M, N, K, gran, layout, sa_rows, fmt_a, fmt_b,
                                      None if bias is None else bias.data_ptr(), act, s.cuda_stream)
    if rc != DG_OK:
        _raise(rc, "dg_gemm_fp8_noalloc")
    return out


def dg_noalloc_scratch_bytes() -> int:
    return _lib.dg_noalloc_scratch_bytes()


def _quantize(x, gran, fmt, q, scales, stream, where):
    if not isinstance(x, torch.Tensor) or x.dim() != 2:
        raise ValueError("x must be a 2-D tensor")
    rows, cols = x.shape
    dev = x.device
    if dev.type != "cuda":
        raise ValueError("x must be a GPU tensor")
    if gran not in _GRANS or cols % gran:
        raise ValueError("gran must be 64, 128 or 256 and divide cols")
    if fmt not in _FP8_OF:
        raise ValueError("fmt must be DG_FMT_E4M3 or DG_FMT_E5M2")
    typed = where.endswith("_typed")
    _check(x, "x", tuple(_IN_OF) if typed else (torch.float32,), (rows, cols), dev)
    if q is None:
        q = torch.empty((rows, cols), dtype=torch.uint8, device=dev)
    brows = 1 if where.startswith("dg_quantize_fp8_rows") else gran  # rows per block
    if scales is None:
        scales = torch.empty(((rows + brows - 1) // brows, cols // gran), dtype=torch.float32, device=dev)
    _check(q, "q", _FP8_OF[fmt], (rows, cols), dev)
    _check(scales, "scales", (torch.float32,), ((rows + brows - 1) // brows, cols // gran), dev)
    s = stream if stream is not None else torch.cuda.current_stream(dev)
    with torch.cuda.device(dev):
        if typed:
            rc = getattr(_lib, where)(x.data_ptr(), _IN_OF[x.dtype], rows, cols, gran, fmt, q.data_ptr(),
                                      scales.data_ptr(), s.cuda_stream)
        elif where == "dg_quantize_fp8_rows":
            rc = _lib.dg_quantize_fp8_rows(x.data_ptr(), rows, cols, gran, fmt, q.data_ptr(), scales.data_ptr(),
                                           s.cuda_stream)
        elif fmt == DG_FMT_E4M3 and where == "dg_quantize_e4m3_blocks":
            rc = _lib.dg_quantize_e4m3_blocks(x.data_ptr(), rows, cols, gran, q.data_ptr(), scales.data_ptr(),
                                              s.cuda_stream)
        else:
            rc = _lib.dg_quantize_fp8_blocks(x.data_ptr(), rows, cols, gran, fmt, q.data_ptr(), scales.data_ptr(),
                                             s.cuda_stream)
    if rc != DG_OK:
        _raise(rc, where)
    return q, scales


def dg_quantize_e4m3_blocks(x, gran: int = 128, q=None, scales=None, stream=None):
    """Block-quantise x [rows, cols] float32 on the GPU -> (q uint8 [rows, cols], scales float32).

    Per gran x gran block (gran 64, 128 or 256): scale = amax / 448 (1.0 for
    an all-zero block) and q = E4M3FN(x / scale), round to nearest even.
    ``scales`` has shape [ceil(rows/gran), cols/gran]. The codes come back as
    uint8 holding E4M3FN bytes (``q.view(torch.float8_e4m3fn)`` reinterprets
    them).
    """
    return _quantize(x, gran, DG_FMT_E4M3, q, scales, stream, "dg_quantize_e4m3_blocks")


def dg_quantize_fp8_blocks(x, gran: int = 128, fmt: int = DG_FMT_E4M3, q=None, scales=None, stream=None):
    """dg_quantize_e4m3_blocks for either format; E5M2 uses scale = amax / 57344."""
    return _quantize(x, gran, fmt, q, scales, stream, "dg_quantize_fp8_blocks")


def dg_quantize_fp8_rows(x, gran: int = 128, fmt: int = DG_FMT_E4M3, q=None, scales=None, stream=None):
    """1 x gran quantisation on the GPU: one factor per row and gran-wide segment, scales [rows, cols/gran]."""
    return _quantize(x, gran, fmt, q, scales, stream, "dg_quantize_fp8_rows")


def dg_quantize_fp8_blocks_typed(x, gran: int = 128, fmt: int = DG_FMT_E4M3, q=None, scales=None, stream=None):
    """dg_quantize_fp8_blocks on float32, bfloat16 or float16 x (the input kind is x's dtype).

    Each element is widened exactly to FP32 first, so a 16-bit x and its FP32
    copy give identical codes and scales.
    """
    return _quantize(x, gran, fmt, q, scales, stream, "dg_quantize_fp8_blocks_typed")


def dg_quantize_fp8_rows_typed(x, gran: int = 128, fmt: int = DG_FMT_E4M3, q=None, scales=None, stream=None):
    """dg_quantize_fp8_rows on float32, bfloat16 or float16 x (the input kind is x's dtype)."""
    return _quantize(x, gran, fmt, q, scales, stream, "dg_quantize_fp8_rows_typed")


# ---- the operators around the product in a transformer layer ----------------

_F32 = (torch.float32,)
_BF16 = (torch.bfloat16,)

# The calls below take a few microseconds on the GPU for a few tokens. Where
# every tensor is given and right, _binding checks and launches them; the code
# here does the rest: it allocates what is not given, takes a given stream and
# names what is wrong. The current stream's and device's raw forms cost 0.06 and
# 0.09 us, the public objects 1.7 and 0.2 us.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)
_raw_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _rows(t, name, dtypes, shape, dev):
    """Checks an input matrix whose rows may lie apart (a slice of a wider one); its row pitch in elements."""
    if isinstance(t, torch.Tensor) and t.dtype in dtypes and t.shape == shape and t.device == dev:
        if t.is_contiguous():
            return shape[1]
        pitch, step = t.stride()
        if (step != 1 and shape[1] > 1) or (pitch < shape[1] and shape[0] > 1):
            raise ValueError("%s must have contiguous rows that do not overlap" % name)
        return pitch if shape[0] > 1 else shape[1]
    _check(t, name, dtypes, shape, dev)  # raises: it asks for no less
    raise ValueError("%s is not what the call takes" % name)


def _out(t, name, dtypes, shape, dev, stream):
    """Checks an output, or allocates it on the call's stream."""
    if t is not None:
        _check(t, name, dtypes, shape, dev)
        return t
    if stream is None:
        return torch.empty(shape, dtype=dtypes[-1], device=dev)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtypes[-1], device=dev)


def _workspace(t, nbytes, dev, stream):
    """The workspace of a call that needs nbytes: the caller's, or one from torch's allocator on the call's stream."""
    if t is None:
        return _out(None, "workspace", (torch.uint8,), (nbytes,), dev, stream)
    _check(t, "workspace", (torch.uint8,), (t.numel(),), dev)
    return t


def _launch(fn, where, dev, stream, *args):
    """Calls fn(*args, stream) with dev current; a status other than DG_OK raises."""
    if dev.type != "cuda":
        raise ValueError("%s needs GPU tensors" % where)
    s = _raw_stream(dev.index) if stream is None else stream.cuda_stream
    if _raw_device() == dev.index:
        rc = fn(*args, s)
    else:
        with torch.cuda.device(dev):
            rc = fn(*args, s)
    if rc:
        _raise(rc, where)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _matrix(t, name):
    if not isinstance(t, torch.Tensor) or t.dim() != 2:
        raise ValueError("%s must be a 2-D tensor" % name)
    return t.shape


def dg_gemm_fp8_residual(a, b, sa, sb, res=None, out=None, gran: int = 128, layout: int = DG_LAYOUT_NT,
                         sa_rows: int | None = None, fmt_a: int = DG_FMT_E4M3, fmt_b: int = DG_FMT_E4M3, bias=None,
                         act: int = DG_ACT_NONE, pre=None, workspace=None, stream=None):
    """out = bf16(act(C + bias) + res), the product with a residual and any activation in its epilogue.

    a, b, sa, sb, gran, layout, sa_rows, formats and bias as dg_gemm_fp8_ws. res: [M,N]
    float32, bfloat16 or float16, rows contiguous (any pitch), or None; it may be out
    itself. act: one of the five DG_ACT_* codes. pre: optional [M,N] bfloat16 that
    receives C + bias, for dg_epilogue_backward_fp8. workspace: a uint8 tensor of
    dg_gemm_fp8_residual_workspace(...) bytes, with which few output tiles and a long K
    are split over workgroups: allocated when None, where dg_gemm_fp8_ws does not split;
    an empty tensor declines the split, so that a row's sums do not depend on the number
    of output tiles through it.
    """
    if stream is None:
        rc = _binding.gemm_residual(a, b, sa, sb, res, out, gran, layout, gran if sa_rows is None else sa_rows, fmt_a, fmt_b, bias,
                                    act, pre, workspace)
        if rc is not None:
            if rc:
                _raise(rc, "dg_gemm_fp8_residual")
            return out
    if act not in (DG_ACT_NONE, DG_ACT_RELU, DG_ACT_GELU, DG_ACT_SILU, DG_ACT_GELU_TANH):
        raise ValueError("act must be one of the DG_ACT_* codes")
    kind, pitch = 0, 0

    def more(M, N, dev):
        nonlocal kind, pitch
        if res is not None:
            pitch = _rows(res, "res", _IN_OF, (M, N), dev)
            kind = _IN_OF[res.dtype]
        if pre is not None:
            _check(pre, "pre", _BF16, (M, N), dev)

    M, N, K, sa_rows, dev = _ws_args(a, b, sa, sb, out, gran, layout, sa_rows, fmt_a, fmt_b, bias, DG_ACT_NONE, more)
    if out is None:
        out = _out(None, "out", _BF16, (M, N), dev, stream)
    need = _lib.dg_gemm_fp8_residual_workspace(M, N, K, gran, layout)
    ws = _workspace(workspace, need, dev, stream) if need > 0 else None
    _launch(_lib.dg_gemm_fp8_residual, "dg_gemm_fp8_residual", dev, stream, a.data_ptr(), b.data_ptr(), sa.data_ptr(),
            sb.data_ptr(), out.data_ptr(), M, N, K, gran, layout, sa_rows, fmt_a, fmt_b, _ptr(bias), act, _ptr(res),
            kind, pitch, _ptr(pre), _ptr(ws), ws.numel() if need > 0 else 0)
    return out


def dg_gemm_fp8_residual_workspace(M: int, N: int, K: int, gran: int = 128, layout: int = DG_LAYOUT_NT) -> int:
    """Workspace bytes with which dg_gemm_fp8_residual splits K (0 where it does not)."""
    n = _lib.dg_gemm_fp8_residual_workspace(M, N, K, gran, layout)
    if n < 0:
        _raise(n, "dg_gemm_fp8_residual_workspace")
    return n


def dg_rmsnorm_quantize_fp8(x, res, weight, eps: float = 1e-6, gran: int = 128, fmt: int = DG_FMT_E4M3, h=None, y=None,
                            rstd=None, q=None, scales=None, stream=None):
    """(q, scales, h): h = x + res, its RMS norm times weight, quantised with one factor per row and gran-wide segment.

    x: [rows, cols] float32, bfloat16 or float16; res: the residual stream, likewise
    (either may have a row pitch), or None, and then h is x. weight: [cols] float32.
    h: optional output of res's dtype (may be res). y (x's dtype) and rstd ([rows]
    float32), where given, receive the normed values and 1 / rms, which
    dg_rmsnorm_backward and the weight gradient's product need. q (uint8 holding fmt's
    codes, or that float8 dtype) and scales [rows, cols/gran] are what
    dg_gemm_fp8_residual takes as a and sa with sa_rows = 1.
    """
    if stream is None:
        rc = _binding.rmsnorm_quantize(x, res, weight, eps, gran, fmt, h, y, rstd, q, scales)
        if rc is not None:
            if rc:
                _raise(rc, "dg_rmsnorm_quantize_fp8")
            return q, scales, x if res is None else h
    rows, cols = shape = _matrix(x, "x")
    dev = x.device
    if gran not in _GRANS or cols % gran:
        raise ValueError("gran must be 64, 128 or 256 and divide cols")
    if fmt not in _FP8_OF:
        raise ValueError("fmt must be DG_FMT_E4M3 or DG_FMT_E5M2")
    ldx = _rows(x, "x", _IN_OF, shape, dev)
    _check(weight, "weight", _F32, (cols,), dev)
    rk, ldres = 0, 0
    if res is not None:
        ldres = _rows(res, "res", _IN_OF, shape, dev)
        rk = _IN_OF[res.dtype]
        h = _out(h, "h", (res.dtype,), shape, dev, stream)
    elif h is not None:
        raise ValueError("h is written only where there is a residual")
    if y is not None:
        _check(y, "y", (x.dtype,), shape, dev)
    if rstd is not None:
        _check(rstd, "rstd", _F32, (rows,), dev)
    q = _out(q, "q", _FP8_OF[fmt], shape, dev, stream)
    scales = _out(scales, "scales", _F32, (rows, cols // gran), dev, stream)
    _launch(_lib.dg_rmsnorm_quantize_fp8, "dg_rmsnorm_quantize_fp8", dev, stream, x.data_ptr(), _IN_OF[x.dtype], ldx,
            _ptr(res), rk, ldres, weight.data_ptr(), eps, rows, cols, gran, fmt, _ptr(h), _ptr(y), _ptr(rstd),
            q.data_ptr(), scales.data_ptr())
    return q, scales, x if res is None else h


def dg_rmsnorm_backward(dy, h, rstd, weight, dh=None, dx=None, dweight=None, workspace=None, stream=None):
    """(dx, dweight): the gradient of dg_rmsnorm_quantize_fp8's norm, from dy, the gradient of y.

    h, rstd, weight: as the forward pass left them. dh: the gradient that reaches the
    stream h past the norm (h's dtype), added to dx; dx may be dh. dx is the gradient
    of x and of the residual alike, of h's dtype; dweight is [cols] float32. workspace:
    a uint8 tensor of dg_rmsnorm_backward_workspace(rows, cols) bytes (allocated when None).
    """
    if stream is None:
        rc = _binding.rmsnorm_backward(dy, h, rstd, weight, dh, dx, dweight, workspace)
        if rc is not None:
            if rc:
                _raise(rc, "dg_rmsnorm_backward")
            return dx, dweight
    rows, cols = shape = _matrix(dy, "dy")
    dev = dy.device
    if cols % 64 or not rows or not cols:
        raise ValueError("dy must have rows, and columns in a multiple of 64")
    lddy = _rows(dy, "dy", _IN_OF, shape, dev)
    ldh = _rows(h, "h", _IN_OF, shape, dev)
    _check(rstd, "rstd", _F32, (rows,), dev)
    _check(weight, "weight", _F32, (cols,), dev)
    lddh = 0 if dh is None else _rows(dh, "dh", (h.dtype,), shape, dev)
    dx = _out(dx, "dx", (h.dtype,), shape, dev, stream)
    dweight = _out(dweight, "dweight", _F32, (cols,), dev, stream)
    need = _lib.dg_rmsnorm_backward_workspace(rows, cols)
    ws = _workspace(workspace, need, dev, stream) if need > 0 else None
    _launch(_lib.dg_rmsnorm_backward, "dg_rmsnorm_backward", dev, stream, dy.data_ptr(), _IN_OF[dy.dtype], lddy,
            h.data_ptr(), _IN_OF[h.dtype], ldh, rstd.data_ptr(), weight.data_ptr(), _ptr(dh), lddh, rows, cols,
            dx.data_ptr(), dweight.data_ptr(), _ptr(ws), ws.numel() if need > 0 else 0)
    return dx, dweight


def dg_rmsnorm_backward_workspace(rows: int, cols: int) -> int:
    """Workspace bytes of dg_rmsnorm_backward."""
    n = _lib.dg_rmsnorm_backward_workspace(rows, cols)
    if n < 0:
        _raise(n, "dg_rmsnorm_backward_workspace")
    return n


def dg_epilogue_backward_fp8(dout, pre, act: int, gran: int = 128, block_rows: int | None = None,
                             fmt: int = DG_FMT_E5M2, dz=None, dbias=None, q=None, scales=None, workspace=None,
                             stream=None):
    """(q, scales): dz = dout * act'(pre) as FP8 codes with factors, the gradient through the product's epilogue.

    dout: [rows, cols] float32, bfloat16 or float16; pre: the bfloat16 pre-activation
    dg_gemm_fp8_residual kept (None with DG_ACT_NONE). block_rows: gran (gran x gran
    blocks, the default: the codes serve both following products) or 1 (a factor per
    row and segment). dz (dout's dtype; may be dout) and dbias ([cols] float32), where
    given, receive the FP32 gradient rounded once and its sum over the rows.
    workspace: a uint8 tensor of dg_epilogue_backward_workspace(...) bytes (allocated when None).
    """
    block_rows = gran if block_rows is None else block_rows
    if stream is None:
        rc = _binding.epilogue_backward(dout, pre, act, gran, block_rows, fmt, dz, dbias, q, scales, workspace)
        if rc is not None:
            if rc:
                _raise(rc, "dg_epilogue_backward_fp8")
            return q, scales
    rows, cols = shape = _matrix(dout, "dout")
    dev = dout.device
    if gran not in _GRANS or cols % gran or not rows or not cols:
        raise ValueError("dout must have rows and columns, and gran must be 64, 128 or 256 and divide cols")
    if fmt not in _FP8_OF:
        raise ValueError("fmt must be DG_FMT_E4M3 or DG_FMT_E5M2")
    if block_rows not in (gran, 1):
        raise ValueError("block_rows must be gran (g x g blocks) or 1 (per-row factors)")
    if act not in (DG_ACT_NONE, DG_ACT_RELU, DG_ACT_GELU, DG_ACT_SILU, DG_ACT_GELU_TANH):
        raise ValueError("act must be one of the DG_ACT_* codes")
    if (act == DG_ACT_NONE) != (pre is None):
        raise ValueError("pre goes with an activation, and only with one")
    lddout = _rows(dout, "dout", _IN_OF, shape, dev)
    ldpre = 0 if pre is None else _rows(pre, "pre", _BF16, shape, dev)
    if dz is not None:
        _check(dz, "dz", (dout.dtype,), shape, dev)
    need = 0
    if dbias is not None:
        _check(dbias, "dbias", _F32, (cols,), dev)
        need = _lib.dg_epilogue_backward_workspace(rows, cols, gran, block_rows)
    q = _out(q, "q", _FP8_OF[fmt], shape, dev, stream)
    scales = _out(scales, "scales", _F32, ((rows + block_rows - 1) // block_rows, cols // gran), dev, stream)
    ws = _workspace(workspace, need, dev, stream) if need > 0 else None
    _launch(_lib.dg_epilogue_backward_fp8, "dg_epilogue_backward_fp8", dev, stream, dout.data_ptr(),
            _IN_OF[dout.dtype], lddout, _ptr(pre), ldpre, act, rows, cols, gran, block_rows, fmt, _ptr(dz), _ptr(dbias),
            q.data_ptr(), scales.data_ptr(), _ptr(ws), ws.numel() if need > 0 else 0)
    return q, scales


def dg_epilogue_backward_workspace(rows: int, cols: int, gran: int = 128, block_rows: int | None = None) -> int:
    """Workspace bytes of dg_epilogue_backward_fp8 with dbias."""
    n = _lib.dg_epilogue_backward_workspace(rows, cols, gran, gran if block_rows is None else block_rows)
    if n < 0:
        _raise(n, "dg_epilogue_backward_workspace")
    return n


# ---- layers whose weights each row chooses: experts and adapters ------------

_I32 = (torch.int32,)
_ID_BYTES = {torch.int32: 4, torch.int64: 8}
_ACTS = (DG_ACT_NONE, DG_ACT_RELU, DG_ACT_GELU, DG_ACT_SILU, DG_ACT_GELU_TANH)


def _count(n, name):
    """A size the library computed, or the error it answered with."""
    if n < 0:
        _raise(n, name)
    return n


def _sizes(name, *sizes):
    """Refuses sizes that no call takes: ctypes would hand the library what is left of them in a C integer."""
    if any(n < 0 or n > DG_MAX_DIM for n in sizes):
        _raise(DG_EINVAL, name)


def _groups(offsets, dev):
    """The number of groups that an offsets array is for."""
    if not isinstance(offsets, torch.Tensor) or offsets.dim() != 1 or not 2 <= offsets.shape[0] <= DG_MAX_GROUPS + 1:
        raise ValueError("offsets must be a 1-D tensor of 2 to DG_MAX_GROUPS + 1 entries")
    _check(offsets, "offsets", _I32, (offsets.shape[0],), dev)
    return offsets.shape[0] - 1


def dg_route_sort(ids, groups: int, align: int = 1, offsets=None, position=None, slot=None, workspace=None, stream=None):
    """(offsets, position, slot): the stable sort of every token's choices by group, as the calls below take it.

    ids: [tokens, k] int32 or int64 (torch.topk's, say); a value outside 0 .. groups - 1
    takes the choice out. align: every group starts at a multiple of it (1, or gran for
    calls with gran x gran factors). offsets [groups + 1] int32: group e has the sorted
    rows offsets[e] .. offsets[e + 1] - 1. position [tokens, k] int32: each choice's row
    (-1: none). slot int32, at least dg_route_rows(...) long: each row's choice t * k + j
    (-1: a row between groups, -2: behind the last). Nothing is copied to the host.
    workspace: a uint8 tensor of dg_route_sort_workspace(...) bytes (allocated when None).
    """
    if stream is None:
        rc = _binding.route_sort(ids, groups, align, offsets, position, slot, workspace)
        if rc is not None:
            if rc:
                _raise(rc, "dg_route_sort")
            return offsets, position, slot
    tokens, k = shape = _matrix(ids, "ids")
    dev = ids.device
    _check(ids, "ids", tuple(_ID_BYTES), shape, dev)
    _sizes("dg_route_sort", tokens, k, groups, align)
    least = _count(_lib.dg_route_rows(tokens, k, groups, align), "dg_route_sort")
    if slot is not None and (not isinstance(slot, torch.Tensor) or slot.dim() != 1 or slot.shape[0] < least):
        raise ValueError("slot must be 1-D with at least dg_route_rows(...) = %d entries" % least)
    rows = least if slot is None else slot.shape[0]
    offsets = _out(offsets, "offsets", _I32, (groups + 1,), dev, stream)
    position = _out(position, "position", _I32, shape, dev, stream)
    slot = _out(slot, "slot", _I32, (rows,), dev, stream)
    need = _lib.dg_route_sort_workspace(tokens, k, groups)
    ws = _workspace(workspace, need, dev, stream) if need > 0 else None
    _launch(_lib.dg_route_sort, "dg_route_sort", dev, stream, ids.data_ptr(), _ID_BYTES[ids.dtype], tokens, k, groups, align,
            offsets.data_ptr(), position.data_ptr(), slot.data_ptr(), rows, _ptr(ws), ws.numel() if need > 0 else 0)
    return offsets, position, slot


def dg_route_rows(tokens: int, k: int, groups: int, align: int = 1) -> int:
    """Sorted rows that hold any routing of tokens x k choices among groups."""
    _sizes("dg_route_rows", tokens, k, groups, align)
    return _count(_lib.dg_route_rows(tokens, k, groups, align), "dg_route_rows")


def dg_route_sort_workspace(tokens: int, k: int, groups: int) -> int:
    """Workspace bytes of dg_route_sort."""
    _sizes("dg_route_sort_workspace", tokens, k, groups)
    return _count(_lib.dg_route_sort_workspace(tokens, k, groups), "dg_route_sort_workspace")


def _routing(x, position, slot, weights, dev):
    """Checks (x, position, slot, weights) of a call on [tokens, k] choices; (tokens, cols, k, rows)."""
    tokens, cols = _matrix(x, "x")
    k = _matrix(position, "position")[1]
    _check(position, "position", _I32, (tokens, k), dev)
    rows = 0
    if slot is not None:
        rows = slot.numel() if isinstance(slot, torch.Tensor) else 0
        _check(slot, "slot", _I32, (rows,), dev)
    if weights is not None:
        _check(weights, "weights", _F32, (tokens, k), dev)
    return tokens, cols, k, rows


def dg_route_quantize_fp8(x, position, slot, weights=None, gran: int = 128, block_rows: int = 1, fmt: int = DG_FMT_E4M3,
                          q=None, scales=None, workspace=None, stream=None):
    """(q, scales): the tokens x as FP8 rows in sorted order, each multiplied by its choice's weight where they are given.

    The dispatch to the experts; with the combine's weights on the gradient of its output,
    the combine's gradient. x: [tokens, cols] float32, bfloat16 or float16 (any row pitch).
    position, slot: from dg_route_sort. weights: [tokens, k] float32. block_rows: 1 (a
    factor per row and segment) or gran (gran x gran blocks of sorted rows, which serve
    the weights' gradient too). q: [rows, cols] uint8 holding fmt's codes, or that float8
    dtype; scales: [ceil(rows/block_rows), cols/gran]. Rows between groups get codes of
    zero, rows behind the last group are left as they were. workspace: a uint8 tensor of
    dg_route_quantize_workspace(...) bytes (allocated when None).
    """
    if stream is None:
        rc = _binding.route_quantize(x, position, slot, weights, gran, block_rows, fmt, q, scales, workspace)
        if rc is not None:
            if rc:
                _raise(rc, "dg_route_quantize_fp8")
            return q, scales
    _matrix(x, "x")
    dev = x.device
    tokens, cols, k, rows = _routing(x, position, slot, weights, dev)
    if gran not in _GRANS or cols % gran or not rows:
        raise ValueError("slot must have rows, and gran must be 64, 128 or 256 and divide cols")
    if block_rows not in (gran, 1):
        raise ValueError("block_rows must be gran (g x g blocks) or 1 (per-row factors)")
    if fmt not in _FP8_OF:
        raise ValueError("fmt must be DG_FMT_E4M3 or DG_FMT_E5M2")
    _sizes("dg_route_quantize_fp8", tokens, cols, k, rows)
    ldx = _rows(x, "x", _IN_OF, (tokens, cols), dev)
    q = _out(q, "q", _FP8_OF[fmt], (rows, cols), dev, stream)
    scales = _out(scales, "scales", _F32, ((rows + block_rows - 1) // block_rows, cols // gran), dev, stream)
    need = _lib.dg_route_quantize_workspace(tokens, cols, k, rows, gran, block_rows)
    ws = _workspace(workspace, need, dev, stream) if need > 0 else None
    _launch(_lib.dg_route_quantize_fp8, "dg_route_quantize_fp8", dev, stream, x.data_ptr(), _IN_OF[x.dtype], ldx, tokens, cols,
            k, position.data_ptr(), slot.data_ptr(), rows, _ptr(weights), gran, block_rows, fmt, q.data_ptr(),
            scales.data_ptr(), _ptr(ws), ws.numel() if need > 0 else 0)
    return q, scales


def dg_route_quantize_workspace(tokens: int, cols: int, k: int, rows: int, gran: int = 128, block_rows: int = 1) -> int:
    """Workspace bytes of dg_route_quantize_fp8."""
    _sizes("dg_route_quantize_workspace", tokens, cols, k, rows, gran, block_rows)
    return _count(_lib.dg_route_quantize_workspace(tokens, cols, k, rows, gran, block_rows), "dg_route_quantize_workspace")


def dg_route_combine(y, position, weights=None, res=None, out=None, stream=None):
    """out[t] = res[t] + sum over j of weights[t, j] * y[position[t, j]], in float32, rounded once.

    y: [rows, cols] float32, bfloat16 or float16, position: [tokens, k] int32 (choices
    without a row add nothing), weights: [tokens, k] float32 or None (1 each: the
    dispatch's gradient), res: [tokens, cols] of out's type or None; it may be out. out's
    type: any of the three, by default res's or y's. Rows of y and res may have a pitch.
    """
    if stream is None:
        rc = _binding.route_combine(y, position, weights, res, out)
        if rc is not None:
            if rc:
                _raise(rc, "dg_route_combine")
            return out
    rows, cols = _matrix(y, "y")
    tokens, k = _matrix(position, "position")
    dev = y.device
    if not rows or not tokens or not k or cols % 8 or not cols:
        raise ValueError("y must have rows, and columns in a multiple of 8; position must have entries")
    _sizes("dg_route_combine", rows, tokens, cols, k)
    _check(position, "position", _I32, (tokens, k), dev)
    if weights is not None:
        _check(weights, "weights", _F32, (tokens, k), dev)
    ldy = _rows(y, "y", _IN_OF, (rows, cols), dev)
    ldres = 0 if res is None else _rows(res, "res", tuple(_IN_OF), (tokens, cols), dev)
    kinds = (res.dtype,) if res is not None else (out.dtype,) if isinstance(out, torch.Tensor) else (y.dtype,)
    if kinds[0] not in _IN_OF:
        raise ValueError("out must be float32, bfloat16 or float16")
    out = _out(out, "out", kinds, (tokens, cols), dev, stream)
    _launch(_lib.dg_route_combine, "dg_route_combine", dev, stream, y.data_ptr(), _IN_OF[y.dtype], ldy, rows, tokens, cols, k,
            position.data_ptr(), _ptr(weights), _ptr(res), ldres, out.data_ptr(), _IN_OF[out.dtype])
    return out


def dg_route_weight_grad(dout, y, position, dweights=None, stream=None):
    """dweights[t, j] = the dot product of dout[t] and y[position[t, j]] in float32: the gradient of the combine's weights.

    dout: [tokens, cols], y: [rows, cols], each float32, bfloat16 or float16 (any row
    pitch); position: [tokens, k] int32; choices without a row get 0.
    """
    if stream is None:
        rc = _binding.route_weight_grad(dout, y, position, dweights)
        if rc is not None:
            if rc:
                _raise(rc, "dg_route_weight_grad")
            return dweights
    tokens, cols = _matrix(dout, "dout")
    rows = _matrix(y, "y")[0]
    dev = dout.device
    k = _matrix(position, "position")[1]
    if not rows or not tokens or not k or cols % 8 or not cols:
        raise ValueError("dout and y must have rows, and columns in a multiple of 8; position must have entries")
    _sizes("dg_route_weight_grad", rows, tokens, cols, k)
    _check(position, "position", _I32, (tokens, k), dev)
    ldd = _rows(dout, "dout", _IN_OF, (tokens, cols), dev)
    ldy = _rows(y, "y", _IN_OF, (rows, cols), dev)
    dweights = _out(dweights, "dweights", _F32, (tokens, k), dev, stream)
    _launch(_lib.dg_route_weight_grad, "dg_route_weight_grad", dev, stream, dout.data_ptr(), _IN_OF[dout.dtype], ldd,
            y.data_ptr(), _IN_OF[y.dtype], ldy, rows, tokens, cols, k, position.data_ptr(), dweights.data_ptr())
    return dweights


def dg_gemm_fp8_grouped(a, b, sa, sb, offsets, out=None, gran: int = 128, layout: int = DG_LAYOUT_NT,
                        sa_rows: int | None = None, fmt_a: int = DG_FMT_E4M3, fmt_b: int = DG_FMT_E4M3,
                        act: int = DG_ACT_NONE, pre=None, stream=None):
    """out[r] = bf16(act(a[r] B_e^T)) for the rows r of group e, every group with its own block-scaled B.

    a: [rows, K]; b: [groups, N, K] (DG_LAYOUT_NT) or [groups, K, N] (DG_LAYOUT_NN, the
    gradient of the rows); sa: [rows, K/gran] with sa_rows = 1, or [ceil(rows/gran),
    K/gran] with sa_rows = gran (the default; every group then starts at a multiple of
    gran); sb: [groups, ceil(N/gran), K/gran]; offsets: from dg_route_sort. act: any
    DG_ACT_* code; pre: optional [rows, N] bfloat16 that receives the product before it,
    for dg_epilogue_backward_fp8. Rows behind the last group are left as they were.
    """
    sa_rows = gran if sa_rows is None else sa_rows
    if stream is None:
        rc = _binding.gemm_grouped(a, b, sa, sb, offsets, out, gran, layout, sa_rows, fmt_a, fmt_b, act, pre)
        if rc is not None:
            if rc:
                _raise(rc, "dg_gemm_fp8_grouped")
            return out
    rows, K = _matrix(a, "a")
    dev = a.device
    groups = _groups(offsets, dev)
    if layout not in (DG_LAYOUT_NT, DG_LAYOUT_NN):
        raise ValueError("layout must be DG_LAYOUT_NT or _NN")
    if not isinstance(b, torch.Tensor) or b.dim() != 3:
        raise ValueError("b must be a 3-D tensor")
    N = b.shape[2] if layout else b.shape[1]
    if gran not in _GRANS or K % gran or not rows or not N or not K:
        raise ValueError("a and b must have entries, and gran must be 64, 128 or 256 and divide K")
    if sa_rows not in (gran, 1):
        raise ValueError("sa_rows must be gran (g x g blocks) or 1 (per-row factors)")
    if fmt_a not in _FP8_OF or fmt_b not in _FP8_OF:
        raise ValueError("formats must be DG_FMT_E4M3 or DG_FMT_E5M2")
    if act not in _ACTS:
        raise ValueError("act must be one of the DG_ACT_* codes")
    _check(a, "a", _FP8_OF[fmt_a], (rows, K), dev)
    _check(b, "b", _FP8_OF[fmt_b], (groups, K, N) if layout else (groups, N, K), dev)
    _check(sa, "sa", _F32, ((rows + sa_rows - 1) // sa_rows, K // gran), dev)
    _check(sb, "sb", _F32, (groups, (N + gran - 1) // gran, K // gran), dev)
    if pre is not None:
        _check(pre, "pre", _BF16, (rows, N), dev)
    out = _out(out, "out", _BF16, (rows, N), dev, stream)
    _launch(_lib.dg_gemm_fp8_grouped, "dg_gemm_fp8_grouped", dev, stream, a.data_ptr(), b.data_ptr(), sa.data_ptr(),
            sb.data_ptr(), offsets.data_ptr(), groups, out.data_ptr(), rows, N, K, gran, layout, sa_rows, fmt_a, fmt_b, act,
            _ptr(pre))
    return out


def dg_gemm_fp8_grouped_wgrad(a, b, sa, sb, offsets, out=None, gran: int = 128, fmt_a: int = DG_FMT_E5M2,
                              fmt_b: int = DG_FMT_E4M3, stream=None):
    """out[e] = bf16(A_e^T B_e) over the rows of group e: the gradient of every group's weights.

    a: [rows, M] codes (the gradient of the product's output, E5M2 by default), b:
    [rows, N] (the product's input), sa: [rows/gran, M/gran] and sb: [rows/gran, N/gran]
    as the quantisers leave their gran x gran blocks; offsets from dg_route_sort with
    align a multiple of gran. out: [groups, M, N] bfloat16; zeros for a group without rows.
    """
    if stream is None:
        rc = _binding.grouped_wgrad(a, b, sa, sb, offsets, out, gran, fmt_a, fmt_b)
        if rc is not None:
            if rc:
                _raise(rc, "dg_gemm_fp8_grouped_wgrad")
            return out
    rows, M = _matrix(a, "a")
    N = _matrix(b, "b")[1]
    dev = a.device
    groups = _groups(offsets, dev)
    if gran not in _GRANS or rows % gran or M % gran or N % gran or not rows or not M or not N:
        raise ValueError("gran must be 64, 128 or 256 and divide rows and the columns of a and b")
    if fmt_a not in _FP8_OF or fmt_b not in _FP8_OF:
        raise ValueError("formats must be DG_FMT_E4M3 or DG_FMT_E5M2")
    _check(a, "a", _FP8_OF[fmt_a], (rows, M), dev)
    _check(b, "b", _FP8_OF[fmt_b], (rows, N), dev)
    _check(sa, "sa", _F32, (rows // gran, M // gran), dev)
    _check(sb, "sb", _F32, (rows // gran, N // gran), dev)
    out = _out(out, "out", _BF16, (groups, M, N), dev, stream)
    _launch(_lib.dg_gemm_fp8_grouped_wgrad, "dg_gemm_fp8_grouped_wgrad", dev, stream, a.data_ptr(), b.data_ptr(), sa.data_ptr(),
            sb.data_ptr(), offsets.data_ptr(), groups, out.data_ptr(), rows, M, N, gran, fmt_a, fmt_b)
    return out


def dg_lora(x, a, b, offsets, position, slot, scale=None, base=None, out=None, workspace=None, stream=None):
    """out[t] = base[t] + scale[l] * (x[t] A_l^T) B_l^T, l the adapter of row t; base alone where it has none.

    x: [tokens, K] bfloat16 or float16 (any row pitch); a: [adapters, rank, K] and b:
    [adapters, N, rank] of its type, rank a multiple of 8 up to 128; scale: [adapters]
    float32 or None. offsets, position, slot: dg_route_sort(adapter_of_row[:, None],
    adapters), once for all projections of a step. base: [tokens, N] float32, bfloat16 or
    float16 (any row pitch), the shared projection's output, or None (zero); out, of its
    type (x's without base), may be base. workspace: a uint8 tensor of
    dg_lora_workspace(...) bytes (allocated when None).
    """
    if stream is None:
        rc = _binding.lora(x, a, b, offsets, position, slot, scale, base, out, workspace)
        if rc is not None:
            if rc:
                _raise(rc, "dg_lora")
            return out
    tokens, K = _matrix(x, "x")
    dev = x.device
    kinds = (torch.bfloat16, torch.float16)
    ldx = _rows(x, "x", kinds, (tokens, K), dev)
    groups = _groups(offsets, dev)
    if not isinstance(a, torch.Tensor) or not isinstance(b, torch.Tensor) or a.dim() != 3 or b.dim() != 3:
        raise ValueError("a and b must be 3-D tensors")
    rank, N = a.shape[1], b.shape[1]
    _check(a, "a", (x.dtype,), (groups, rank, K), dev)
    _check(b, "b", (x.dtype,), (groups, N, rank), dev)
    _sizes("dg_lora", tokens, K, N, rank)
    need = _count(_lib.dg_lora_workspace(tokens, K, N, rank, groups), "dg_lora")
    _check(position, "position", _I32, (tokens, 1), dev)
    _check(slot, "slot", _I32, (tokens,), dev)
    if scale is not None:
        _check(scale, "scale", _F32, (groups,), dev)
    ldbase = 0 if base is None else _rows(base, "base", tuple(_IN_OF), (tokens, N), dev)
    kind = base.dtype if base is not None else out.dtype if isinstance(out, torch.Tensor) else x.dtype
    if kind not in _IN_OF:
        raise ValueError("out must be float32, bfloat16 or float16")
    out = _out(out, "out", (kind,), (tokens, N), dev, stream)
    ws = _workspace(workspace, need, dev, stream)
    _launch(_lib.dg_lora, "dg_lora", dev, stream, x.data_ptr(), _IN_OF[x.dtype], ldx, tokens, K, a.data_ptr(), b.data_ptr(),
            _ptr(scale), N, rank, groups, offsets.data_ptr(), position.data_ptr(), slot.data_ptr(), _ptr(base), ldbase,
            out.data_ptr(), _IN_OF[kind], ws.data_ptr(), ws.numel())
    return out


def dg_lora_workspace(tokens: int, K: int, N: int, rank: int, adapters: int) -> int:
    """Workspace bytes of dg_lora."""
    _sizes("dg_lora_workspace", tokens, K, N, rank, adapters)
    return _count(_lib.dg_lora_workspace(tokens, K, N, rank, adapters), "dg_lora_workspace")


__all__ = ["dg_gemm_fp8_nt", "dg_gemm_fp8_nt_fmt", "dg_gemm_fp8_nt_epi", "dg_gemm_fp8_nt_ex", "dg_gemm_fp8_layout",
           "dg_gemm_fp8_ws", "dg_workspace", "dg_gemm_fp8_noalloc", "dg_noalloc_scratch_bytes", "DG_ESCRATCH",
           "DG_LAYOUT_NT", "DG_LAYOUT_NN", "DG_LAYOUT_TT", "DG_LAYOUT_TN", "DG_ACT_NONE",
           "DG_ACT_RELU", "DG_ACT_GELU", "dg_quantize_e4m3_blocks", "dg_quantize_fp8_blocks", "dg_quantize_fp8_rows",
           "dg_quantize_fp8_blocks_typed", "dg_quantize_fp8_rows_typed", "DG_IN_F32", "DG_IN_BF16", "DG_IN_F16",
           "dg_query_tile", "dg_strerror", "dg_version", "DGError", "DGArgumentError", "DG_OK", "DG_EINVAL",
           "dg_gemm_fp8_residual", "dg_gemm_fp8_residual_workspace", "dg_rmsnorm_quantize_fp8", "dg_rmsnorm_backward",
           "dg_rmsnorm_backward_workspace",
           "dg_route_sort", "dg_route_rows", "dg_route_sort_workspace", "dg_route_quantize_fp8", "dg_route_quantize_workspace",
           "dg_route_combine", "dg_route_weight_grad", "dg_gemm_fp8_grouped", "dg_gemm_fp8_grouped_wgrad", "dg_lora",
           "dg_lora_workspace", "DG_MAX_GROUPS",
           "dg_epilogue_backward_fp8", "dg_epilogue_backward_workspace", "DG_ACT_SILU", "DG_ACT_GELU_TANH",
           "DG_EALIGN", "DG_EUNSUPPORTED", "DG_ELAUNCH", "DG_FMT_E4M3", "DG_FMT_E5M2", "DG_MAX_DIM", "LIB_PATH"]

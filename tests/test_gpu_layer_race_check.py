"""The race check build (libdg_sync.so: extra waits and barriers around every
reduction through LDS) of the norm's and the gradients' kernels gives the
release build's bits."""

import ctypes

import pytest
import torch

from tests import _layer_ref as ref
from tests._gpu import say
from tests.test_gpu_layer import weight

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def dg():
    import fp8_block_scaled_scales_amd as dg

    return dg


def _raw(lib, dg, what, t):
    """One call through the C ABI of `lib`; every output, cleared first."""
    p = lambda x: None if x is None else x.data_ptr()  # noqa: E731
    for k in t["outs"]:
        if t[k] is not None:
            t[k].view(torch.uint8).fill_(0x5A)
    kind = {F32: 0, BF16: 1, F16: 2}
    st = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    ws, nb = t["ws"], t["ws"].numel()
    if what == "norm":
        x, res = t["x"], t["res"]
        rc = lib.dg_rmsnorm_quantize_fp8(p(x), kind[x.dtype], x.shape[1], p(res), kind[res.dtype], res.shape[1], p(t["w"]), 1e-6, *x.shape, 64, 0,
                                         p(t["h"]), p(t["y"]), p(t["rstd"]), p(t["q"]), p(t["s"]), st)
    elif what == "norm_bwd":
        dy, h = t["x"], t["res"]
        rc = lib.dg_rmsnorm_backward(p(dy), kind[dy.dtype], dy.shape[1], p(h), kind[h.dtype], h.shape[1], p(t["rstd"]), p(t["w"]), p(t["dh"]),
                                     dy.shape[1], *dy.shape, p(t["dx"]), p(t["dw"]), p(ws), nb, st)
    else:
        d = t["x"]
        rc = lib.dg_epilogue_backward_fp8(p(d), kind[d.dtype], d.shape[1], p(t["pre"]), d.shape[1], 2, *d.shape, t["g"], t["br"], 1, p(t["dz"]),
                                          p(t["db"]), p(t["q"]), p(t["s"]), p(ws), nb, st)
    torch.cuda.synchronize()
    assert rc == 0, lib.dg_strerror(rc)
    return {k: t[k].clone() for k in t["outs"] if t[k] is not None}


def _same(a, b):
    return all(torch.equal(a[k].view(torch.uint8), b[k].view(torch.uint8)) for k in a)


@pytest.mark.parametrize("xk,rk", [(BF16, BF16), (BF16, F32)])
@pytest.mark.parametrize("rows,cols", [(700, 512), (700, 1024), (700, 2048), (300, 4096), (300, 8192), (150, 16384), (70, 32768), (40, 40960),
                                       (2500, 512), (4000, 2048), (1800, 4096), (900, 8192), (500, 16384)])
def test_norm_race_check_build(dg, rows, cols, xk, rk):
    """Every number of threads per row, one and two launches backward: the build with extra waits and barriers around the
    reductions through LDS gives the same bits."""
    sync = dg.load_library(dg.SYNC_LIB_PATH)
    e = lambda *shape, dtype=F32: torch.empty(*shape, dtype=dtype, device=DEV)  # noqa: E731
    t = dict(x=ref.stream(rows, rows, cols, xk).to(DEV), res=ref.stream(cols, rows, cols, rk).to(DEV), w=weight(cols).to(DEV),
             h=e(rows, cols, dtype=rk), y=e(rows, cols, dtype=xk), rstd=e(rows), q=e(rows, cols, dtype=torch.uint8), s=e(rows, cols // 64),
             ws=e(max(16, dg.dg_rmsnorm_backward_workspace(rows, cols)), dtype=torch.uint8), outs=("h", "y", "rstd", "q", "s"))
    say("norm race check %dx%d %s" % (rows, cols, rk))
    assert _same(_raw(dg.lib, dg, "norm", t), _raw(sync, dg, "norm", t))
    t.update(dh=t["h"].clone(), dx=e(rows, cols, dtype=rk), dw=e(cols), outs=("dx", "dw"))
    assert _same(_raw(dg.lib, dg, "norm_bwd", t), _raw(sync, dg, "norm_bwd", t))


@pytest.mark.parametrize("dk", [BF16, F32])
@pytest.mark.parametrize("rows,cols,g,by_rows", [(100, 1024, 128, False), (600, 1024, 64, False), (600, 1024, 128, False), (600, 1024, 256, False),
                                                 (600, 1024, 64, True), (3000, 1280, 64, False), (3000, 1280, 128, False), (3000, 1280, 256, False),
                                                 (3000, 1280, 128, True), (4200, 8192, 128, False)])
def test_epilogue_backward_race_check_build(dg, rows, cols, g, by_rows, dk):
    sync = dg.load_library(dg.SYNC_LIB_PATH)
    br = 1 if by_rows else g
    e = lambda *shape, dtype=F32: torch.empty(*shape, dtype=dtype, device=DEV)  # noqa: E731
    t = dict(x=(ref.stream(rows, rows, cols, F32) * 0.01).to(dk).to(DEV), pre=ref.stream(cols, rows, cols, BF16).to(DEV), dz=e(rows, cols, dtype=dk),
             db=e(cols), q=e(rows, cols, dtype=torch.uint8), s=e(-(-rows // br), cols // g), g=g, br=br,
             ws=e(max(16, dg.dg_epilogue_backward_workspace(rows, cols, g, br)), dtype=torch.uint8), outs=("dz", "db", "q", "s"))
    say("epilogue backward race check %dx%d g=%d rows=%d %s" % (rows, cols, g, by_rows, dk))
    assert _same(_raw(dg.lib, dg, "epi", t), _raw(sync, dg, "epi", t))

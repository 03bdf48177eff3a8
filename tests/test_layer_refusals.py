"""The calls around the product (norm, residual epilogue, their gradients) on
the CPU: bad arguments are refused with the documented status before any HIP
call, and the Python binding raises before it calls the library. Also the
64-bit references of the GPU tests against differences."""

import ctypes

import pytest
import torch

from tests import _layer_ref as ref


@pytest.fixture(scope="module")
def dg():
    import fp8_block_scaled_scales_amd as dg

    return dg


# fake device addresses, aligned and 2^40 apart
X, RES, W, H, Y, RSTD, Q, S, DX, DW, WS, PRE = ((i + 1) << 40 for i in range(12))
BIG = 1 << 30


def _norm(dg, x=X, xk=1, ldx=256, res=RES, rk=0, ldres=256, w=W, eps=1e-6, rows=8, cols=256, g=128, fmt=0, h=H, y=Y,
          rstd=RSTD, q=Q, s=S):
    return dg.lib.dg_rmsnorm_quantize_fp8(x, xk, ldx, res, rk, ldres, w, eps, rows, cols, g, fmt, h, y, rstd, q, s, None)


@pytest.mark.parametrize("kw,want", [
    (dict(x=0), "EINVAL"), (dict(w=0), "EINVAL"), (dict(q=0), "EINVAL"), (dict(s=0), "EINVAL"),
    (dict(res=0), "EINVAL"), (dict(h=0), "EINVAL"),  # h goes with a residual
    (dict(xk=3), "EINVAL"), (dict(rk=-1), "EINVAL"), (dict(fmt=2), "EINVAL"),
    (dict(rows=0), "EINVAL"), (dict(cols=0), "EINVAL"), (dict(rows=-1), "EINVAL"), (dict(rows=1 << 24), "EINVAL"),
    (dict(cols=192, ldx=192, ldres=192), "EINVAL"), (dict(g=96), "EINVAL"), (dict(g=32), "EINVAL"),
    (dict(ldx=255), "EINVAL"), (dict(ldres=128), "EINVAL"), (dict(ldx=1 << 24), "EINVAL"),
    (dict(eps=-1e-6), "EINVAL"), (dict(eps=float("nan")), "EINVAL"), (dict(eps=float("inf")), "EINVAL"),
    (dict(x=X + 8), "EALIGN"), (dict(ldx=260), "EALIGN"), (dict(res=RES + 4), "EALIGN"), (dict(ldres=257), "EALIGN"),
    (dict(w=W + 4), "EALIGN"), (dict(h=H + 8), "EALIGN"), (dict(y=Y + 2), "EALIGN"), (dict(q=Q + 4), "EALIGN"),
    (dict(rstd=RSTD + 2), "EALIGN"), (dict(s=S + 1), "EALIGN"),
    (dict(h=X), "EINVAL"), (dict(y=X), "EINVAL"), (dict(q=W), "EINVAL"), (dict(s=RES), "EINVAL"), (dict(y=H), "EINVAL"),
    (dict(h=RES + 16), "EINVAL"), (dict(h=RES, ldres=512), "EINVAL"),  # in place only on the residual itself
])
def test_norm_refuses(dg, kw, want):
    assert _norm(dg, **kw) == getattr(dg, "DG_" + want)


def _bwd(dg, dy=X, dk=1, lddy=256, h=H, hk=0, ldh=256, rstd=RSTD, w=W, dh=RES, lddh=256, rows=64, cols=256, dx=DX,
         dw=DW, ws=WS, nb=BIG):
    return dg.lib.dg_rmsnorm_backward(dy, dk, lddy, h, hk, ldh, rstd, w, dh, lddh, rows, cols, dx, dw, ws, nb, None)


@pytest.mark.parametrize("kw,want", [
    (dict(dy=0), "EINVAL"), (dict(h=0), "EINVAL"), (dict(rstd=0), "EINVAL"), (dict(w=0), "EINVAL"), (dict(dx=0), "EINVAL"),
    (dict(dw=0), "EINVAL"), (dict(dk=5), "EINVAL"), (dict(hk=3), "EINVAL"), (dict(rows=0), "EINVAL"),
    (dict(cols=200), "EINVAL"), (dict(cols=0), "EINVAL"), (dict(lddy=192), "EINVAL"), (dict(ldh=0), "EINVAL"),
    (dict(lddh=64), "EINVAL"), (dict(rows=4096, ws=0, nb=0), "EINVAL"), (dict(rows=4096, nb=64), "EINVAL"),
    (dict(nb=-1), "EINVAL"), (dict(dy=X + 2), "EALIGN"), (dict(lddy=257), "EALIGN"), (dict(ldh=258), "EALIGN"),
    (dict(lddh=259), "EALIGN"), (dict(w=W + 4), "EALIGN"), (dict(dx=DX + 8), "EALIGN"), (dict(dw=DW + 2), "EALIGN"),
    (dict(ws=WS + 8), "EALIGN"), (dict(dx=H), "EINVAL"), (dict(dx=X), "EINVAL"), (dict(dw=W), "EINVAL"),
    (dict(dx=RES + 16), "EINVAL"), (dict(dx=RES, lddh=512), "EINVAL"), (dict(rows=4096, ws=H), "EINVAL"),
])
def test_norm_backward_refuses(dg, kw, want):
    assert _bwd(dg, **kw) == getattr(dg, "DG_" + want)


def _epi(dg, dout=X, dk=1, lddout=256, pre=PRE, ldpre=256, act=2, rows=300, cols=256, g=128, br=128, fmt=1, dz=Y, db=DW,
         q=Q, s=S, ws=WS, nb=BIG):
    return dg.lib.dg_epilogue_backward_fp8(dout, dk, lddout, pre, ldpre, act, rows, cols, g, br, fmt, dz, db, q, s, ws, nb,
                                           None)


@pytest.mark.parametrize("kw,want", [
    (dict(dout=0), "EINVAL"), (dict(q=0), "EINVAL"), (dict(s=0), "EINVAL"), (dict(pre=0), "EINVAL"),
    (dict(act=0), "EINVAL"), (dict(act=5), "EINVAL"), (dict(act=-1), "EINVAL"), (dict(dk=3), "EINVAL"),
    (dict(fmt=2), "EINVAL"), (dict(rows=0), "EINVAL"), (dict(cols=192), "EINVAL"), (dict(g=96, br=96), "EINVAL"),
    (dict(br=64), "EINVAL"), (dict(br=0), "EINVAL"), (dict(lddout=255), "EINVAL"), (dict(ldpre=0), "EINVAL"),
    (dict(rows=4096, ws=0, nb=0), "EINVAL"), (dict(rows=4096, nb=16), "EINVAL"), (dict(nb=-1, db=0), "EINVAL"),
    (dict(dout=X + 8), "EALIGN"), (dict(lddout=257), "EALIGN"), (dict(ldpre=260), "EALIGN"), (dict(dz=Y + 8), "EALIGN"),
    (dict(q=Q + 4), "EALIGN"), (dict(db=DW + 2), "EALIGN"), (dict(s=S + 2), "EALIGN"), (dict(ws=WS + 4), "EALIGN"),
    (dict(dz=PRE), "EINVAL"), (dict(q=X), "EINVAL"), (dict(db=PRE), "EINVAL"), (dict(dz=X, lddout=512), "EINVAL"),
    (dict(rows=4096, ws=X), "EINVAL"), (dict(s=Q), "EINVAL"),
    # more than 2^22 - 1 blocks of 128, 2^24 - 1 of 64 (addresses spread far enough that nothing overlaps)
    (dict(rows=1 << 20, cols=1 << 16, lddout=1 << 16, ldpre=1 << 16, nb=1 << 34), "EINVAL"),
    (dict(rows=1 << 20, cols=1 << 16, lddout=1 << 16, ldpre=1 << 16, g=64, br=64, nb=1 << 36), "EINVAL"),
])
def test_epilogue_backward_refuses(dg, kw, want):
    assert _epi(dg, **kw) == getattr(dg, "DG_" + want)


def _gemm(dg, a=X, b=W, sa=S, sb=RSTD, out=H, M=256, N=256, K=256, g=128, layout=0, sa_rows=128, fa=0, fb=0, bias=0, act=2,
          res=RES, rk=1, ldres=256, pre=PRE, ws=0, nb=0):
    return dg.lib.dg_gemm_fp8_residual(a, b, sa, sb, out, M, N, K, g, layout, sa_rows, fa, fb, bias or None, act,
                                       res or None, rk, ldres, pre or None, ws or None, nb, None)


@pytest.mark.parametrize("kw,want", [
    (dict(a=0), "EINVAL"), (dict(out=0), "EINVAL"), (dict(M=0), "EINVAL"), (dict(K=192), "EINVAL"),
    (dict(layout=4), "EINVAL"), (dict(sa_rows=2), "EINVAL"), (dict(fa=2), "EINVAL"), (dict(act=5), "EINVAL"),
    (dict(act=-1), "EINVAL"), (dict(rk=3), "EINVAL"), (dict(ldres=255), "EINVAL"), (dict(ldres=1 << 24), "EINVAL"),
    (dict(res=RES + 1), "EALIGN"), (dict(res=RES + 2, rk=0), "EALIGN"), (dict(pre=PRE + 1), "EALIGN"),
    (dict(bias=Q + 2), "EALIGN"), (dict(out=H + 1), "EALIGN"), (dict(a=X + 8), "EALIGN"),
    (dict(pre=H), "EINVAL"), (dict(pre=RES), "EINVAL"), (dict(pre=X), "EINVAL"), (dict(out=X), "EINVAL"),
    (dict(res=H, rk=0), "EINVAL"), (dict(res=H + 2), "EINVAL"), (dict(res=H, ldres=264), "EINVAL"),
    (dict(ws=WS, nb=0), "EINVAL"), (dict(ws=0, nb=64), "EINVAL"), (dict(nb=-1), "EINVAL"), (dict(ws=WS + 16, nb=64), "EALIGN"),
    (dict(ws=PRE, nb=64), "EINVAL"), (dict(ws=RES, nb=64), "EINVAL"), (dict(ws=H, nb=64), "EINVAL"),
    (dict(M=64, N=64, K=32768, ldres=64, ws=WS, nb=64), "EINVAL"),  # less than the split needs
])
def test_residual_product_refuses(dg, kw, want):
    assert _gemm(dg, **kw) == getattr(dg, "DG_" + want)


def test_the_plain_calls_keep_their_activations(dg):
    for act in (dg.DG_ACT_SILU, dg.DG_ACT_GELU_TANH):
        assert dg.lib.dg_gemm_fp8_layout(X, W, S, RSTD, H, 256, 256, 256, 128, 0, 0, 0, None, act, None) == dg.DG_EINVAL


def test_workspace_sizes(dg):
    for rows, cols in [(1, 64), (3, 7168), (2000, 16384), (8192, 8192), (1 << 20, 64), (dg.DG_MAX_DIM, 64), (5, 1 << 23)]:
        n = dg.dg_rmsnorm_backward_workspace(rows, cols)
        assert n >= 0 and n % (4 * cols) == 0
        for g in (64, 128, 256):
            if cols % g == 0:
                for br in (g, 1):
                    m = dg.dg_epilogue_backward_workspace(rows, cols, g, br)
                    assert m >= 0 and m % (4 * cols) == 0 and m // (4 * cols) <= rows
    assert dg.dg_epilogue_backward_workspace(128, 4096, 128) == 0  # one row of blocks: its sums are dbias
    for bad in [(0, 64), (8, 100), (8, 0), (1 << 24, 64)]:
        with pytest.raises(ValueError):
            dg.dg_rmsnorm_backward_workspace(*bad)
    # a K split: from 8192, with a transposed operand from 6144, and at least eight ways
    for M, N, K, layout, splits in [(64, 512, 8064, 0, 0), (64, 512, 8192, 0, 16), (64, 512, 6144, 3, 12), (64, 512, 6016, 1, 0),
                                    (64, 64, 8192, 2, 16), (64, 2176, 8192, 3, 8), (64, 2560, 8192, 3, 0), (4096, 4096, 8192, 3, 0)]:
        tiles = -(-M // 64) * -(-N // 64)
        assert dg.dg_gemm_fp8_residual_workspace(M, N, K, 128, layout) == 4 * 64 * 64 * tiles * splits, (M, N, K, layout)
    for bad in [(0, 64, 128), (64, 64, 192)]:
        with pytest.raises(ValueError):
            dg.dg_gemm_fp8_residual_workspace(*bad)
    with pytest.raises(ValueError):
        dg.dg_epilogue_backward_workspace(8, 192, 128)
    with pytest.raises(ValueError):
        dg.dg_epilogue_backward_workspace(8, 256, 128, 2)


def test_new_codes_match_header(dg):
    import os
    import re

    text = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "dg.h")).read()
    for name in ("DG_ACT_SILU", "DG_ACT_GELU_TANH"):
        assert int(re.search(r"#define %s (\d+)" % name, text).group(1)) == getattr(dg, name)


def test_binding_refuses(dg):
    x = torch.zeros(4, 256, dtype=torch.bfloat16)
    w = torch.ones(256)
    pre = torch.zeros(4, 256, dtype=torch.bfloat16)
    for fn, message in [
        (lambda: dg.dg_rmsnorm_quantize_fp8(x, None, w), "GPU"),
        (lambda: dg.dg_rmsnorm_quantize_fp8(x, None, w, h=x), "residual"),
        (lambda: dg.dg_rmsnorm_quantize_fp8(x, x[:3], w), "res has shape"),
        (lambda: dg.dg_rmsnorm_quantize_fp8(x, x.t().contiguous().t(), w), "contiguous rows"),
        (lambda: dg.dg_rmsnorm_quantize_fp8(x, x[:1].expand(4, 256), w), "contiguous rows"),
        (lambda: dg.dg_rmsnorm_quantize_fp8(x, x, w, h=x.float()), "h has dtype"),
        (lambda: dg.dg_rmsnorm_quantize_fp8(x, x, w.bfloat16()), "weight has dtype"),
        (lambda: dg.dg_rmsnorm_quantize_fp8(x, x, w[:128]), "weight has shape"),
        (lambda: dg.dg_rmsnorm_quantize_fp8(x.double(), None, w), "x has dtype"),
        (lambda: dg.dg_rmsnorm_quantize_fp8(x[0], None, w), "2-D"),
        (lambda: dg.dg_rmsnorm_quantize_fp8(x, None, w, gran=96), "gran"),
        (lambda: dg.dg_rmsnorm_quantize_fp8(x, None, w, fmt=2), "fmt"),
        (lambda: dg.dg_rmsnorm_quantize_fp8(x, None, w, y=x.float()), "y has dtype"),
        (lambda: dg.dg_rmsnorm_quantize_fp8(x, None, w, q=torch.zeros(4, 256, dtype=torch.float8_e5m2)), "q has dtype"),
        (lambda: dg.dg_rmsnorm_backward(x, x, torch.ones(4), w), "GPU"),
        (lambda: dg.dg_rmsnorm_backward(x, x, torch.ones(5), w), "rstd has shape"),
        (lambda: dg.dg_rmsnorm_backward(x, x, torch.ones(4), w, dh=x.float()), "dh has dtype"),
        (lambda: dg.dg_rmsnorm_backward(x[:, :100], x[:, :100], torch.ones(4), w[:100]), "multiple of 64"),
        (lambda: dg.dg_rmsnorm_backward(x[:0], x[:0], torch.ones(0), w), "rows"),
        (lambda: dg.dg_epilogue_backward_fp8(x, pre, 2), "GPU"),
        (lambda: dg.dg_epilogue_backward_fp8(x, None, 2), "pre goes with"),
        (lambda: dg.dg_epilogue_backward_fp8(x, pre, 0), "pre goes with"),
        (lambda: dg.dg_epilogue_backward_fp8(x, pre, 9), "act"),
        (lambda: dg.dg_epilogue_backward_fp8(x, pre.float(), 1), "pre has dtype"),
        (lambda: dg.dg_epilogue_backward_fp8(x, pre, 1, block_rows=64), "block_rows"),
        (lambda: dg.dg_epilogue_backward_fp8(x, pre, 1, dbias=w.bfloat16()), "dbias has dtype"),
        (lambda: dg.dg_epilogue_backward_fp8(x, pre, 1, dz=x.float()), "dz has dtype"),
    ]:
        with pytest.raises(ValueError, match=message):
            fn()
    a = torch.zeros(64, 256, dtype=torch.float8_e4m3fn)
    b = torch.zeros(32, 256, dtype=torch.float8_e4m3fn)
    s = torch.zeros(1, 2)
    res = torch.zeros(64, 32, dtype=torch.bfloat16)
    for kw, message in [(dict(res=res), "GPU"), (dict(res=res[:10]), "res has shape"), (dict(res=res.double()), "res has dtype"),
                        (dict(pre=res.float()), "pre has dtype"), (dict(act=7), "act"), (dict(sa_rows=3), "sa_rows")]:
        with pytest.raises(ValueError, match=message):
            dg.dg_gemm_fp8_residual(a, b, s, s, **kw)


def test_norm_reference_gradient_against_differences():
    x, w = ref.stream(1, 3, 64, torch.float64), 1 + 0.3 * torch.randn(64, generator=torch.Generator().manual_seed(2)).double()
    dy, dh = ref.stream(3, 3, 64, torch.float64), ref.stream(4, 3, 64, torch.float64)

    def loss(x, w):
        rstd = 1 / torch.sqrt((x * x).mean(1) + 1e-6)
        return float((x * rstd[:, None] * w * dy).sum() + (x * dh).sum())

    rstd = 1 / torch.sqrt((x * x).mean(1) + 1e-6)
    dx, dw, _, _ = ref.norm_bwd(dy, x, rstd, w, dh)
    for (r, c), step in [((0, 0), 1e-5), ((1, 17), 1e-5), ((2, 63), 1e-5)]:
        d = torch.zeros_like(x)
        d[r, c] = step
        assert abs((loss(x + d, w) - loss(x - d, w)) / (2 * step) - dx[r, c]) <= 1e-7 * (1 + abs(dx[r, c])) * 10
        d = torch.zeros_like(w)
        d[c] = step
        assert abs((loss(x, w + d) - loss(x, w - d)) / (2 * step) - dw[c]) <= 1e-7 * (1 + abs(dw[c])) * 10


@pytest.mark.parametrize("code", range(5))
def test_activation_reference_gradient_against_differences(code):
    z = torch.tensor([-9.0, -4.1, -1.7, -0.75, -1e-3, 2e-3, 0.4, 1.0, 3.3, 8.0], dtype=torch.float64)
    d = (ref.act(z + 1e-6, code) - ref.act(z - 1e-6, code)) / 2e-6
    assert ((d - ref.act_grad(z, code)).abs() <= 1e-8).all()


def test_every_new_call_is_declared_and_bound(dg):
    for name in ("dg_gemm_fp8_residual", "dg_rmsnorm_quantize_fp8", "dg_rmsnorm_backward", "dg_epilogue_backward_fp8"):
        assert isinstance(getattr(dg.lib, name), ctypes._CFuncPtr) and name in dg.__all__

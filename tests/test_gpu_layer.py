"""The operators around the product on the GPU against their 64-bit forms
(tests/_layer_ref.py): the RMS norm with residual and FP8 output and its
gradient, the product with a residual in its epilogue, and the gradient through
that epilogue. Bounds count FP32 roundings and half steps of each output type."""

import numpy as np
import pytest
import torch

import oracle
import synth
from tests import _common
from tests import _layer_ref as ref
from tests._gpu import device_inputs, say

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
NORM_REL = 64 * ref.U32  # FP32 y: sum of squares of depth below 64 (halved by the root), and a few roundings


@pytest.fixture(scope="module")
def dg():
    import fp8_block_scaled_scales_amd as dg

    return dg


def weight(cols, seed=5):
    return 1.0 + 0.3 * torch.randn(cols, generator=torch.Generator().manual_seed(seed))


def close(got, want, bound, label):
    off = (got.cpu().double() - want).abs()
    bad = ~(off <= bound)
    assert not bad.any(), "%s: %d of %d outside, worst %g of the bound" % (
        label, int(bad.sum()), bad.numel(), float((off / bound.clamp(min=1e-300)).max()))


# Rows of one wave, of 256 and of 1024 threads, with one to four pieces each, and
# the rows that are read twice (past 32768); lengths of one row and odd counts.
SHAPES = [(1, 64, 64), (1, 7168, 128), (13, 192, 64), (130, 512, 256), (9, 768, 256), (33, 2048, 128), (6, 4096, 256),
          (5, 8192, 128), (3, 8256, 64), (4, 16384, 64), (2, 32768, 256), (2, 33024, 64), (3, 65536, 128)]


@pytest.mark.parametrize("xk,rk,pad", [(BF16, BF16, 0), (BF16, F32, 64), (F16, None, 8), (F32, F32, 4), (F32, BF16, 0),
                                       (F16, F16, 16), (BF16, None, 0), (F32, None, 0)])
@pytest.mark.parametrize("rows,cols,g", SHAPES)
def test_norm(dg, rows, cols, g, xk, rk, pad):
    eps, fmt = 1e-5, (rows + cols // 64) % 2
    x = ref.stream(rows + cols, rows, cols, xk, zero_rows=(2,))
    res = None if rk is None else ref.stream(rows + 7, rows, cols, rk, zero_rows=(2,))
    w = weight(cols)
    h, rstd, y = ref.norm(x, res, w, eps)
    say("norm %dx%d g=%d fmt=%d %s %s pad=%d" % (rows, cols, g, fmt, xk, rk, pad))
    gy = torch.empty(rows, cols, dtype=xk, device=DEV)
    gr = torch.empty(rows, device=DEV)
    q, s, gh = dg.dg_rmsnorm_quantize_fp8(ref.padded(x, pad), None if res is None else ref.padded(res, pad), w.to(DEV), eps,
                                          gran=g, fmt=fmt, y=gy, rstd=gr)
    torch.cuda.synchronize()
    assert torch.equal(gh.cpu(), h)
    close(gr, rstd, 64 * ref.U32 * rstd, "rstd")
    tiny = 2.0 ** -25 if xk == F16 else 0.0  # half of FP16's smallest step
    close(gy, y, (NORM_REL + (0 if xk == F32 else ref.half_step(xk))) * 1.01 * y.abs() + tiny, "y")
    ref.check_codes(q.cpu(), s.cpu(), y, 1, g, fmt, NORM_REL)
    if xk == F32:  # y is what the codes are of: the quantiser itself agrees to the bit
        qq, ss = dg.dg_quantize_fp8_rows(gy, gran=g, fmt=fmt)
        assert torch.equal(qq, q) and torch.equal(ss, s)
    q2, s2, h2 = dg.dg_rmsnorm_quantize_fp8(x.to(DEV), None if res is None else res.to(DEV), w.to(DEV), eps, gran=g, fmt=fmt)
    assert torch.equal(q2, q) and torch.equal(s2, s) and torch.equal(h2.cpu(), h)  # serving form, no pitch


def test_norm_in_place_on_the_residual(dg):
    for rows, cols in [(3, 512), (40, 7168), (2, 65536)]:
        x, res, w = ref.stream(1, rows, cols, BF16).to(DEV), ref.stream(2, rows, cols, F32).to(DEV), weight(cols).to(DEV)
        say("norm in place %dx%d" % (rows, cols))
        q, s, h = dg.dg_rmsnorm_quantize_fp8(x, res, w)
        q2, s2, h2 = dg.dg_rmsnorm_quantize_fp8(x, res, w, h=res)
        assert h2 is res and torch.equal(h2, h) and torch.equal(q2, q) and torch.equal(s2, s)


def test_norm_of_zeros_and_extremes(dg):
    """Rows of zeros give codes of 0 and factors of 1; one large value among tiny ones; 16-bit subnormals."""
    x = torch.zeros(4, 256)
    x[1, 7] = 3.0e4
    x[1, 8:] = 1e-7
    x[2] = 6e-8
    x[3, ::2] = -6e4
    for dtype in (F32, F16, BF16):
        xd, w = x.to(dtype), torch.ones(256)
        _, rstd, y = ref.norm(xd, None, w, 1e-6)
        say("norm extremes %s" % dtype)
        q, s, _ = dg.dg_rmsnorm_quantize_fp8(xd.to(DEV), None, w.to(DEV), 1e-6, gran=64)
        assert not q[0].any() and (s[0] == 1).all()
        ref.check_codes(q.cpu(), s.cpu(), y, 1, 64, 0, NORM_REL)


@pytest.mark.parametrize("dk,hk,with_dh,pad", [(BF16, BF16, True, 0), (BF16, F32, True, 8), (F16, F16, False, 8),
                                               (F32, F32, True, 0), (F32, BF16, True, 64), (F16, F32, False, 0)])
@pytest.mark.parametrize("rows,cols", [(1, 64), (1, 8192), (3, 192), (64, 7168), (130, 512), (257, 2048), (19, 8256),
                                       (300, 4096), (40, 16384), (5, 32768), (3, 65536), (1000, 64),
                                       # two launches, for every number of threads per row
                                       (2100, 64), (2100, 512), (2600, 768), (3200, 2048), (1700, 4096), (900, 8192),
                                       (420, 16384), (1030, 6208)])
def test_norm_backward(dg, rows, cols, dk, hk, with_dh, pad):
    h, dy = ref.stream(rows, rows, cols, hk), ref.stream(cols, rows, cols, dk)
    dh = ref.stream(rows + cols, rows, cols, hk) if with_dh else None
    w = weight(cols)
    rstd = (1 / torch.sqrt(h.double().square().mean(1) + 1e-6)).float()
    dx, dw, bx, bw = ref.norm_bwd(dy, h, rstd, w, dh)
    say("norm backward %dx%d %s %s dh=%d pad=%d" % (rows, cols, dk, hk, with_dh, pad))
    args = (ref.padded(dy, pad), ref.padded(h, pad), rstd.to(DEV), w.to(DEV))
    gdh = None if dh is None else ref.padded(dh, pad)
    gx, gw = dg.dg_rmsnorm_backward(*args, dh=gdh)
    torch.cuda.synchronize()
    assert gx.dtype == hk and gw.dtype == F32
    tiny = 2.0 ** -25 if hk == F16 else 1e-37
    close(gx, dx, bx * 1.01 + (0 if hk == F32 else ref.half_step(hk)) * 1.01 * dx.abs() + tiny, "dx")
    close(gw, dw, bw + ref.U32 * dw.abs() + 1e-37, "dw")
    again = dg.dg_rmsnorm_backward(*args, dh=gdh)
    assert torch.equal(again[0], gx) and torch.equal(again[1], gw)  # fixed order of sums
    if dh is not None:
        over = dh.to(DEV)
        got = dg.dg_rmsnorm_backward(*args, dh=over, dx=over)[0]  # dx over dh
        assert got is over and torch.equal(over, gx)


def test_norm_backward_of_the_forward(dg):
    """The gradient of sum(y dy) + sum(h dh) through both kernels, against differences of the 64-bit loss."""
    rows, cols = 7, 320
    x, res, w = ref.stream(1, rows, cols, F32), ref.stream(2, rows, cols, F32), weight(cols)
    dy, dh = ref.stream(3, rows, cols, F32), ref.stream(4, rows, cols, F32)
    rstd = torch.empty(rows, device=DEV)
    say("norm forward and backward")
    _, _, h = dg.dg_rmsnorm_quantize_fp8(x.to(DEV), res.to(DEV), w.to(DEV), 1e-6, gran=64, rstd=rstd)
    dx, dw = dg.dg_rmsnorm_backward(dy.to(DEV), h, rstd, w.to(DEV), dh=dh.to(DEV))
    base = h.cpu().double()

    def loss(h, w):
        k = 1 / torch.sqrt((h * h).mean(1) + 1e-6)
        return float((h * k[:, None] * w * dy.double()).sum() + (h * dh.double()).sum())

    for r, c in [(0, 0), (3, 100), (6, 319)]:
        d = torch.zeros_like(base)
        d[r, c] = 1e-4
        slope = (loss(base + d, w.double()) - loss(base - d, w.double())) / 2e-4
        assert abs(slope - float(dx[r, c])) <= 1e-5 * (1 + abs(slope))
        d = torch.zeros(cols, dtype=torch.float64)
        d[c] = 1e-4
        slope = (loss(base, w.double() + d) - loss(base, w.double() - d)) / 2e-4
        assert abs(slope - float(dw[c])) <= 1e-5 * (1 + abs(slope))


# dz: the derivative is within 4e-7 of the exact one (GELU's polynomial 1e-7, the
# rest roundings of values up to 1.13), then one FP32 product.
ACT_ABS = 4e-7


@pytest.mark.parametrize("act", range(5))
@pytest.mark.parametrize("rows,cols,g,by_rows,dk,pad,fmt", [
    (1, 64, 64, False, BF16, 0, 1), (1, 64, 64, True, F32, 0, 1), (64, 4096, 128, False, BF16, 0, 1),
    (129, 256, 128, False, F32, 8, 0), (300, 512, 256, False, BF16, 8, 1), (65, 192, 64, False, F16, 0, 0),
    (2000, 576, 64, True, BF16, 64, 1), (37, 1280, 256, True, F16, 8, 0), (5, 128, 128, True, F32, 0, 1),
    (513, 1024, 128, False, F16, 0, 1), (700, 640, 64, False, BF16, 0, 0),
    # dbias in a second launch; the last by 512 threads per block, nontemporally
    (1100, 640, 64, False, F16, 8, 1), (1500, 1152, 128, False, BF16, 0, 0), (1300, 1280, 256, False, F32, 0, 1),
    (300, 640, 128, True, BF16, 0, 1), (1030, 1600, 64, True, F32, 4 * 2, 0), (4200, 4096, 128, False, BF16, 0, 1)])
def test_epilogue_backward(dg, act, rows, cols, g, by_rows, dk, pad, fmt):
    dout = ref.stream(rows + cols, rows, cols, dk, zero_rows=(3,)) * 0.01
    pre = (torch.randn(rows, cols, generator=torch.Generator().manual_seed(rows)) * 2).to(BF16)
    pre[0, :9] = torch.tensor([0.0, -0.0, 30.0, -30.0, 5.5, -5.5, 1e4, -1e4, 1e-30], dtype=BF16)
    dz = dout.double() * ref.act_grad(pre.double(), act)
    exact = act in (0, 1)
    bound = (0 if exact else 1) * ACT_ABS * dout.double().abs()
    say("epilogue backward act=%d %dx%d g=%d rows=%d %s pad=%d" % (act, rows, cols, g, by_rows, dk, pad))
    gz = torch.empty(rows, cols, dtype=dk, device=DEV)
    gb = torch.empty(cols, device=DEV)
    br = 1 if by_rows else g
    gpre = ref.padded(pre, pad) if act else None
    q, s = dg.dg_epilogue_backward_fp8(ref.padded(dout, pad), gpre, act, gran=g, block_rows=br, fmt=fmt, dz=gz, dbias=gb)
    torch.cuda.synchronize()
    tiny = 2.0 ** -25 if dk == F16 else 1e-37
    close(gz, dz, bound + ((0 if exact else 2 * ref.U32) + (0 if dk == F32 else ref.half_step(dk)) * 1.01) * dz.abs() + tiny, "dz")
    close(gb, dz.sum(0), bound.sum(0) + (rows + 8) * ref.U32 * dz.abs().sum(0) + 1e-37, "dbias")
    ref.check_codes(q.cpu(), s.cpu(), dz, br, g, fmt, 2 * ref.U32, absolute=float(bound.max()))
    if dk == F32 or exact:  # dz is what the codes are of
        fn = dg.dg_quantize_fp8_rows_typed if by_rows else dg.dg_quantize_fp8_blocks_typed
        qq, ss = fn(gz, gran=g, fmt=fmt)
        assert torch.equal(ss, s) and torch.equal(qq, q)
    q2, s2 = dg.dg_epilogue_backward_fp8(dout.to(DEV), pre.to(DEV) if act else None, act, gran=g, block_rows=br, fmt=fmt)
    assert torch.equal(q2, q) and torch.equal(s2, s)
    over, b2 = dout.to(DEV), torch.empty(cols, device=DEV)
    q3, _ = dg.dg_epilogue_backward_fp8(over, pre.to(DEV) if act else None, act, gran=g, block_rows=br, fmt=fmt, dz=over, dbias=b2)
    assert torch.equal(q3, q) and torch.equal(over, gz) and torch.equal(b2, gb)


@pytest.mark.parametrize("act", range(1, 5))
def test_every_pre_activation(dg, act):
    """act' at every finite BF16 pre-activation."""
    bits = torch.arange(1 << 16, dtype=torch.int32).to(torch.int16).view(BF16)
    pre = torch.where(torch.isfinite(bits), bits, torch.zeros_like(bits)).reshape(256, 256)
    gz = torch.empty(256, 256, device=DEV)
    say("every pre-activation act=%d" % act)
    dg.dg_epilogue_backward_fp8(torch.ones(256, 256, device=DEV), pre.to(DEV), act, dz=gz)
    torch.cuda.synchronize()
    close(gz, ref.act_grad(pre.double(), act), torch.full((256, 256), 1e-12 if act == 1 else ACT_ABS, dtype=torch.float64), "act'")


# ---- the product with a residual -------------------------------------------------

GEMMS = [  # M, N, K, g, tile: every kernel class, ragged edges
    (1, 16, 256, 64, (32, 32)), (64, 4096, 1024, 128, (32, 32)), (50, 523, 2048, 256, (32, 32)),
    (300, 1031, 1024, 128, (64, 64)), (600, 1000, 2048, 64, (64, 64)), (1000, 3000, 512, 64, (128, 128)),
    (777, 3333, 2048, 128, (128, 128)), (4000, 4000, 768, 128, (256, 256)), (3583, 3585, 512, 64, (256, 256)),
    (2000, 4000, 1024, 64, (256, 128)), (2000, 4000, 1024, 128, (256, 128))]


def _operands(M, N, K, g, rowa=False, fa=0, fb=0):
    qa = oracle.quantize_rows_fmt if rowa else oracle.quantize_blocks_fmt
    a8, sa = qa(synth.normal(7100 + M, (M, K)), g, fa)
    b8, sb = oracle.quantize_blocks_fmt(synth.normal(7200 + N, (N, K), sigma=0.02), g, fb)
    return a8, sa, b8, sb


@pytest.mark.parametrize("M,N,K,g,tile", GEMMS)
def test_pre_and_plain_forms_bitwise(dg, M, N, K, g, tile):
    """pre is bf16(C + bias), the plain call's output with that bias, to the bit; without a residual and pre the plain
    call's result; without an activation a residual of zeros changes nothing."""
    t = dg.dg_query_tile(M, N, K, g)
    assert (t["bm"], t["bn"]) == tile, t
    a8, sa, b8, sb = _operands(M, N, K, g)
    ta, tsa, tb, tsb = device_inputs(a8, sa, b8, sb)
    bias = torch.from_numpy(synth.normal(7300 + N, (N,), sigma=0.5).astype(np.float32)).to(DEV)
    say("residual product, plain forms %dx%dx%d g=%d" % (M, N, K, g))
    plain = dg.dg_gemm_fp8_nt_epi(ta, tb, tsa, tsb, gran=g, bias=bias)
    pre = torch.empty_like(plain)
    gelu = dg.dg_gemm_fp8_residual(ta, tb, tsa, tsb, gran=g, bias=bias, act=dg.DG_ACT_GELU, pre=pre)
    assert torch.equal(pre.view(torch.int16), plain.view(torch.int16))
    want = dg.dg_gemm_fp8_nt_epi(ta, tb, tsa, tsb, gran=g, bias=bias, act=dg.DG_ACT_GELU)
    assert torch.equal(gelu.view(torch.int16), want.view(torch.int16))
    same = dg.dg_gemm_fp8_residual(ta, tb, tsa, tsb, gran=g, bias=bias, act=dg.DG_ACT_GELU)
    assert torch.equal(same.view(torch.int16), want.view(torch.int16))
    zeros = torch.zeros(M, N, dtype=F16, device=DEV)
    assert torch.equal(dg.dg_gemm_fp8_residual(ta, tb, tsa, tsb, res=zeros, gran=g, bias=bias), plain)


@pytest.mark.parametrize("act", range(5))
@pytest.mark.parametrize("res_kind,pad", [(BF16, 0), (F32, 8), (F16, 5), (None, 0)])
@pytest.mark.parametrize("M,N,K,g,tile", GEMMS)
def test_residual_closed_form(dg, M, N, K, g, tile, res_kind, pad, act):
    """Operands of ones with power-of-two factors: C is exact, so out is act(C + bias) + residual within the
    activation's own error and one BF16 rounding, and pre is exact in FP32 before its rounding."""
    nkb = K // g
    a8 = torch.full((M, K), 0x38, dtype=torch.uint8, device=DEV)
    b8 = torch.full((N, K), 0x38, dtype=torch.uint8, device=DEV)
    sa = torch.tensor([[2.0 ** ((mb - kb) % 5 - 2) for kb in range(nkb)] for mb in range(-(-M // g))])
    sb = torch.tensor([[2.0 ** ((nb + kb) % 3) for kb in range(nkb)] for nb in range(-(-N // g))]) / (g * nkb)
    # a power of two in place of g * nkb keeps everything exact
    sb = torch.exp2(torch.floor(torch.log2(sb)))
    C = g * (sa.double()[torch.arange(M) // g] @ sb.double()[torch.arange(N) // g].t())
    bias = (torch.arange(N) % 29).float() / 4 - 4.0
    z = C + bias.double()
    res = None if res_kind is None else ref.stream(M + N, M, N, res_kind)
    say("residual closed form act=%d res=%s pad=%d %dx%dx%d g=%d" % (act, res_kind, pad, M, N, K, g))
    pre = torch.empty(M, N, dtype=BF16, device=DEV)
    out = dg.dg_gemm_fp8_residual(a8, b8, sa.float().to(DEV), sb.float().to(DEV), res=None if res is None else ref.padded(res, pad),
                                  gran=g, bias=bias.to(DEV), act=act, pre=pre)
    torch.cuda.synchronize()
    assert torch.equal(pre.cpu(), z.float().to(BF16))
    want = ref.act(z, act) + (0 if res is None else res.double())
    slack = 0.0 if act < 2 else 4e-7  # erf's polynomial (1.5e-7) and roundings, per unit of |z|
    close(out, want, ref.half_step(BF16) * 1.01 * want.abs() + slack * (1 + z.abs()) + 2 * ref.U32 * (z.abs() + want.abs()) + 1e-37, "out")


@pytest.mark.parametrize("layout", range(4))
@pytest.mark.parametrize("rowa", [False, True])
@pytest.mark.parametrize("M,N,K,g,fa,fb", [(33, 1031, 512, 128, 0, 1), (301, 1030, 1024, 64, 1, 0), (1001, 3003, 512, 64, 0, 0),
                                           (777, 3333, 1024, 128, 1, 1), (3583, 3585, 512, 128, 0, 0), (3583, 3585, 512, 64, 0, 0),
                                           (2000, 4000, 512, 256, 0, 1), (2001, 4003, 512, 64, 1, 0)])
def test_residual_layouts_formats_row_factors(dg, M, N, K, g, fa, fb, rowa, layout):
    """Every layout, factor form and format pair: pre equals the plain call's bits, out is bf16(z + residual)."""
    a8, sa, b8, sb = _operands(M, N, K, g, rowa, fa, fb)
    ta, tsa, tb, tsb = device_inputs(a8.T if layout & 2 else a8, sa, b8.T if layout & 1 else b8, sb)
    kw = dict(gran=g, layout=layout, sa_rows=1 if rowa else g, fmt_a=fa, fmt_b=fb)
    res = ref.stream(N, M, N, BF16)
    say("residual layout %d rows=%d %dx%dx%d g=%d fmt=%d,%d" % (layout, rowa, M, N, K, g, fa, fb))
    plain = dg.dg_gemm_fp8_ws(ta, tb, tsa, tsb, **kw)
    pre = torch.empty(M, N, dtype=BF16, device=DEV)
    out = dg.dg_gemm_fp8_residual(ta, tb, tsa, tsb, res=res.to(DEV), pre=pre, **kw)
    torch.cuda.synchronize()
    assert torch.equal(pre.view(torch.int16), plain.view(torch.int16))
    # z is known within half a step of pre
    z = pre.cpu().double()
    want = z + res.double()
    close(out, want, ref.half_step(BF16) * 1.02 * (z.abs() + want.abs()) + 1e-37, "out")


def test_residual_against_the_oracle(dg):
    M, N, K, g = 300, 520, 2048, 128
    a8, sa, b8, sb = _operands(M, N, K, g, rowa=True)
    ta, tsa, tb, tsb = device_inputs(a8, sa, b8, sb)
    res = ref.stream(3, M, N, F32)
    say("residual product against the oracle")
    out = dg.dg_gemm_fp8_residual(ta, tb, tsa, tsb, res=res.to(DEV), gran=g, sa_rows=1, act=dg.DG_ACT_SILU)
    want = ref.act(torch.from_numpy(oracle.gemm_ref_rowa(a8, b8, sa, sb, g)), 3) + res.double()
    ok, _ = _common.within_tolerance(out.float().cpu().numpy(), want.numpy())
    assert ok.all()


@pytest.mark.parametrize("M,N,K", [(5, 300, 512), (300, 1031, 1024), (1000, 3000, 512), (4000, 4000, 512)])
def test_residual_in_place(dg, M, N, K):
    g = 128
    ta, tsa, tb, tsb = device_inputs(*_operands(M, N, K, g))
    res = ref.stream(1, M, N, BF16).to(DEV)
    say("residual in place %dx%dx%d" % (M, N, K))
    out = dg.dg_gemm_fp8_residual(ta, tb, tsa, tsb, res=res, gran=g)
    got = dg.dg_gemm_fp8_residual(ta, tb, tsa, tsb, res=res, out=res, gran=g)
    assert got is res and torch.equal(res, out)


@pytest.mark.parametrize("M,N,K,g,layout", [(19, 51, 12352, 64, 3), (64, 512, 6144, 128, 1), (130, 68, 8192, 256, 2),
                                            (64, 512, 16384, 128, 0), (1, 1, 16384, 64, 0)])
def test_residual_with_a_split_k(dg, M, N, K, g, layout):
    """Few tiles and a long K: pre is the split plain call's output to the bit, out is bf16(act(z) + residual), with the
    workspace left to the call, given, and (without one) unsplit within the product's tolerance."""
    need = dg.dg_gemm_fp8_residual_workspace(M, N, K, g, layout)
    assert need > 0
    a8, sa, b8, sb = _operands(M, N, K, g, rowa=True)
    ta, tsa, tb, tsb = device_inputs(a8.T if layout & 2 else a8, sa, b8.T if layout & 1 else b8, sb)
    kw = dict(gran=g, layout=layout, sa_rows=1, bias=torch.arange(N, device=DEV).float() / N)
    res = ref.stream(N, M, N, F32)
    say("residual split K %dx%dx%d layout %d" % (M, N, K, layout))
    pre, pre2, out2 = (torch.empty(M, N, dtype=BF16, device=DEV) for _ in range(3))
    out = dg.dg_gemm_fp8_residual(ta, tb, tsa, tsb, res=ref.padded(res, 3), pre=pre, act=1, **kw)
    with _common.forced_split(g):
        plain = dg.dg_gemm_fp8_ws(ta, tb, tsa, tsb, workspace=dg.dg_workspace(M, N, K, g, layout), **kw)
    torch.cuda.synchronize()
    assert torch.equal(pre.view(torch.int16), plain.view(torch.int16))
    z = pre.cpu().double()
    want = z.clamp(min=0) + res.double()
    close(out, want, ref.half_step(BF16) * 1.02 * (z.abs() + want.abs()) + 1e-37, "out")
    ws = torch.full((need,), 255, dtype=torch.uint8, device=DEV)
    dg.dg_gemm_fp8_residual(ta, tb, tsa, tsb, res=ref.padded(res, 3), out=out2, pre=pre2, act=1, workspace=ws, **kw)
    assert torch.equal(out2, out) and torch.equal(pre2, pre)
    whole = oracle.gemm_ref_rowa(a8, b8, sa, sb, g) + (np.arange(N) / N)[None, :]
    ok, _ = _common.within_tolerance(pre.float().cpu().numpy(), whole)
    assert ok.all()


def test_residual_race_check_build(dg):
    """The build with extra waits and barriers gives the same bits."""
    lib = dg.load_library(dg.SYNC_LIB_PATH)
    for M, N, K, g in [(50, 523, 2048, 128), (300, 1031, 1024, 64), (777, 3333, 512, 128), (3583, 3585, 512, 128), (2000, 4000, 512, 64)]:
        ta, tsa, tb, tsb = device_inputs(*_operands(M, N, K, g))
        res = ref.stream(1, M, N, BF16).to(DEV)
        pre, out = (torch.empty(M, N, dtype=BF16, device=DEV) for _ in range(2))
        say("residual race check %dx%dx%d" % (M, N, K))
        want = dg.dg_gemm_fp8_residual(ta, tb, tsa, tsb, res=res, gran=g, act=4)
        rc = lib.dg_gemm_fp8_residual(ta.data_ptr(), tb.data_ptr(), tsa.data_ptr(), tsb.data_ptr(), out.data_ptr(), M, N, K, g, 0,
                                      g, 0, 0, None, 4, res.data_ptr(), 1, N, pre.data_ptr(), None, 0,
                                      torch.cuda.current_stream().cuda_stream)
        torch.cuda.synchronize()
        assert rc == 0 and torch.equal(out, want)


# ---- streams, graphs, long offsets ------------------------------------------------


def _layer(dg, t, stream=None):
    """Norm, product with bias and GELU, its gradient, the norm's gradient: outputs into t's buffers."""
    kw = dict(stream=stream)
    dg.dg_rmsnorm_quantize_fp8(t["x"], t["res"], t["w"], h=t["h"], y=t["y"], rstd=t["rstd"], q=t["q"], scales=t["s"], **kw)
    dg.dg_gemm_fp8_residual(t["q"], t["b"], t["s"], t["sb"], t["res2"], t["out"], sa_rows=1, bias=t["bias"], act=2, pre=t["pre"], **kw)
    dg.dg_epilogue_backward_fp8(t["out"], t["pre"], 2, q=t["dq"], scales=t["ds"], dbias=t["db"], workspace=t["ws1"], **kw)
    dg.dg_rmsnorm_backward(t["y"], t["h"], t["rstd"], t["w"], dh=t["x"], dx=t["dx"], dweight=t["dw"], workspace=t["ws2"], **kw)


OUTPUTS = ("h", "y", "rstd", "q", "s", "out", "pre", "dq", "ds", "db", "dx", "dw")


def _buffers(dg, rows, cols, N, seed):
    e = lambda *shape, dtype=F32: torch.empty(*shape, dtype=dtype, device=DEV)  # noqa: E731
    b8, sb = oracle.quantize_blocks(synth.normal(seed, (N, cols), sigma=0.02), 128)
    t = dict(x=ref.stream(seed, rows, cols, BF16).to(DEV), res=ref.stream(seed + 1, rows, cols, BF16).to(DEV), w=weight(cols).to(DEV),
             b=torch.from_numpy(b8).to(DEV), sb=torch.from_numpy(sb).to(DEV), res2=ref.stream(seed + 2, rows, N, BF16).to(DEV),
             bias=torch.randn(N, generator=torch.Generator().manual_seed(seed)).to(DEV))
    t.update(h=e(rows, cols, dtype=BF16), y=e(rows, cols, dtype=BF16), rstd=e(rows), q=e(rows, cols, dtype=torch.uint8),
             s=e(rows, cols // 128), out=e(rows, N, dtype=BF16), pre=e(rows, N, dtype=BF16), dq=e(rows, N, dtype=torch.uint8),
             ds=e(-(-rows // 128), N // 128), db=e(N), dx=e(rows, cols, dtype=BF16), dw=e(cols),
             ws1=e(max(16, dg.dg_epilogue_backward_workspace(rows, N)), dtype=torch.uint8),
             ws2=e(max(16, dg.dg_rmsnorm_backward_workspace(rows, cols)), dtype=torch.uint8))
    return t


def test_graph_replays(dg):
    t = _buffers(dg, 300, 1024, 1280, 11)
    say("layer in a graph")
    _layer(dg, t)
    torch.cuda.synchronize()
    want = {k: t[k].clone() for k in OUTPUTS}
    graph, cap = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    cap.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(cap):
        with torch.cuda.graph(graph, stream=cap):
            _layer(dg, t, cap)
    torch.cuda.synchronize()
    for r in range(4):
        for k in OUTPUTS + ("ws1", "ws2"):
            t[k].zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for k in OUTPUTS:
            assert torch.equal(t[k].view(torch.uint8), want[k].view(torch.uint8)), "replay %d: %s" % (r, k)
        _layer(dg, _buffers(dg, 40, 256, 128, 50 + r))  # eager work between the replays
        torch.cuda.synchronize()


def test_streams_side_by_side(dg):
    sets = [_buffers(dg, 300 + 77 * i, 1024, 1280, 21 + i) for i in range(3)]
    say("layers on three streams")
    want = []
    for t in sets:
        _layer(dg, t)
        torch.cuda.synchronize()
        want.append({k: t[k].clone() for k in OUTPUTS})
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(3):
        for t in sets:
            for k in OUTPUTS:
                t[k].zero_()
        for t, s in zip(sets, streams):
            s.wait_stream(torch.cuda.current_stream())
            _layer(dg, t, s)
        torch.cuda.synchronize()
        for t, w in zip(sets, want):
            for k in OUTPUTS:
                assert torch.equal(t[k].view(torch.uint8), w[k].view(torch.uint8)), k


def test_given_stream_allocates_there(dg):
    """Outputs and workspaces that a call makes itself belong to the stream it runs on."""
    rows, cols = 600, 2048
    dy, h, w = ref.stream(1, rows, cols, BF16).to(DEV), ref.stream(2, rows, cols, BF16).to(DEV), weight(cols).to(DEV)
    rstd = (1 / torch.sqrt(h.float().square().mean(1) + 1e-6)).float()
    say("a given stream")
    want = dg.dg_rmsnorm_backward(dy, h, rstd, w)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        got = dg.dg_rmsnorm_backward(dy, h, rstd, w, stream=s)
        junk = torch.full((8 << 20,), 3.0, device=DEV)  # the current stream reuses its own memory meanwhile
        torch.cuda.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        del junk


def test_current_stream(dg):
    """Without a stream argument a call runs on torch's current stream: it is captured there, and outputs and
    workspaces left to the call (the Python way) or given (the short way) give the same bits."""
    t = _buffers(dg, 200, 512, 640, 31)
    args = (t["y"], t["h"], t["rstd"], t["w"])
    say("the current stream")
    _layer(dg, t)
    torch.cuda.synchronize()
    want = {k: t[k].clone() for k in OUTPUTS}
    for k in OUTPUTS:
        t[k].zero_()
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side), torch.cuda.graph(graph, stream=side):
        _layer(dg, t)
    torch.cuda.synchronize()
    assert not t["q"].any()  # captured, not run
    graph.replay()
    torch.cuda.synchronize()
    for k in OUTPUTS:
        assert torch.equal(t[k].view(torch.uint8), want[k].view(torch.uint8)), k
    dx, dw = dg.dg_rmsnorm_backward(*args, dh=t["x"])
    assert torch.equal(dx, want["dx"]) and torch.equal(dw, want["dw"])
    dw2 = torch.empty_like(dw)
    dx2, _ = dg.dg_rmsnorm_backward(*args, dh=t["x"], dx=torch.empty_like(dx), dweight=dw2)  # the workspace left to the call
    assert torch.equal(dx2, dx) and torch.equal(dw2, dw)


def test_short_way_refuses_the_same(dg):
    """A status from a call whose tensors are right raises; wrong tensors are named by the Python checks."""
    x, w = torch.ones(4, 256, dtype=BF16, device=DEV), torch.ones(256, device=DEV)
    h, q, s = torch.empty_like(x), torch.empty(4, 256, dtype=torch.uint8, device=DEV), torch.empty(4, 2, device=DEV)
    say("refusals on the GPU")
    with pytest.raises(dg.DGArgumentError):
        dg.dg_rmsnorm_quantize_fp8(x, x, w, 1e-6, h=h, q=q, scales=s, y=h)  # two outputs in one place
    with pytest.raises(dg.DGArgumentError):
        dg.dg_rmsnorm_quantize_fp8(x, x, w, -1.0, h=h, q=q, scales=s)
    with pytest.raises(ValueError, match="scales has shape"):
        dg.dg_rmsnorm_quantize_fp8(x, x, w, 1e-6, h=h, q=q, scales=s[:3])
    with pytest.raises(ValueError, match="q has dtype"):
        dg.dg_rmsnorm_quantize_fp8(x, x, w, 1e-6, h=h, q=q.view(torch.float8_e5m2), scales=s)
    with pytest.raises(ValueError, match="weight is on"):
        dg.dg_rmsnorm_quantize_fp8(x, x, w.cpu(), 1e-6, h=h, q=q, scales=s)
    with pytest.raises(dg.DGArgumentError):  # a row pitch that is no multiple of 16 bytes
        wide = torch.ones(4, 257, dtype=BF16, device=DEV)
        dg.dg_rmsnorm_quantize_fp8(wide[:, :256], x, w, 1e-6, h=h, q=q, scales=s)
    many = torch.ones(5000, 256, dtype=BF16, device=DEV)
    with pytest.raises(dg.DGArgumentError):  # a workspace that is too small
        dg.dg_rmsnorm_backward(many, many, torch.ones(5000, device=DEV), w, dx=torch.empty_like(many),
                               dweight=torch.empty_like(w), workspace=torch.empty(64, dtype=torch.uint8, device=DEV))


@pytest.mark.parametrize("rows,cols", [(70000, 512), (36000, 1024), (18000, 2048), (9000, 4096), (4500, 8192), (2300, 16384)])
def test_large_calls_equal_their_parts(dg, rows, cols):
    """A matrix past the size from which data bypasses the caches gives what its row slices, below that size, give."""
    gen = torch.Generator(device=DEV).manual_seed(rows)
    x, res, dy = (torch.randn(rows, cols, generator=gen, device=DEV).to(BF16) for _ in range(3))
    w = weight(cols).to(DEV)
    y, rstd = torch.empty_like(x), torch.empty(rows, device=DEV)
    say("large calls %dx%d" % (rows, cols))
    q, s, h = dg.dg_rmsnorm_quantize_fp8(x, res, w, gran=64, y=y, rstd=rstd)
    dx, dw = dg.dg_rmsnorm_backward(dy, h, rstd, w, dh=res)
    eq, es = dg.dg_epilogue_backward_fp8(dy, x, dg.DG_ACT_SILU, gran=64, block_rows=1)
    bq, bs = dg.dg_epilogue_backward_fp8(dy, x, dg.DG_ACT_SILU, gran=64)
    torch.cuda.synchronize()
    total, size = torch.zeros(cols, dtype=torch.float64, device=DEV), torch.zeros(cols, dtype=torch.float64, device=DEV)
    step = -(-rows // 9 // 64) * 64
    for r in range(0, rows, step):
        at = slice(r, min(r + step, rows))
        py, pr = torch.empty_like(x[at]), torch.empty_like(rstd[at])
        pq, ps, ph = dg.dg_rmsnorm_quantize_fp8(x[at], res[at], w, gran=64, y=py, rstd=pr)
        for got, want in ((pq, q), (ps, s), (ph, h), (py, y), (pr, rstd)):
            assert torch.equal(got, want[at])
        px, _ = dg.dg_rmsnorm_backward(dy[at], h[at], rstd[at], w, dh=res[at])
        assert torch.equal(px, dx[at])
        pq, ps = dg.dg_epilogue_backward_fp8(dy[at], x[at], dg.DG_ACT_SILU, gran=64, block_rows=1)
        assert torch.equal(pq, eq[at]) and torch.equal(ps, es[at])
        pq, ps = dg.dg_epilogue_backward_fp8(dy[at], x[at], dg.DG_ACT_SILU, gran=64)
        assert torch.equal(pq, bq[at]) and torch.equal(ps, bs[r // 64 : r // 64 + ps.shape[0]])
        terms = dy[at].double() * (h[at].double() * rstd[at].double()[:, None])
        total += terms.sum(0)
        size += terms.abs().sum(0)
    # a column's terms are added in chains of at most rows / 64, then by trees of depth below 96
    assert ((dw.double() - total).abs() <= (rows / 64 + 96) * ref.U32 * size).all()


def test_offsets_past_32_bits(dg):
    """More than 2^32 elements: the last rows against the reference on those rows."""
    rows, cols, n = (1 << 19) + 5, 8192, 4
    x = torch.ones(rows, cols, dtype=BF16, device=DEV)
    x[-n:] = ref.stream(9, n, cols, BF16).to(DEV)
    w = weight(cols).to(DEV)
    say("norm of %d elements" % (rows * cols))
    q, s, _ = dg.dg_rmsnorm_quantize_fp8(x, None, w)
    torch.cuda.synchronize()
    _, rstd, y = ref.norm(x[-n:].cpu(), None, w.cpu(), 1e-6)
    ref.check_codes(q[-n:].cpu(), s[-n:].cpu(), y, 1, 128, 0, NORM_REL)
    del s
    full = torch.ones(rows, device=DEV)
    full[-n:] = rstd.float().to(DEV)
    say("norm backward of as many")
    dx, _ = dg.dg_rmsnorm_backward(x, x, full, w)
    torch.cuda.synchronize()
    want, _, bx, _ = ref.norm_bwd(x[-n:].cpu(), x[-n:].cpu(), rstd.float(), w.cpu(), None)
    close(dx[-n:], want, bx * 1.01 + ref.half_step(BF16) * 1.01 * want.abs() + 1e-37, "dx")
    del dx
    say("epilogue backward of as many")
    q, s = dg.dg_epilogue_backward_fp8(x, x, dg.DG_ACT_RELU, q=q, block_rows=1, fmt=0, dbias=torch.empty(cols, device=DEV))
    torch.cuda.synchronize()
    dz = x[-n:].cpu().double() * (x[-n:].cpu().double() > 0)
    ref.check_codes(q[-n:].cpu(), s[-n:].cpu(), dz, 1, 128, 0, 2 * ref.U32)


def test_norm_of_more_threads_than_a_grid_holds(dg):
    """2^22 rows of 1024 threads pass 2^32 threads: further rows go into a second launch."""
    rows, cols, n = (1 << 22) + 3, 4160, 5
    x = torch.ones(rows, cols, dtype=BF16, device=DEV)
    x[-n:] = ref.stream(9, n, cols, BF16).to(DEV)
    w = weight(cols).to(DEV)
    say("norm of %d rows" % rows)
    q, s, _ = dg.dg_rmsnorm_quantize_fp8(x, None, w, gran=64)
    torch.cuda.synchronize()
    _, _, y = ref.norm(x[-n:].cpu(), None, w.cpu(), 1e-6)
    ref.check_codes(q[-n:].cpu(), s[-n:].cpu(), y, 1, 64, 0, NORM_REL)
    assert torch.equal(q[0], q[rows // 2]) and torch.equal(s[0], s[rows - n - 1])

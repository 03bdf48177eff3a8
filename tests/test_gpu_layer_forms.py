"""More forms of the operators around the product on the GPU: the remaining pairs of element types, the residual updated
in place by every tile that reads it early and through a K split, and large calls with FP32 and FP16 operands. Bounds as
in tests/test_gpu_layer.py, from tests/_layer_ref.py."""

import pytest
import torch

from tests import _layer_ref as ref
from tests._gpu import device_inputs, say
from tests.test_gpu_layer import ACT_ABS, NORM_REL, _operands, close, weight

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def dg():
    import fp8_block_scaled_scales_amd as dg

    return dg


# ---- type pairs ------------------------------------------------------------------


@pytest.mark.parametrize("xk,rk", [(F16, F32), (BF16, F16), (F16, BF16), (F32, F16)])
@pytest.mark.parametrize("rows,cols,g,pad", [(1, 64, 64, 0), (5, 832, 64, 8), (33, 2048, 256, 0), (3, 8192, 128, 16), (4, 16384, 64, 0),
                                             (2, 33024, 64, 8)])
def test_norm_type_pairs(dg, rows, cols, g, pad, xk, rk):
    fmt = cols // 64 % 2
    x, res, w = ref.stream(rows + cols, rows, cols, xk, zero_rows=(2,)), ref.stream(rows + 7, rows, cols, rk, zero_rows=(2,)), weight(cols)
    h, rstd, y = ref.norm(x, res, w, 1e-5)
    say("norm type pairs %dx%d %s %s" % (rows, cols, xk, rk))
    gy, gr = torch.empty(rows, cols, dtype=xk, device=DEV), torch.empty(rows, device=DEV)
    q, s, gh = dg.dg_rmsnorm_quantize_fp8(ref.padded(x, pad), ref.padded(res, pad), w.to(DEV), 1e-5, gran=g, fmt=fmt, y=gy, rstd=gr)
    torch.cuda.synchronize()
    assert gh.dtype == rk and torch.equal(gh.cpu(), h)
    close(gr, rstd, 64 * ref.U32 * rstd, "rstd")
    close(gy, y, (NORM_REL + (0 if xk == F32 else ref.half_step(xk))) * 1.01 * y.abs() + (2.0 ** -25 if xk == F16 else 0.0), "y")
    ref.check_codes(q.cpu(), s.cpu(), y, 1, g, fmt, NORM_REL)
    over = res.to(DEV)
    q2, s2, h2 = dg.dg_rmsnorm_quantize_fp8(x.to(DEV), over, w.to(DEV), 1e-5, gran=g, fmt=fmt, h=over)
    assert h2 is over and torch.equal(over, gh) and torch.equal(q2, q) and torch.equal(s2, s)


@pytest.mark.parametrize("dk,hk", [(F32, F16), (BF16, F16), (F16, BF16)])
@pytest.mark.parametrize("rows,cols", [(1, 64), (3, 192), (257, 2048), (19, 8256), (40, 16384), (3, 65536),
                                       (2100, 512), (3200, 2048), (1700, 4096), (900, 8192), (420, 16384)])
def test_norm_backward_type_pairs(dg, rows, cols, dk, hk):
    h, dy, dh = ref.stream(rows, rows, cols, hk), ref.stream(cols, rows, cols, dk), ref.stream(rows + cols, rows, cols, hk)
    w = weight(cols)
    rstd = (1 / torch.sqrt(h.double().square().mean(1) + 1e-6)).float()
    dx, dw, bx, bw = ref.norm_bwd(dy, h, rstd, w, dh)
    say("norm backward type pairs %dx%d %s %s" % (rows, cols, dk, hk))
    gx, gw = dg.dg_rmsnorm_backward(ref.padded(dy, 8), h.to(DEV), rstd.to(DEV), w.to(DEV), dh=ref.padded(dh, 8))
    torch.cuda.synchronize()
    assert gx.dtype == hk
    close(gx, dx, bx * 1.01 + ref.half_step(hk) * 1.01 * dx.abs() + (2.0 ** -25 if hk == F16 else 1e-37), "dx")
    close(gw, dw, bw + ref.U32 * dw.abs() + 1e-37, "dw")


# ---- the residual updated in place -----------------------------------------------


@pytest.mark.parametrize("M,N,K,g,layout,tile", [(2000, 4000, 512, 128, 0, (256, 128)), (2001, 4003, 512, 64, 0, (256, 128)),
                                                 (2000, 4000, 1024, 64, 3, (256, 128)), (777, 3333, 512, 64, 1, (128, 128)),
                                                 (3583, 3585, 512, 64, 2, (256, 256))])
@pytest.mark.parametrize("with_pre", [False, True])
def test_residual_in_place_tiles(dg, M, N, K, g, layout, tile, with_pre):
    t = dg.dg_query_tile(M, N, K, g, layout)
    assert (t["bm"], t["bn"]) == tile, t
    a8, sa, b8, sb = _operands(M, N, K, g)
    ta, tsa, tb, tsb = device_inputs(a8.T if layout & 2 else a8, sa, b8.T if layout & 1 else b8, sb)
    res = ref.stream(1, M, N, BF16).to(DEV)
    pre = torch.empty_like(res) if with_pre else None
    say("residual in place %dx%dx%d layout %d" % (M, N, K, layout))
    want = dg.dg_gemm_fp8_residual(ta, tb, tsa, tsb, res=res, gran=g, layout=layout, act=3, pre=pre)
    want_pre = None if pre is None else pre.clone()
    got = dg.dg_gemm_fp8_residual(ta, tb, tsa, tsb, res=res, out=res, gran=g, layout=layout, act=3, pre=pre)
    assert got is res and torch.equal(res, want) and (pre is None or torch.equal(pre, want_pre))


@pytest.mark.parametrize("M,N,K,g,layout", [(19, 51, 12352, 64, 3), (64, 512, 8192, 128, 0), (130, 68, 8192, 256, 2), (1, 1, 16384, 64, 0)])
def test_residual_in_place_with_a_split_k(dg, M, N, K, g, layout):
    need = dg.dg_gemm_fp8_residual_workspace(M, N, K, g, layout)
    assert need > 0
    a8, sa, b8, sb = _operands(M, N, K, g)
    ta, tsa, tb, tsb = device_inputs(a8.T if layout & 2 else a8, sa, b8.T if layout & 1 else b8, sb)
    res, ws = ref.stream(2, M, N, BF16).to(DEV), torch.full((need,), 255, dtype=torch.uint8, device=DEV)
    say("residual in place, split K %dx%dx%d layout %d" % (M, N, K, layout))
    want = dg.dg_gemm_fp8_residual(ta, tb, tsa, tsb, res=res, gran=g, layout=layout, act=1, workspace=ws)
    got = dg.dg_gemm_fp8_residual(ta, tb, tsa, tsb, res=res, out=res, gran=g, layout=layout, act=1, workspace=ws)
    assert got is res and torch.equal(res, want)


# ---- large calls with FP32 and FP16 operands ---------------------------------------


@pytest.mark.parametrize("xk,rk", [(BF16, F32), (F32, F32), (F16, F16), (F32, BF16)])
@pytest.mark.parametrize("rows,cols", [(4500, 8192), (2300, 16384), (36000, 1024)])
def test_large_norm_equals_its_parts(dg, rows, cols, xk, rk):
    """Past the sizes from which data bypasses the caches (64 MB of inputs, 128 MB backward), against row slices below."""
    gen = torch.Generator(device=DEV).manual_seed(rows)
    x, dy = (torch.randn(rows, cols, generator=gen, device=DEV).to(xk) for _ in range(2))
    res, dh = (torch.randn(rows, cols, generator=gen, device=DEV).to(rk) for _ in range(2))
    w, y, rstd = weight(cols).to(DEV), torch.empty_like(x), torch.empty(rows, device=DEV)
    size = x.element_size() + res.element_size()
    assert rows * cols * size >= 64 << 20 and rows * cols * (size + res.element_size()) >= 128 << 20
    say("large norm %dx%d %s %s" % (rows, cols, xk, rk))
    q, s, h = dg.dg_rmsnorm_quantize_fp8(x, res, w, gran=64, y=y, rstd=rstd)
    dx, dw = dg.dg_rmsnorm_backward(dy, h, rstd, w, dh=dh)
    torch.cuda.synchronize()
    total, mass = torch.zeros(cols, dtype=torch.float64, device=DEV), torch.zeros(cols, dtype=torch.float64, device=DEV)
    step = -(-rows // 12)
    assert step * cols * (size + res.element_size()) < 64 << 20
    for r in range(0, rows, step):
        at = slice(r, min(r + step, rows))
        py, pr = torch.empty_like(x[at]), torch.empty_like(rstd[at])
        pq, ps, ph = dg.dg_rmsnorm_quantize_fp8(x[at], res[at], w, gran=64, y=py, rstd=pr)
        for got, want in ((pq, q), (ps, s), (ph, h), (py, y), (pr, rstd)):
            assert torch.equal(got, want[at])
        px, _ = dg.dg_rmsnorm_backward(dy[at], h[at], rstd[at], w, dh=dh[at])
        assert torch.equal(px, dx[at])
        terms = dy[at].double() * (h[at].double() * rstd[at].double()[:, None])
        total += terms.sum(0)
        mass += terms.abs().sum(0)
    # as in test_large_calls_equal_their_parts: chains of at most rows / 64 terms, then trees of depth below 96
    assert ((dw.double() - total).abs() <= (rows / 64 + 96) * ref.U32 * mass).all()
    # a few rows against the definition
    n = [0, rows // 2, rows - 1]
    hd, rd, yd = ref.norm(x[n].cpu(), res[n].cpu(), w.cpu(), 1e-6)
    assert torch.equal(h[n].cpu(), hd)
    ref.check_codes(q[n].cpu(), s[n].cpu(), yd, 1, 64, 0, NORM_REL)
    want, _, bx, _ = ref.norm_bwd(dy[n].cpu(), hd, rstd[n].cpu(), w.cpu(), dh[n].cpu())
    tiny = 2.0 ** -25 if rk == F16 else 1e-37
    close(dx[n], want, bx * 1.01 + (0 if rk == F32 else ref.half_step(rk)) * 1.01 * want.abs() + tiny, "dx")


@pytest.mark.parametrize("dk", [F32, F16])
@pytest.mark.parametrize("g", [64, 128, 256])
def test_large_epilogue_backward_equals_its_parts(dg, g, dk):
    rows, cols, act = 4500, 8192, 2
    gen = torch.Generator(device=DEV).manual_seed(g)
    dout = (torch.randn(rows, cols, generator=gen, device=DEV) * 0.01).to(dk)
    pre = (torch.randn(rows, cols, generator=gen, device=DEV) * 1.5).to(BF16)
    dz, db = torch.empty_like(dout), torch.empty(cols, device=DEV)
    say("large epilogue backward g=%d %s" % (g, dk))
    q, s = dg.dg_epilogue_backward_fp8(dout, pre, act, gran=g, dz=dz, dbias=db)
    rq, rs = dg.dg_epilogue_backward_fp8(dout, pre, act, gran=g, block_rows=1)
    torch.cuda.synchronize()
    step = 512
    for r in range(0, rows, step):
        at = slice(r, min(r + step, rows))
        pz = torch.empty_like(dz[at])
        pq, ps = dg.dg_epilogue_backward_fp8(dout[at], pre[at], act, gran=g, dz=pz)
        assert torch.equal(pq, q[at]) and torch.equal(pz, dz[at]) and torch.equal(ps, s[r // g : r // g + ps.shape[0]])
        pq, ps = dg.dg_epilogue_backward_fp8(dout[at], pre[at], act, gran=g, block_rows=1)
        assert torch.equal(pq, rq[at]) and torch.equal(ps, rs[at])
    n = [0, rows // 2, rows - 1]
    want = dout[n].cpu().double() * ref.act_grad(pre[n].cpu().double(), act)
    bound = ACT_ABS * dout[n].cpu().double().abs()
    tiny = 2.0 ** -25 if dk == F16 else 1e-37
    close(dz[n], want, bound + (2 * ref.U32 + (0 if dk == F32 else ref.half_step(dk)) * 1.01) * want.abs() + tiny, "dz")
    # dbias: FP32 sums of the FP32 dz, which dz holds rounded once
    exact = dz.double().sum(0)
    room = ((rows + 8) * ref.U32 + (0 if dk == F32 else ref.half_step(dk)) * 1.01) * dz.double().abs().sum(0) + rows * tiny
    assert ((db.double() - exact).abs() <= room).all()

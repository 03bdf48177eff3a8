"""What dg_gemm_fp8_residual promises about the plain calls' bits, with a K
split and without one, on the shapes where the two calls' plans differ: the
residual form splits K from 8192 (6144 transposed), the plain calls from 16384."""

import pytest
import torch

from tests import _common
from tests import _layer_ref as ref

A, B, SA, SB, OUT, WS = ((i + 1) << 40 for i in range(6))  # fake device addresses

# M, N, K, g, layout: the residual form's plan splits K; the last two also the plain plan
SPLITS = [(64, 512, 8192, 128, 0), (19, 51, 12352, 64, 3), (64, 64, 6144, 128, 1), (64, 512, 16384, 128, 0), (33, 96, 16384, 256, 2)]


@pytest.fixture(scope="module")
def dg():
    import fp8_block_scaled_scales_amd as dg

    return dg


@pytest.mark.skipif(torch.cuda.is_available(), reason="an accepted call would launch on these addresses")
@pytest.mark.parametrize("M,N,K,g,layout", SPLITS)
def test_the_plain_form_asks_for_the_plain_workspace(dg, M, N, K, g, layout):
    """Without res and pre a workspace that is enough for dg_gemm_fp8_ws is enough (the call goes on as far as the device,
    which is not there), and one that is too small for it is refused."""
    ws = 256  # far below any split's partial tiles
    need = dg.dg_query_tile(M, N, K, g, layout, workspace=True)["workspace_bytes"]
    assert dg.dg_gemm_fp8_residual_workspace(M, N, K, g, layout) >= max(need, 1)
    for act in (dg.DG_ACT_NONE, dg.DG_ACT_RELU, dg.DG_ACT_GELU):
        want = dg.lib.dg_gemm_fp8_ws(A, B, SA, SB, OUT, M, N, K, g, layout, g, 0, 0, None, act, WS, ws, None)
        got = dg.lib.dg_gemm_fp8_residual(A, B, SA, SB, OUT, M, N, K, g, layout, g, 0, 0, None, act, None, 0, 0, None, WS, ws, None)
        assert got == want and (got == dg.DG_EINVAL) == (need > 0)
    # the residual form still names what it needs
    assert dg.lib.dg_gemm_fp8_residual(A, B, SA, SB, OUT, M, N, K, g, layout, g, 0, 0, None, dg.DG_ACT_SILU, None, 0, 0, None, WS, ws,
                                       None) == dg.DG_EINVAL


def _operands(M, N, K, g, layout, seed):
    gen = torch.Generator(device="cuda:0").manual_seed(seed)
    code = lambda r, c: (torch.randn(r, c, generator=gen, device="cuda:0") * 60).clamp(-448, 448).to(torch.float8_e4m3fn)  # noqa: E731
    factor = lambda r: torch.rand(r, K // g, generator=gen, device="cuda:0") * 0.01 + 0.001  # noqa: E731
    a, b = code(M, K), code(N, K)
    return (a.t().contiguous() if layout & 2 else a, b.t().contiguous() if layout & 1 else b, factor(-(-M // g)), factor(-(-N // g)), a, b)


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K,g,layout", SPLITS + [(64, 512, 4096, 128, 0)])
def test_bits_of_the_plain_calls(dg, M, N, K, g, layout):
    from tests._gpu import say

    a, b, sa, sb, a_nk, b_nk = _operands(M, N, K, g, layout, M + K)
    kw = dict(gran=g, layout=layout, bias=torch.arange(N, device="cuda:0").float() / N)
    res = ref.stream(N, M, N, torch.float32).to("cuda:0")
    none = torch.empty(0, dtype=torch.uint8, device="cuda:0")  # an empty workspace declines the split
    bits = lambda t: t.view(torch.int16)  # noqa: E731
    say("residual contract %dx%dx%d layout %d" % (M, N, K, layout))
    for act in (0, 1, 2):
        plain = dg.dg_gemm_fp8_ws(a, b, sa, sb, act=act, **kw)
        split = dg.dg_gemm_fp8_ws(a, b, sa, sb, act=act, workspace=dg.dg_workspace(M, N, K, g, layout), **kw)
        out = torch.empty_like(plain)
        for o in (None, out):  # outputs left to the call (the Python way) and given (the short way)
            assert torch.equal(bits(dg.dg_gemm_fp8_residual(a, b, sa, sb, out=o, act=act, workspace=none, **kw)), bits(plain))
            assert torch.equal(bits(dg.dg_gemm_fp8_residual(a, b, sa, sb, out=o, act=act, **kw)), bits(split))
    plain = dg.dg_gemm_fp8_ws(a, b, sa, sb, **kw)
    pre, out = torch.empty_like(plain), torch.empty_like(plain)
    for o in (None, out):
        pre.zero_()
        dg.dg_gemm_fp8_residual(a, b, sa, sb, res=res, out=o, pre=pre, act=1, workspace=none, **kw)
        assert torch.equal(bits(pre), bits(plain))  # unsplit: the plain output's bits
    dg.dg_gemm_fp8_residual(a, b, sa, sb, res=res, out=out, pre=pre, act=1, **kw)
    torch.cuda.synchronize()
    # split or not, pre and out are the product's within its parity bar
    spread = lambda s, n: s.repeat_interleave(g, 0)[:n].repeat_interleave(g, 1).double()  # noqa: E731
    z = (a_nk.double() * spread(sa, M)) @ (b_nk.double() * spread(sb, N)).t() + kw["bias"].double()
    for got, want in ((pre, z), (plain, z), (out, z.clamp(min=0) + res.double())):
        ok, _ = _common.within_tolerance(got.float().cpu().numpy(), want.cpu().numpy())
        assert ok.all()

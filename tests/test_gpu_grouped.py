"""The products over groups of rows: every group's rows against the plain product
of those rows, to the bit, on every tile; rows behind the last group untouched;
and the gradient of the weights."""

import pytest
import torch

from tests import _layer_ref as ref
from tests import _route_ref as rr
from tests._gpu import say

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
F32, BF16 = torch.float32, torch.bfloat16
TILES = {64: (7, 3, 1, 10, 5), 128: (6, 2, 0, 9, 4), 256: (6, 2, 0, 9, 4)}  # 32x32, 64x64, 128x128, 256x128, 256x256


@pytest.fixture(scope="module")
def dg():
    import fp8_block_scaled_scales_amd as dg

    return dg


def codes(seed, *shape, fmt=0):
    """Random finite codes, all of the format's values but the largest binades."""
    gen = torch.Generator(device=DEV).manual_seed(seed)
    v = torch.randn(*shape, generator=gen, device=DEV)
    return v.to(ref.F8[fmt]).view(torch.uint8)


def factors(seed, *shape):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    return torch.exp2(torch.randint(-2, 3, shape, generator=gen, device=DEV).float()) * (1 + torch.rand(*shape, generator=gen, device=DEV))


def starts(lengths, align=1):
    off = [0]
    for n in lengths:
        off.append(off[-1] + -(-n // align) * align)
    return off


LENGTHS = [0, 1, 31, 0, 32, 33, 64, 0, 129, 255, 256, 257, 1, 0]


def plain(dg, t, e, lo, hi, tile, monkeypatch, **kw):
    """The group's rows through the plain product on the same tile: (out, pre)."""
    pre = torch.empty(hi - lo, t["out"].shape[1], dtype=BF16, device=DEV)
    sa = t["sa"][lo:hi] if kw["sa_rows"] == 1 else t["sa"][lo // kw["gran"] : -(-hi // kw["gran"])]
    out = dg.dg_gemm_fp8_residual(t["a"][lo:hi], t["b"][e], sa, t["sb"][e], pre=pre, workspace=torch.empty(0, dtype=torch.uint8, device=DEV), **kw)
    return out, pre


@pytest.mark.parametrize("layout", [0, 1])
@pytest.mark.parametrize("blocks", [False, True])
@pytest.mark.parametrize("g,N,K,fa,fb", [(128, 523, 384, 0, 0), (64, 300, 448, 1, 0), (256, 257, 512, 0, 1), (128, 131, 128, 1, 1), (64, 30, 64, 0, 1)])
@pytest.mark.parametrize("which", range(5))
def test_each_group_is_the_plain_product(dg, monkeypatch, which, g, N, K, fa, fb, blocks, layout):
    tile = TILES[g][which]
    off = starts(LENGTHS, g if blocks else 1)
    E, end, rows = len(LENGTHS), off[-1], off[-1] + 300
    t = dict(a=codes(1, rows, K, fmt=fa), b=codes(2, E, K, N, fmt=fb) if layout else codes(2, E, N, K, fmt=fb),
             sa=factors(3, -(-rows // g) if blocks else rows, K // g), sb=factors(4, E, -(-N // g), K // g),
             out=torch.full((rows, N), -77.0, dtype=BF16, device=DEV))
    pre = torch.full((rows, N), -78.0, dtype=BF16, device=DEV)
    kw = dict(gran=g, layout=layout, sa_rows=g if blocks else 1, fmt_a=fa, fmt_b=fb, act=(which + layout) % 5)
    monkeypatch.setenv("DG_FORCE_TILE", str(tile))
    say("grouped tile %d g=%d %dx%d layout %d blocks %d fmt %d,%d" % (tile, g, N, K, layout, blocks, fa, fb))
    offsets = torch.tensor(off, dtype=torch.int32, device=DEV)
    got = dg.dg_gemm_fp8_grouped(t["a"], t["b"], t["sa"], t["sb"], offsets, out=t["out"], pre=pre, **kw)
    torch.cuda.synchronize()
    assert got is t["out"]
    for e in range(E):
        lo, hi = off[e], off[e + 1]
        if hi > lo:
            o, p = plain(dg, t, e, lo, hi, tile, monkeypatch, **kw)
            assert torch.equal(got[lo:hi].view(torch.int16), o.view(torch.int16)), (e, lo, hi)
            assert torch.equal(pre[lo:hi].view(torch.int16), p.view(torch.int16)), (e, lo, hi)
    assert (got[end:] == -77.0).all() and (pre[end:] == -78.0).all()
    again = dg.dg_gemm_fp8_grouped(t["a"], t["b"], t["sa"], t["sb"], offsets, **kw)  # out left to the call, no pre
    assert torch.equal(again[:end].view(torch.int16), got[:end].view(torch.int16))


@pytest.mark.parametrize("E,rows", [(1, 1), (1, 700), (65, 500), (300, 1200), (1024, 3000), (1024, 40)])
def test_many_groups(dg, E, rows):
    """One group to the most of them, empty ones among them, against 64 bits."""
    N, K, g = 200, 256, 128
    ids = rr.routing(E, rows, 1, E, idle=0.1)
    offsets, position, slot = rr.sort(ids, E, 1, rows)
    a, b, sa, sb = codes(1, rows, K), codes(2, E, N, K), factors(3, rows, K // g), factors(4, E, -(-N // g), K // g)
    say("%d groups, %d rows" % (E, rows))
    out = torch.full((rows, N), -3.0, dtype=BF16, device=DEV)
    dg.dg_gemm_fp8_grouped(a, b, sa, sb, offsets.to(DEV), out=out, gran=g, sa_rows=1)
    torch.cuda.synchronize()
    end = int(offsets[-1])
    of = torch.repeat_interleave(torch.arange(E), (offsets[1:] - offsets[:-1]).long()).to(DEV)
    av = a.view(torch.float8_e4m3fn).double() * sa.double().repeat_interleave(g, 1)
    bv = b.view(torch.float8_e4m3fn).double() * sb.double().repeat_interleave(g, 1)[:, :N].repeat_interleave(g, 2)
    want = torch.zeros(end, N, dtype=torch.float64, device=DEV)
    size = torch.zeros_like(want)
    for lo in range(0, end, 256):
        at = slice(lo, min(lo + 256, end))
        want[at] = (bv[of[at]] * av[at][:, None, :]).sum(2)
        size[at] = (bv[of[at]].abs() * av[at].abs()[:, None, :]).sum(2)
    # the matrix instruction adds groups of eight products aligned to the largest (a few 2^-22 of the terms' sizes)
    off = (out[:end].double() - want).abs()
    assert (off <= ref.half_step(BF16) * 1.01 * want.abs() + 1e-5 * size).all(), float(off.max())
    assert (out[end:] == -3.0).all()


def test_offsets_that_make_no_sense(dg):
    """Offsets outside the rows, or that descend, are cut: nothing outside is read or written."""
    N, K, g, rows = 96, 128, 128, 200
    a, b, sa, sb = codes(1, rows, K), codes(2, 4, N, K), factors(3, rows, 1), factors(4, 4, 1, 1)
    for off in ([0, 50, 20, 300, 1 << 30], [-5, -1, 90, 40, 200], [-(1 << 31), (1 << 31) - 1, 0, 0, 0], [200, 200, 200, 200, 200]):
        guard = torch.full((rows + 200, N), -9.0, dtype=BF16, device=DEV)
        say("offsets %s" % off)
        dg.dg_gemm_fp8_grouped(a, b, sa, sb, torch.tensor(off, dtype=torch.int32, device=DEV), out=guard[100 : 100 + rows], gran=g, sa_rows=1)
        torch.cuda.synchronize()
        assert (guard[:100] == -9.0).all() and (guard[100 + rows :] == -9.0).all()


@pytest.mark.parametrize("which", [0, 1])
@pytest.mark.parametrize("g,M,N,fa,fb", [(128, 512, 384, 1, 0), (64, 320, 576, 1, 0), (256, 768, 256, 0, 0), (64, 64, 64, 0, 1), (128, 256, 1152, 1, 1)])
def test_weights_gradient_is_the_plain_product(dg, monkeypatch, g, M, N, fa, fb, which):
    """Every group's gradient against the plain TN product of its rows on the same tile, to the bit; zeros without rows."""
    tile = {64: (1, 5), 128: (0, 4), 256: (0, 4)}[g][which]
    off = starts([0, 1, g, 0, 3 * g, 2 * g + 5, 9 * g, 0], g)
    E, end = len(off) - 1, off[-1]
    rows = end + 2 * g
    a, b = codes(1, rows, M, fmt=fa), codes(2, rows, N, fmt=fb)
    sa, sb = factors(3, rows // g, M // g), factors(4, rows // g, N // g)
    monkeypatch.setenv("DG_FORCE_TILE", str(tile))
    say("weights' gradient tile %d g=%d %dx%d fmt %d,%d" % (tile, g, M, N, fa, fb))
    out = torch.full((E, M, N), -5.0, dtype=BF16, device=DEV)
    dg.dg_gemm_fp8_grouped_wgrad(a, b, sa, sb, torch.tensor(off, dtype=torch.int32, device=DEV), out=out, gran=g, fmt_a=fa, fmt_b=fb)
    torch.cuda.synchronize()
    for e in range(E):
        lo, hi = off[e], off[e + 1]
        if hi == lo:
            assert not out[e].any(), e
        else:
            want = dg.dg_gemm_fp8_layout(a[lo:hi], b[lo:hi], sa[lo // g : hi // g].t().contiguous(), sb[lo // g : hi // g].t().contiguous(), gran=g,
                                         layout=dg.DG_LAYOUT_TN, fmt_a=fa, fmt_b=fb)
            assert torch.equal(out[e].view(torch.int16), want.view(torch.int16)), (e, lo, hi)


def test_weights_gradient_against_64_bits(dg):
    """The default tiles, of a routing with skewed groups, and offsets that make no sense."""
    g, M, N = 128, 384, 256
    ids = rr.routing(1, 900, 2, 9, idle=0.1)
    rows = rr.rows_of(900, 2, 9, g)
    offsets, position, slot = rr.sort(ids, 9, g, rows)
    a, b, sa, sb = codes(1, rows, M, fmt=1), codes(2, rows, N), factors(3, rows // g, M // g), factors(4, rows // g, N // g)
    say("weights' gradient against 64 bits")
    out = dg.dg_gemm_fp8_grouped_wgrad(a, b, sa, sb, offsets.to(DEV))
    av = a.view(torch.float8_e5m2).double() * rr.spread(sa, g, g, rows)
    bv = b.view(torch.float8_e4m3fn).double() * rr.spread(sb, g, g, rows)
    for e in range(9):
        lo, hi = int(offsets[e]), int(offsets[e + 1])
        want, size = av[lo:hi].t() @ bv[lo:hi], av[lo:hi].abs().t() @ bv[lo:hi].abs()
        assert ((out[e].double() - want).abs() <= ref.half_step(BF16) * 1.01 * want.abs() + 1e-5 * size).all(), e
    for off in ([0, 130, 60, 5000, 1 << 30, 1, 2, 3, 4, 5], [-7, 100, 200, 333, rows, rows, rows + 1, -1, 0, 77]):
        say("weights' gradient, offsets %s" % off)
        wild = torch.full((11, M, N), -9.0, dtype=BF16, device=DEV)
        dg.dg_gemm_fp8_grouped_wgrad(a, b, sa, sb, torch.tensor(off, dtype=torch.int32, device=DEV), out=wild[1:10])
        torch.cuda.synchronize()
        assert (wild[0] == -9.0).all() and (wild[10] == -9.0).all()

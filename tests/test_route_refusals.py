"""The calls of experts and adapters on the CPU: bad arguments are refused with
the documented status before any HIP call, the Python functions raise before they
call the library, the size queries, and the references of the GPU tests against
other forms of themselves."""

import ctypes

import pytest
import torch

from tests import _layer_ref as ref
from tests import _route_ref as rr


@pytest.fixture(scope="module")
def dg():
    import fp8_block_scaled_scales_amd as dg

    return dg


# fake device addresses, aligned and 2^40 apart
IDS, OFF, POS, SLOT, WS, X, W, Q, S, Y, RES, OUT, DW, A, B, SA, SB, PRE, SCALE = ((i + 1) << 40 for i in range(19))
MAX = (1 << 24) - 256


def _check(dg, call, kw, want):
    assert call(dg, **kw) == getattr(dg, "DG_" + want)


def _sort(dg, ids=IDS, nb=4, tokens=100, k=2, groups=8, align=16, off=OFF, pos=POS, slot=SLOT, rows=1000, ws=0, wsb=0):
    return dg.lib.dg_route_sort(ids, nb, tokens, k, groups, align, off, pos, slot, rows, ws, wsb, None)


@pytest.mark.parametrize("kw,want", [
    (dict(ids=0), "EINVAL"), (dict(off=0), "EINVAL"), (dict(pos=0), "EINVAL"), (dict(slot=0), "EINVAL"), (dict(nb=2), "EINVAL"),
    (dict(tokens=0), "EINVAL"), (dict(tokens=-1), "EINVAL"), (dict(k=0), "EINVAL"), (dict(k=-2), "EINVAL"), (dict(groups=0), "EINVAL"),
    (dict(groups=1025), "EINVAL"), (dict(align=0), "EINVAL"), (dict(align=-1), "EINVAL"), (dict(rows=319), "EINVAL"), (dict(rows=0), "EINVAL"),
    (dict(rows=1 << 24), "EINVAL"), (dict(tokens=1 << 23, k=2, rows=MAX), "EINVAL"), (dict(tokens=1 << 40, k=1 << 30, rows=MAX), "EINVAL"),
    (dict(tokens=10000, rows=30000), "EINVAL"), (dict(tokens=10000, rows=30000, ws=WS, wsb=64), "EINVAL"), (dict(wsb=-1), "EINVAL"),
    (dict(ids=IDS + 2), "EALIGN"), (dict(ids=IDS + 4, nb=8), "EALIGN"), (dict(off=OFF + 1), "EALIGN"), (dict(pos=POS + 2), "EALIGN"),
    (dict(slot=SLOT + 3), "EALIGN"), (dict(tokens=10000, rows=30000, ws=WS + 8, wsb=1 << 20), "EALIGN"),
    (dict(off=IDS), "EINVAL"), (dict(pos=IDS + 4), "EINVAL"), (dict(slot=POS), "EINVAL"), (dict(off=SLOT + 400), "EINVAL"),
    (dict(tokens=10000, rows=30000, ws=IDS, wsb=1 << 20), "EINVAL"),
])
def test_sort_refuses(dg, kw, want):
    _check(dg, _sort, kw, want)


def _rows(dg, x=X, xk=1, ldx=256, tokens=100, cols=256, k=2, pos=POS, slot=SLOT, rows=512, w=W, g=128, br=128, fmt=0, q=Q, s=S, ws=WS, wsb=1 << 30):
    return dg.lib.dg_route_quantize_fp8(x, xk, ldx, tokens, cols, k, pos, slot, rows, w, g, br, fmt, q, s, ws, wsb, None)


@pytest.mark.parametrize("kw,want", [
    (dict(x=0), "EINVAL"), (dict(pos=0), "EINVAL"), (dict(slot=0), "EINVAL"), (dict(q=0), "EINVAL"), (dict(s=0), "EINVAL"), (dict(xk=3), "EINVAL"),
    (dict(fmt=2), "EINVAL"), (dict(g=96), "EINVAL"), (dict(cols=192, ldx=192), "EINVAL"), (dict(cols=0), "EINVAL"), (dict(tokens=0), "EINVAL"),
    (dict(k=0), "EINVAL"), (dict(rows=0), "EINVAL"), (dict(rows=1 << 24), "EINVAL"), (dict(br=64), "EINVAL"), (dict(br=0), "EINVAL"),
    (dict(ldx=255), "EINVAL"), (dict(ldx=1 << 24), "EINVAL"), (dict(rows=MAX, cols=1 << 16, ldx=1 << 16), "EINVAL"), (dict(wsb=-1, br=1), "EINVAL"),
    (dict(x=X + 8), "EALIGN"), (dict(ldx=260), "EALIGN"), (dict(pos=POS + 2), "EALIGN"), (dict(slot=SLOT + 1), "EALIGN"), (dict(w=W + 2), "EALIGN"),
    (dict(q=Q + 8), "EALIGN"), (dict(s=S + 2), "EALIGN"), (dict(q=X), "EINVAL"), (dict(s=POS), "EINVAL"), (dict(q=SLOT), "EINVAL"), (dict(s=W), "EINVAL"),
    (dict(s=Q + 512), "EINVAL"),
])
def test_rows_refuse(dg, kw, want):
    _check(dg, _rows, kw, want)


def _combine(dg, y=Y, yk=1, ldy=256, rows=512, tokens=100, cols=256, k=2, pos=POS, w=W, res=RES, ldres=256, out=OUT, ok=0):
    return dg.lib.dg_route_combine(y, yk, ldy, rows, tokens, cols, k, pos, w, res, ldres, out, ok, None)


@pytest.mark.parametrize("kw,want", [
    (dict(y=0), "EINVAL"), (dict(pos=0), "EINVAL"), (dict(out=0), "EINVAL"), (dict(yk=3), "EINVAL"), (dict(ok=-1), "EINVAL"), (dict(rows=0), "EINVAL"),
    (dict(tokens=0), "EINVAL"), (dict(k=0), "EINVAL"), (dict(cols=252, ldy=256), "EINVAL"), (dict(cols=0), "EINVAL"), (dict(ldy=255), "EINVAL"),
    (dict(ldres=8), "EINVAL"), (dict(y=Y + 8), "EALIGN"), (dict(ldy=260), "EALIGN"), (dict(res=RES + 4), "EALIGN"), (dict(ldres=257), "EALIGN"),
    (dict(out=OUT + 8), "EALIGN"), (dict(pos=POS + 2), "EALIGN"), (dict(w=W + 1), "EALIGN"), (dict(out=Y), "EINVAL"), (dict(out=POS), "EINVAL"),
    (dict(out=W), "EINVAL"), (dict(out=RES + 16), "EINVAL"), (dict(out=RES, ldres=512), "EINVAL"),
])
def test_combine_refuses(dg, kw, want):
    _check(dg, _combine, kw, want)


def _wgt(dg, x=X, xk=1, ldx=256, y=Y, yk=1, ldy=256, rows=512, tokens=100, cols=256, k=2, pos=POS, dw=DW):
    return dg.lib.dg_route_weight_grad(x, xk, ldx, y, yk, ldy, rows, tokens, cols, k, pos, dw, None)


@pytest.mark.parametrize("kw,want", [
    (dict(x=0), "EINVAL"), (dict(y=0), "EINVAL"), (dict(pos=0), "EINVAL"), (dict(dw=0), "EINVAL"), (dict(xk=3), "EINVAL"), (dict(yk=4), "EINVAL"),
    (dict(rows=0), "EINVAL"), (dict(tokens=0), "EINVAL"), (dict(cols=250), "EINVAL"), (dict(k=0), "EINVAL"), (dict(ldx=8), "EINVAL"),
    (dict(ldy=8), "EINVAL"), (dict(x=X + 8), "EALIGN"), (dict(y=Y + 2), "EALIGN"), (dict(ldx=257), "EALIGN"), (dict(dw=DW + 2), "EALIGN"),
    (dict(pos=POS + 2), "EALIGN"), (dict(dw=X), "EINVAL"), (dict(dw=Y + 64), "EINVAL"), (dict(dw=POS), "EINVAL"),
])
def test_weight_grad_refuses(dg, kw, want):
    _check(dg, _wgt, kw, want)


def _grouped(dg, a=A, b=B, sa=SA, sb=SB, off=OFF, groups=8, out=OUT, rows=512, N=96, K=256, g=128, layout=0, sr=1, fa=0, fb=0, act=2, pre=PRE):
    return dg.lib.dg_gemm_fp8_grouped(a, b, sa, sb, off, groups, out, rows, N, K, g, layout, sr, fa, fb, act, pre or None, None)


@pytest.mark.parametrize("kw,want", [
    (dict(a=0), "EINVAL"), (dict(b=0), "EINVAL"), (dict(sa=0), "EINVAL"), (dict(sb=0), "EINVAL"), (dict(off=0), "EINVAL"), (dict(out=0), "EINVAL"),
    (dict(groups=0), "EINVAL"), (dict(groups=1025), "EINVAL"), (dict(rows=0), "EINVAL"), (dict(N=0), "EINVAL"), (dict(K=192), "EINVAL"),
    (dict(K=0), "EINVAL"), (dict(g=32), "EINVAL"), (dict(layout=2), "EINVAL"), (dict(layout=3), "EINVAL"), (dict(layout=-1), "EINVAL"),
    (dict(sr=64), "EINVAL"), (dict(fa=2), "EINVAL"), (dict(fb=-1), "EINVAL"), (dict(act=5), "EINVAL"), (dict(act=-1), "EINVAL"),
    (dict(rows=MAX, N=MAX), "EINVAL"), (dict(a=A + 8), "EALIGN"), (dict(b=B + 4), "EALIGN"), (dict(sa=SA + 2), "EALIGN"), (dict(sb=SB + 1), "EALIGN"),
    (dict(off=OFF + 2), "EALIGN"), (dict(out=OUT + 1), "EALIGN"), (dict(pre=PRE + 1), "EALIGN"), (dict(out=A), "EINVAL"), (dict(out=B + 100), "EINVAL"),
    (dict(pre=OUT), "EINVAL"), (dict(out=SB), "EINVAL"), (dict(pre=OFF), "EINVAL"),
])
def test_grouped_refuses(dg, kw, want):
    _check(dg, _grouped, kw, want)


def _wgrad(dg, a=A, b=B, sa=SA, sb=SB, off=OFF, groups=8, out=OUT, rows=512, M=256, N=384, g=128, fa=1, fb=0):
    return dg.lib.dg_gemm_fp8_grouped_wgrad(a, b, sa, sb, off, groups, out, rows, M, N, g, fa, fb, None)


@pytest.mark.parametrize("kw,want", [
    (dict(a=0), "EINVAL"), (dict(b=0), "EINVAL"), (dict(sa=0), "EINVAL"), (dict(sb=0), "EINVAL"), (dict(off=0), "EINVAL"), (dict(out=0), "EINVAL"),
    (dict(groups=0), "EINVAL"), (dict(groups=2000), "EINVAL"), (dict(rows=500), "EINVAL"), (dict(rows=0), "EINVAL"), (dict(M=200), "EINVAL"),
    (dict(N=64), "EINVAL"), (dict(g=48), "EINVAL"), (dict(fa=2), "EINVAL"), (dict(fb=2), "EINVAL"), (dict(M=1 << 24), "EINVAL"),
    (dict(M=MAX // 256 * 256, N=MAX // 256 * 256, groups=1024), "EINVAL"), (dict(a=A + 8), "EALIGN"), (dict(b=B + 8), "EALIGN"),
    (dict(sa=SA + 2), "EALIGN"), (dict(sb=SB + 2), "EALIGN"), (dict(off=OFF + 2), "EALIGN"), (dict(out=OUT + 1), "EALIGN"), (dict(out=A), "EINVAL"),
    (dict(out=B), "EINVAL"), (dict(out=SA), "EINVAL"), (dict(out=OFF), "EINVAL"),
])
def test_wgrad_refuses(dg, kw, want):
    _check(dg, _wgrad, kw, want)


def _lora(dg, x=X, xk=1, ldx=256, tokens=64, K=256, a=A, b=B, scale=SCALE, N=96, rank=16, groups=8, off=OFF, pos=POS, slot=SLOT, base=RES, ldb=96,
          out=OUT, ok=1, ws=WS, wsb=1 << 30):
    return dg.lib.dg_lora(x, xk, ldx, tokens, K, a, b, scale, N, rank, groups, off, pos, slot, base, ldb, out, ok, ws, wsb, None)


@pytest.mark.parametrize("kw,want", [
    (dict(x=0), "EINVAL"), (dict(a=0), "EINVAL"), (dict(b=0), "EINVAL"), (dict(off=0), "EINVAL"), (dict(pos=0), "EINVAL"), (dict(slot=0), "EINVAL"),
    (dict(out=0), "EINVAL"), (dict(ws=0), "EINVAL"), (dict(xk=0), "EINVAL"), (dict(xk=3), "EINVAL"), (dict(ok=3), "EINVAL"), (dict(tokens=0), "EINVAL"),
    (dict(K=252, ldx=256), "EINVAL"), (dict(K=0), "EINVAL"), (dict(N=0), "EINVAL"), (dict(rank=0), "EINVAL"), (dict(rank=12), "EINVAL"),
    (dict(rank=136), "EINVAL"), (dict(groups=0), "EINVAL"), (dict(groups=1025), "EINVAL"), (dict(ldx=248), "EINVAL"), (dict(ldb=95), "EINVAL"),
    (dict(wsb=64), "EINVAL"), (dict(wsb=-1), "EINVAL"), (dict(tokens=MAX, N=1 << 20, ldb=1 << 20, wsb=1 << 40), "EINVAL"), (dict(x=X + 8), "EALIGN"),
    (dict(ldx=260), "EALIGN"), (dict(a=A + 8), "EALIGN"), (dict(b=B + 2), "EALIGN"), (dict(scale=SCALE + 2), "EALIGN"), (dict(off=OFF + 2), "EALIGN"),
    (dict(base=RES + 1), "EALIGN"), (dict(out=OUT + 2, ok=0), "EALIGN"), (dict(ws=WS + 8), "EALIGN"), (dict(out=X), "EINVAL"), (dict(out=A), "EINVAL"),
    (dict(ws=X), "EINVAL"), (dict(ws=OUT), "EINVAL"), (dict(out=RES + 2), "EINVAL"), (dict(out=RES, ldb=104), "EINVAL"), (dict(out=SLOT), "EINVAL"),
])
def test_lora_refuses(dg, kw, want):
    _check(dg, _lora, kw, want)


def test_sizes(dg):
    for tokens, k, groups, align in [(1, 1, 1, 1), (1, 8, 64, 1), (100, 2, 8, 16), (8192, 8, 64, 128), (5, 1, 1000, 256), (MAX, 1, 1024, 1)]:
        n = tokens * k
        rows = dg.dg_route_rows(tokens, k, groups, align)
        assert rows == rr.rows_of(tokens, k, groups, align) and rows >= n // align * align and rows % align == 0
        assert 0 <= dg.dg_route_sort_workspace(tokens, k, groups) <= 256 * 4 * groups
    # the worst routing for the rows: every group but one has one slot
    for n, groups, align in [(7, 7, 64), (20, 3, 8), (9, 100, 16), (1000, 10, 128)]:
        ids = torch.tensor([min(i, min(groups, n) - 1) for i in range(n)], dtype=torch.int32)[:, None]
        assert int(rr.sort(ids, groups, align, 1 << 16)[0][-1]) <= dg.dg_route_rows(n, 1, groups, align)
    for bad in [(0, 1, 1, 1), (1, 0, 1, 1), (1, 1, 0, 1), (1, 1, 1025, 1), (1, 1, 1, 0), (MAX, 2, 4, 1), (MAX, 1, 4, 128), (1 << 62, 1 << 30, 4, 1)]:
        with pytest.raises(ValueError):
            dg.dg_route_rows(*bad)
    for bad in [(0, 1, 1), (4, 4, 1025)]:
        with pytest.raises(ValueError):
            dg.dg_route_sort_workspace(*bad)
    for tokens, K, N, rank, groups in [(1, 8, 1, 8, 1), (64, 7168, 4096, 16, 128), (8192, 4096, 4096, 64, 8), (MAX, 4096, 64, 128, 1024)]:
        n = dg.dg_lora_workspace(tokens, K, N, rank, groups)
        assert n > 0 and n % (4 * tokens * rank) == 0 and n <= 64 * tokens * rank
    for bad in [(0, 8, 8, 8, 1), (8, 12, 8, 8, 1), (8, 8, 8, 4, 1), (8, 8, 8, 136, 1), (8, 8, 8, 8, 0)]:
        with pytest.raises(ValueError):
            dg.dg_lora_workspace(*bad)
    assert dg.dg_route_quantize_workspace(100, 256, 2, 512, 128, 1) >= 0
    for bad in [(100, 192, 2, 512, 128, 1), (100, 256, 2, 0, 128, 1), (100, 256, 2, 512, 128, 64), (0, 256, 2, 512, 128, 1)]:
        with pytest.raises(ValueError):
            dg.dg_route_quantize_workspace(*bad)


def test_most_groups_matches_header(dg):
    import os
    import re

    text = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "dg.h")).read()
    assert int(re.search(r"#define DG_MAX_GROUPS (\d+)", text).group(1)) == dg.DG_MAX_GROUPS


def test_every_new_call_is_declared_and_bound(dg):
    for name in ("dg_route_sort", "dg_route_rows", "dg_route_sort_workspace", "dg_route_quantize_fp8", "dg_route_quantize_workspace", "dg_route_combine",
                 "dg_route_weight_grad", "dg_gemm_fp8_grouped", "dg_gemm_fp8_grouped_wgrad", "dg_lora", "dg_lora_workspace"):
        assert isinstance(getattr(dg.lib, name), ctypes._CFuncPtr) and name in dg.__all__


def test_binding_refuses(dg):
    z = torch.zeros
    bf, i32, u8 = torch.bfloat16, torch.int32, torch.uint8
    x, pos, slot, off = z(4, 256, dtype=bf), z(4, 2, dtype=i32), z(16, dtype=i32), z(4, dtype=i32)
    a, b, sa, sb = z(16, 256, dtype=u8), z(3, 32, 256, dtype=u8), z(16, 2), z(3, 1, 2)
    la, lb, lpos, lslot = z(3, 8, 256, dtype=bf), z(3, 32, 8, dtype=bf), z(4, 1, dtype=i32), z(4, dtype=i32)
    for fn, message in [
        (lambda: dg.dg_route_sort(pos, 3), "GPU"),
        (lambda: dg.dg_route_sort(pos.float(), 3), "ids has dtype"),
        (lambda: dg.dg_route_sort(pos[0], 3), "2-D"),
        (lambda: dg.dg_route_sort(pos.t(), 3), "contiguous"),
        (lambda: dg.dg_route_sort(pos, 0), "invalid argument"),
        (lambda: dg.dg_route_sort(pos, 3, 0), "invalid argument"),
        (lambda: dg.dg_route_sort(pos, 3, 128, slot=slot), "at least dg_route_rows"),
        (lambda: dg.dg_route_sort(pos, 3, offsets=off[:3]), "offsets has shape"),
        (lambda: dg.dg_route_sort(pos, 3, position=pos.float()), "position has dtype"),
        (lambda: dg.dg_route_quantize_fp8(x, pos, slot), "GPU"),
        (lambda: dg.dg_route_quantize_fp8(x, pos[:3], slot), "position has shape"),
        (lambda: dg.dg_route_quantize_fp8(x, pos, slot.long()), "slot has dtype"),
        (lambda: dg.dg_route_quantize_fp8(x, pos, slot[:0]), "rows"),
        (lambda: dg.dg_route_quantize_fp8(x, pos, slot, z(4, 3)), "weights has shape"),
        (lambda: dg.dg_route_quantize_fp8(x, pos, slot, z(4, 2, dtype=bf)), "weights has dtype"),
        (lambda: dg.dg_route_quantize_fp8(x, pos, slot, gran=96), "gran"),
        (lambda: dg.dg_route_quantize_fp8(x, pos, slot, block_rows=2), "block_rows"),
        (lambda: dg.dg_route_quantize_fp8(x, pos, slot, fmt=3), "fmt"),
        (lambda: dg.dg_route_quantize_fp8(x.double(), pos, slot), "x has dtype"),
        (lambda: dg.dg_route_quantize_fp8(x, pos, slot, q=z(4, 256, dtype=u8)), "q has shape"),
        (lambda: dg.dg_route_combine(x, pos), "GPU"),
        (lambda: dg.dg_route_combine(x, pos.long()), "position has dtype"),
        (lambda: dg.dg_route_combine(x[:, :100], pos), "multiple of 8"),
        (lambda: dg.dg_route_combine(x[:0], pos), "rows"),
        (lambda: dg.dg_route_combine(x, pos, z(2, 4)), "weights has shape"),
        (lambda: dg.dg_route_combine(x, pos, res=x[:3]), "res has shape"),
        (lambda: dg.dg_route_combine(x, pos, res=x, out=x.float()), "out has dtype"),
        (lambda: dg.dg_route_combine(x, pos, out=x.double()), "out must"),
        (lambda: dg.dg_route_weight_grad(x, x, pos), "GPU"),
        (lambda: dg.dg_route_weight_grad(x, x[:, :64], pos), "y has shape"),
        (lambda: dg.dg_route_weight_grad(x, x, pos[:2]), "position has shape"),
        (lambda: dg.dg_route_weight_grad(x, x, pos, z(4, 2, dtype=bf)), "dweights has dtype"),
        (lambda: dg.dg_gemm_fp8_grouped(a, b, sa, sb, off, sa_rows=1), "GPU"),
        (lambda: dg.dg_gemm_fp8_grouped(a, b, sa, sb, off), "sa has shape"),
        (lambda: dg.dg_gemm_fp8_grouped(a, b, sa, sb, off[:3], sa_rows=1), "b has shape"),
        (lambda: dg.dg_gemm_fp8_grouped(a, b, sa, sb, off.long(), sa_rows=1), "offsets has dtype"),
        (lambda: dg.dg_gemm_fp8_grouped(a, b, sa, sb, off[:1], sa_rows=1), "offsets must"),
        (lambda: dg.dg_gemm_fp8_grouped(a, b[0], sa, sb, off, sa_rows=1), "3-D"),
        (lambda: dg.dg_gemm_fp8_grouped(a, b, sa, sb, off, sa_rows=1, layout=3), "layout"),
        (lambda: dg.dg_gemm_fp8_grouped(a, b, sa, sb, off, sa_rows=1, layout=1), "b has shape"),
        (lambda: dg.dg_gemm_fp8_grouped(a, b, sa, sb[:2], off, sa_rows=1), "sb has shape"),
        (lambda: dg.dg_gemm_fp8_grouped(a, b, sa, sb, off, sa_rows=1, act=9), "act"),
        (lambda: dg.dg_gemm_fp8_grouped(a, b, sa, sb, off, sa_rows=1, pre=z(16, 32)), "pre has dtype"),
        (lambda: dg.dg_gemm_fp8_grouped(a, b, sa, sb, off, sa_rows=1, out=z(16, 31, dtype=bf)), "out has shape"),
        (lambda: dg.dg_gemm_fp8_grouped_wgrad(a, a, sa, sa, off), "gran"),
        (lambda: dg.dg_gemm_fp8_grouped_wgrad(z(128, 256, dtype=u8), z(128, 128, dtype=u8), z(1, 2), z(1, 1), off), "GPU"),
        (lambda: dg.dg_gemm_fp8_grouped_wgrad(z(128, 256, dtype=u8), z(128, 128, dtype=u8), z(2, 1), z(1, 1), off), "sa has shape"),
        (lambda: dg.dg_gemm_fp8_grouped_wgrad(z(128, 256, dtype=u8), z(64, 128, dtype=u8), z(1, 2), z(1, 1), off), "b has shape"),
        (lambda: dg.dg_lora(x, la, lb, off, lpos, lslot), "GPU"),
        (lambda: dg.dg_lora(x.float(), la, lb, off, lpos, lslot), "x has dtype"),
        (lambda: dg.dg_lora(x, la.half(), lb, off, lpos, lslot), "a has dtype"),
        (lambda: dg.dg_lora(x, la[0], lb, off, lpos, lslot), "3-D"),
        (lambda: dg.dg_lora(x, la, lb[:2], off, lpos, lslot), "b has shape"),
        (lambda: dg.dg_lora(x, la, lb, off[:3], lpos, lslot), "a has shape"),
        (lambda: dg.dg_lora(x, la[:, :4], lb, off, lpos, lslot), "a must be|b has shape"),
        (lambda: dg.dg_lora(x, la, lb, off, pos, lslot), "position has shape"),
        (lambda: dg.dg_lora(x, la, lb, off, lpos, slot), "slot has shape"),
        (lambda: dg.dg_lora(x, la, lb, off, lpos, lslot, scale=z(2)), "scale has shape"),
        (lambda: dg.dg_lora(x, la, lb, off, lpos, lslot, base=z(4, 31, dtype=bf)), "base has shape"),
        (lambda: dg.dg_lora(x, la, lb, off, lpos, lslot, base=z(4, 32, dtype=bf), out=z(4, 32)), "out has dtype"),
    ]:
        with pytest.raises(ValueError, match=message):
            fn()


def test_sort_reference_by_counting():
    """The reference against a sort by hand, slot by slot."""
    for seed, tokens, k, groups, align in [(1, 30, 3, 7, 1), (2, 17, 2, 4, 8), (3, 5, 1, 9, 3)]:
        ids = rr.routing(seed, tokens, k, groups, idle=0.2)
        rows = rr.rows_of(tokens, k, groups, align)
        offsets, position, slot = rr.sort(ids, groups, align, rows)
        at = 0
        for e in range(groups):
            assert int(offsets[e]) == at
            for i, v in enumerate(ids.reshape(-1).tolist()):
                if v == e:
                    assert int(position.reshape(-1)[i]) == at and int(slot[at]) == i
                    at += 1
            while at % align:
                assert int(slot[at]) == -1
                at += 1
        assert int(offsets[-1]) == at and (slot[at:] == -2).all()
        assert (position.reshape(-1)[ids.reshape(-1) < 0] == -1).all()


def test_references_against_differences():
    """combine is linear in y and the weights: its differences are the references' gradients."""
    ids = rr.routing(5, 6, 2, 3, idle=0.1)
    _, position, slot = rr.sort(ids, 3, 4, rr.rows_of(6, 2, 3, 4))
    gen = torch.Generator().manual_seed(1)
    y, c = torch.randn(slot.shape[0], 8, generator=gen).double(), torch.randn(6, 8, generator=gen).double()
    w = torch.randn(6, 2, generator=gen).double()
    loss = lambda w, y: float((rr.combine(y, position, w, None)[0] * c).sum())  # noqa: E731
    dw = rr.weight_grad(c, y, position)[0]
    dy = rr.gathered(c.float(), slot, 2, w.float())
    for t in range(6):
        for j in range(2):
            d = torch.zeros_like(w)
            d[t, j] = 1.0
            assert abs(loss(w + d, y) - loss(w, y) - float(dw[t, j])) <= 1e-12 * 100
    for r in range(slot.shape[0]):
        d = torch.zeros_like(y)
        d[r, 3] = 1.0
        assert abs(loss(w, y + d) - loss(w, y) - float(dy[r, 3])) <= 1e-6
    assert ref.U32 == rr.U32


def test_things_that_are_no_tensors(dg):
    z = torch.zeros
    x, pos, slot, off = z(4, 256, dtype=torch.bfloat16), z(4, 2, dtype=torch.int32), z(16, dtype=torch.int32), z(4, dtype=torch.int32)
    for fn in (lambda: dg.dg_route_sort([[0, 1]], 3), lambda: dg.dg_route_sort(pos, 3, slot=[0] * 8), lambda: dg.dg_route_sort(pos, 3, offsets=[0]),
               lambda: dg.dg_route_quantize_fp8(x, pos, [0] * 8), lambda: dg.dg_route_quantize_fp8(x, pos, None), lambda: dg.dg_route_quantize_fp8(x, None, slot),
               lambda: dg.dg_route_combine(x, pos, [1.0]), lambda: dg.dg_route_combine(x, pos, None, 1.0), lambda: dg.dg_route_combine(x, pos, out=1.0),
               lambda: dg.dg_route_weight_grad(x, None, pos), lambda: dg.dg_gemm_fp8_grouped(x, 1, x, x, off), lambda: dg.dg_lora(x, 1, 1, off, pos, slot),
               lambda: dg.dg_lora(x, x, x, None, pos, slot)):
        with pytest.raises((TypeError, ValueError)):
            fn()

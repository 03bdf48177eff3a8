"""More forms of the calls of experts and adapters on the GPU: matrices large enough for the ways that read every token
once and past the caches, more choices than a wave has lanes, streams, two calls at once, the calls without the tensor
binding, and the race check build. Large results against the library's quantisers on the gathered matrix or 64 bits, on
the GPU."""

import ctypes

import pytest
import torch

from tests import _layer_ref as ref
from tests import _route_ref as rr
from tests._gpu import say

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def dg():
    import fp8_block_scaled_scales_amd as dg

    return dg


def normal(seed, *shape, dtype=F32):
    return torch.randn(*shape, generator=torch.Generator(device=DEV).manual_seed(seed), device=DEV).to(dtype)


# ---- large matrices ----------------------------------------------------------------

BY_TOKENS = [(1200, 10, 40, 128, 7168, 128, False, BF16, 0), (1200, 10, 40, 128, 7168, 128, True, BF16, 1), (700, 24, 16, 64, 4160, 64, True, F32, 0),
             (300, 70, 9, 256, 4096, 256, True, F16, 1), (2100, 9, 12, 256, 4352, 256, False, F32, 1), (40, 129, 130, 192, 14400, 64, False, F16, 0),
             (9000, 3, 8, 128, 4096, 128, True, BF16, 1)]


@pytest.mark.parametrize("tokens,k,groups,align,cols,g,weighted,xk,fmt", BY_TOKENS)
def test_large_blocks(dg, tokens, k, groups, align, cols, g, weighted, xk, fmt):
    ids = rr.routing(tokens, tokens, k, groups, idle=0.1)
    ids[tokens // 3] = -1
    off, pos, slot = dg.dg_route_sort(ids.to(DEV), groups, align)
    rows, end = slot.numel(), int(off[-1])
    assert dg.dg_route_quantize_workspace(tokens, cols, k, rows, g, g) > 0  # the way by tokens
    x = normal(cols, tokens, cols + 64)
    x[1] = 0.0
    x = x.to(xk)[:, :cols]
    w = normal(7, tokens, k) if weighted else None
    if weighted:
        w[0, 0], w[2, 1] = 0.0, 1e-30
    say("large blocks %dx%d of %d cols %d g=%d weights=%d %s" % (tokens, k, groups, cols, g, weighted, xk))
    q = torch.full((rows, cols), 0xAB, dtype=torch.uint8, device=DEV)
    s = torch.full((-(-rows // g), cols // g), -5.0, device=DEV)
    dg.dg_route_quantize_fp8(x, pos, slot, w, gran=g, block_rows=g, fmt=fmt, q=q, scales=s)
    at = slot[:end].long()
    v = x[at.clamp(min=0) // k].float()
    if weighted:
        v *= w.reshape(-1)[at.clamp(min=0)][:, None]
    v[at < 0] = 0.0
    wq, ws = dg.dg_quantize_fp8_blocks(v, gran=g, fmt=fmt)
    assert torch.equal(q[:end], wq) and torch.equal(s[: -(-end // g)], ws)
    assert (q[end:] == 0xAB).all() and (s[-(-end // g):] == -5.0).all()


@pytest.mark.parametrize("tokens,k,cols,g,weighted,xk", [(4100, 6, 6144, 128, False, BF16), (4100, 6, 6144, 64, True, BF16), (3300, 3, 8192, 256, True, F32),
                                                         (150, 140, 8192, 64, True, F16), (1000, 65, 2048, 256, False, F32)])
def test_large_rows(dg, tokens, k, cols, g, weighted, xk):
    """A factor per row, more than 128 MB in and out: nontemporal."""
    ids = rr.routing(k, tokens, k, 11, idle=0.1)
    off, pos, slot = dg.dg_route_sort(ids.to(DEV), 11, 8)
    end = int(off[-1])
    x, w = normal(cols, tokens, cols, dtype=xk), normal(7, tokens, k) if weighted else None
    say("large rows %dx%d cols %d g=%d weights=%d %s" % (tokens, k, cols, g, weighted, xk))
    q, s = dg.dg_route_quantize_fp8(x, pos, slot, w, gran=g)
    at = slot[:end].long()
    v = x[at.clamp(min=0) // k].float()
    if weighted:
        v *= w.reshape(-1)[at.clamp(min=0)][:, None]
    v[at < 0] = 0.0
    wq, ws = dg.dg_quantize_fp8_rows(v, gran=g)
    assert torch.equal(q[:end], wq) and torch.equal(s[:end], ws)


@pytest.mark.parametrize("tokens,k,cols,yk,ok", [(4100, 5, 4096, BF16, BF16), (1500, 4, 7168, F32, F32), (300, 67, 4096, F16, BF16)])
def test_large_combine_and_weight_grad(dg, tokens, k, cols, yk, ok):
    """More than 128 MB of rows: nontemporal. Bounds as in test_gpu_route.py."""
    ids = rr.routing(k, tokens, k, 5, idle=0.1)
    off, pos, slot = dg.dg_route_sort(ids.to(DEV), 5)
    y, w, res = normal(1, slot.numel(), cols, dtype=yk), normal(2, tokens, k), normal(3, tokens, cols, dtype=ok)
    assert tokens * k * cols * y.element_size() >= 128 << 20
    y[slot < 0] = float("nan")
    say("large combine %dx%d cols %d %s %s" % (tokens, k, cols, yk, ok))
    out = dg.dg_route_combine(y, pos, w, res)
    dw = dg.dg_route_weight_grad(res, y, pos)
    want, size = res.double(), res.double().abs()
    wdw, sdw = torch.zeros(tokens, k, dtype=torch.float64, device=DEV), torch.zeros(tokens, k, dtype=torch.float64, device=DEV)
    for j in range(k):
        t = torch.nonzero(pos[:, j] >= 0)[:, 0]
        yj = y[pos[t, j].long()].double()
        wdw[t, j], sdw[t, j] = (yj * res[t].double()).sum(1), (yj * res[t].double()).abs().sum(1)
        yj *= w[t, j, None].double()
        want[t] += yj
        size[t] += yj.abs()
    room = (k + 1) * ref.U32 * 1.01 * size + (ref.U32 if ok == F32 else ref.half_step(ok)) * 1.01 * want.abs() + 1e-37
    assert ((out.double() - want).abs() <= room).all()
    assert ((dw.double() - wdw).abs() <= (cols / 256 + 20) * ref.U32 * sdw + ref.U32 * wdw.abs()).all()


@pytest.mark.parametrize("tokens,k,cols,g", [(50, 3, 1024, 128), (50, 3, 1024, 64), (40, 5, 512, 256), (1100, 11, 6400, 128)])
@pytest.mark.parametrize("xk", [BF16, F32])
def test_infinities_and_nan(dg, tokens, k, cols, g, xk):
    """Codes and factors are the quantisers' on the gathered matrix with infinities and NaN of both signs in it and in the
    weights, in one block or row alone and beside finite values; in tokens that no group takes they change nothing."""
    ids = rr.routing(tokens, tokens, k, 6, idle=0.1)
    ids[7] = -1
    x = normal(tokens, tokens, cols)
    x[3, 5], x[4, 70], x[5, 0], x[6, 9], x[7] = float("inf"), float("-inf"), float("nan"), -float("nan"), float("nan")
    x[8], x[9] = float("nan"), float("inf")
    x = x.to(xk)
    w = normal(9, tokens, k)
    w[3, 0], w[10, 0], w[11, 1], w[12, 0], w[9, 0] = 0.0, float("inf"), float("nan"), float("-inf"), 0.0
    off, pos, slot = dg.dg_route_sort(ids.to(DEV), 6, g)
    end = int(off[-1])
    at = slot[:end].long()
    for weights in (None, w):
        v = x[at.clamp(min=0) // k].float()
        if weights is not None:
            v *= w.reshape(-1)[at.clamp(min=0)][:, None]
        v[at < 0] = 0.0
        for fmt in (0, 1):
            say("infinities %dx%d cols %d g=%d %s weights=%d fmt=%d" % (tokens, k, cols, g, xk, weights is not None, fmt))
            for br, plain in ((1, dg.dg_quantize_fp8_rows), (g, dg.dg_quantize_fp8_blocks)):
                q, s = dg.dg_route_quantize_fp8(x, pos, slot, weights, gran=g, block_rows=br, fmt=fmt)
                wq, ws = plain(v, gran=g, fmt=fmt)
                dt = (torch.float8_e4m3fn, torch.float8_e5m2)[fmt]
                got, want = q[:end].view(dt).float(), wq.view(dt).float()
                # a NaN's sign is not held to anything
                assert torch.equal(torch.isnan(got), torch.isnan(want))
                assert torch.equal(torch.where(torch.isnan(want), 0, q[:end]), torch.where(torch.isnan(want), 0, wq))
                assert torch.equal(torch.nan_to_num(s[: ws.shape[0]], 7.0, 8.0), torch.nan_to_num(ws, 7.0, 8.0))


# ---- every call at once --------------------------------------------------------------


class Step:
    """Every call on one routing, its inputs and outputs: sort, rows both ways, products both ways, combine, gradients, adapters."""

    def __init__(self, dg, seed, tokens=600, k=3, groups=9, hidden=512, ffn=384, g=128, adapters=4):
        self.dg, self.g, self.groups, self.adapters = dg, g, groups, adapters
        self.ids = rr.routing(seed, tokens, k, groups, idle=0.1).to(DEV)
        self.which = rr.routing(seed + 1, tokens, 1, adapters, idle=0.2).to(DEV)
        self.x, self.dout = normal(seed, tokens, hidden, dtype=BF16), normal(seed + 2, tokens, hidden, dtype=BF16)
        self.w = torch.rand(tokens, k, generator=torch.Generator().manual_seed(seed)).to(DEV)
        self.w1, self.s1 = dg.dg_quantize_fp8_blocks(normal(1, groups * ffn, hidden), gran=g)
        self.w1, self.s1 = self.w1.reshape(groups, ffn, hidden), self.s1.reshape(groups, ffn // g, hidden // g)
        self.la, self.lb = normal(3, adapters, 16, hidden, dtype=BF16), normal(4, adapters, ffn, 16, dtype=BF16)
        self.scale = torch.rand(adapters, generator=torch.Generator().manual_seed(9)).to(DEV)
        self.s1t = self.s1.transpose(1, 2).contiguous()

    def run(self, stream=None):
        """stream: given to every call; the clears of what calls leave partly unwritten go there too."""
        dg, g = self.dg, self.g

        def zeros(rows, cols):
            with torch.cuda.stream(stream):
                return torch.zeros(rows, cols, dtype=BF16, device=DEV)

        s = dict(stream=stream)
        off, pos, slot = dg.dg_route_sort(self.ids, self.groups, g, **s)
        q, sq = dg.dg_route_quantize_fp8(self.x, pos, slot, gran=g, block_rows=g, **s)
        pre, a, b = (zeros(q.shape[0], self.w1.shape[1]) for _ in range(3))
        r1, t1 = dg.dg_route_quantize_fp8(self.x, pos, slot, self.w, gran=g, fmt=1, **s)
        dg.dg_gemm_fp8_grouped(q, self.w1, sq, self.s1, off, a, gran=g, act=dg.DG_ACT_SILU, pre=pre, **s)
        dg.dg_gemm_fp8_grouped(r1, self.w1, t1, self.s1, off, b, gran=g, sa_rows=1, fmt_a=1, **s)
        out = dg.dg_route_combine(a, pos, self.w, **s)
        d, sd = dg.dg_route_quantize_fp8(out, pos, slot, self.w, gran=g, block_rows=g, fmt=1, **s)
        dx = zeros(*q.shape)
        dg.dg_gemm_fp8_grouped(d, self.w1, sd, self.s1t, off, dx, gran=g, layout=dg.DG_LAYOUT_NN, fmt_a=1, **s)
        dw1 = dg.dg_gemm_fp8_grouped_wgrad(d, q, sd, sq, off, gran=g, **s)
        back = dg.dg_route_combine(dx, pos, None, self.dout, **s)
        dw = dg.dg_route_weight_grad(out, a, pos, **s)
        low = dg.dg_lora(self.x, self.la, self.lb, *dg.dg_route_sort(self.which, self.adapters, **s), self.scale, out, **s)
        return off, pos, slot, a, b, pre, out, dw1, back, dw, low


def same(got, want):
    for i, (a, b) in enumerate(zip(got, want)):
        assert torch.equal(a, b), i


def test_without_the_binding(dg, monkeypatch):
    step = Step(dg, 1)
    say("every call with and without the tensor binding")
    want = step.run()
    monkeypatch.setattr(dg, "_binding", dg._NoBinding)
    same(step.run(), want)


def test_on_other_streams(dg):
    """The current stream, a stream given as an argument, and two streams at once, each with its own routing."""
    one, two = Step(dg, 1), Step(dg, 2, tokens=900)
    say("every call on other streams")
    want = one.run(), two.run()
    torch.cuda.synchronize()
    streams = torch.cuda.Stream(), torch.cuda.Stream()
    with torch.cuda.stream(streams[0]):
        same(one.run(), want[0])
    given = one.run(stream=streams[1])
    torch.cuda.synchronize()
    same(given, want[0])
    got = [], []
    for _ in range(4):
        for i, step in enumerate((one, two)):
            with torch.cuda.stream(streams[i]):
                got[i].append(step.run())
    torch.cuda.synchronize()
    for i in range(2):
        for g in got[i]:
            same(g, want[i])


def test_in_a_graph(dg):
    """Captured once; replayed with other choices, weights and tokens, eager calls between."""
    step, other = Step(dg, 1), Step(dg, 5)
    say("every call in a graph")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step.run()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step.run()
    for i in range(5):
        if i:
            other = Step(dg, 10 + i)
            for n in ("ids", "which", "x", "dout", "w"):
                getattr(step, n).copy_(getattr(other, n))
        want = step.run()
        torch.cuda.synchronize()
        graph.replay()
        other.run()
        torch.cuda.synchronize()
        same(held, want)


# ---- the race check build --------------------------------------------------------------


def _both(dg, outs, call):
    """The outputs that `call(lib)` leaves, from the release and from the race check build, cleared before each."""
    res = []
    for lib in (dg.lib, dg.load_library(dg.SYNC_LIB_PATH)):
        for o in outs:
            o.view(torch.uint8).fill_(0x5A)
        torch.cuda.synchronize()
        rc = call(lib)
        assert rc == 0, lib.dg_strerror(rc)
        torch.cuda.synchronize()
        res.append([o.clone() for o in outs])
    for a, b in zip(*res):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def _empty(*shape, dtype=F32):
    return torch.empty(*shape, dtype=dtype, device=DEV)


@pytest.mark.parametrize("tokens,k,groups,align,cols,g", [(40, 4, 5, 1, 512, 128), (700, 3, 9, 64, 2048, 64), (900, 6, 33, 256, 4096, 256),
                                                          (1200, 10, 40, 128, 7168, 128), (3000, 4, 1024, 1, 1024, 128)])
def test_route_race_check_build(dg, tokens, k, groups, align, cols, g):
    p = lambda t: None if t is None else t.data_ptr()  # noqa: E731
    st = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    ids, rows = rr.routing(tokens, tokens, k, groups, idle=0.1).to(DEV), rr.rows_of(tokens, k, groups, align)
    i32 = torch.int32
    off, pos, slot = _empty(groups + 1, dtype=i32), _empty(tokens, k, dtype=i32), _empty(rows, dtype=i32)
    nb = max(16, dg.dg_route_sort_workspace(tokens, k, groups))
    ws = _empty(nb, dtype=torch.uint8)
    say("route race check %dx%d of %d cols %d" % (tokens, k, groups, cols))
    _both(dg, (off, pos, slot), lambda lib: lib.dg_route_sort(p(ids), 4, tokens, k, groups, align, p(off), p(pos), p(slot), rows, p(ws), nb, st))
    x, w = normal(1, tokens, cols, dtype=BF16), normal(2, tokens, k)
    for br in (1, g):
        q, s = _empty(rows, cols, dtype=torch.uint8), _empty(-(-rows // br), cols // g)
        need = max(16, dg.dg_route_quantize_workspace(tokens, cols, k, rows, g, br))
        qws = _empty(need, dtype=torch.uint8)
        for wt in (None, w):
            _both(dg, (q, s), lambda lib: lib.dg_route_quantize_fp8(p(x), 1, cols, tokens, cols, k, p(pos), p(slot), rows, p(wt), g, br, 0,
                                                                    p(q), p(s), p(qws), need, st))
    y, out, dw = normal(3, rows, cols, dtype=BF16), _empty(tokens, cols, dtype=BF16), _empty(tokens, k)
    _both(dg, (out,), lambda lib: lib.dg_route_combine(p(y), 1, cols, rows, tokens, cols, k, p(pos), p(w), p(x), cols, p(out), 1, st))
    _both(dg, (dw,), lambda lib: lib.dg_route_weight_grad(p(x), 1, cols, p(y), 1, cols, rows, tokens, cols, k, p(pos), p(dw), st))


@pytest.mark.parametrize("g", [64, 128, 256])
@pytest.mark.parametrize("rows,groups,N,K", [(70, 9, 300, 512), (1500, 6, 768, 1024), (6000, 4, 2048, 512), (9000, 3, 4096, 256)])
def test_grouped_race_check_build(dg, rows, groups, N, K, g):
    p = lambda t: None if t is None else t.data_ptr()  # noqa: E731
    st = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    rows = -(-rows // g) * g
    cut = torch.sort(torch.randint(0, rows // g + 1, (groups - 1,), generator=torch.Generator().manual_seed(rows)))[0] * g
    off = torch.cat([torch.zeros(1), cut, torch.tensor([rows])]).to(torch.int32).to(DEV)
    Np = -(-N // g) * g
    a, sa1 = dg.dg_quantize_fp8_rows(normal(1, rows, K), gran=g)
    ab, sab = dg.dg_quantize_fp8_blocks(normal(1, rows, K), gran=g)
    b, sb = dg.dg_quantize_fp8_blocks(normal(2, groups * Np, K), gran=g)
    b = b.reshape(groups, Np, K)[:, :N].contiguous()
    out, pre = _empty(rows, N, dtype=BF16), _empty(rows, N, dtype=BF16)
    say("grouped race check rows %d N %d K %d g=%d" % (rows, N, K, g))
    for x, s, sr, act, keep in ((a, sa1, 1, 2, True), (ab, sab, g, 0, False)):
        _both(dg, (out,) + ((pre,) if keep else ()), lambda lib: lib.dg_gemm_fp8_grouped(
            p(x), p(b), p(s), p(sb), p(off), groups, p(out), rows, N, K, g, 0, sr, 0, 0, act, p(pre) if keep else None, st))
    d, sd = dg.dg_quantize_fp8_blocks(normal(4, rows, Np), gran=g)
    dw = _empty(groups, Np, K, dtype=BF16)
    _both(dg, (dw,), lambda lib: lib.dg_gemm_fp8_grouped_wgrad(p(d), p(ab), p(sd), p(sab), p(off), groups, p(dw), rows, Np, K, g, 0, 0, st))
    dx = _empty(rows, K, dtype=BF16)
    bt = b if N % g == 0 else dg.dg_quantize_fp8_blocks(normal(2, groups * Np, K), gran=g)[0].reshape(groups, Np, K)
    sbt = sb.reshape(groups, Np // g, K // g).transpose(1, 2).contiguous()
    _both(dg, (dx,), lambda lib: lib.dg_gemm_fp8_grouped(p(d), p(bt), p(sd), p(sbt), p(off), groups, p(dx), rows, K, Np, g, 1, g, 0, 0, 0, None, st))


@pytest.mark.parametrize("tokens,groups,N,K,rank", [(64, 128, 1024, 2048, 16), (300, 40, 1000, 712, 8), (2000, 6, 2048, 4096, 64), (3000, 3, 515, 1032, 128)])
@pytest.mark.parametrize("xk", [BF16, F16])
def test_lora_race_check_build(dg, tokens, groups, N, K, rank, xk):
    p = lambda t: None if t is None else t.data_ptr()  # noqa: E731
    st = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    off, pos, slot = dg.dg_route_sort(rr.routing(tokens, tokens, 1, groups, idle=0.1).to(DEV), groups)
    x, a, b = normal(1, tokens, K, dtype=xk), normal(2, groups, rank, K, dtype=xk), normal(3, groups, N, rank, dtype=xk)
    base, scale, kind = normal(4, tokens, N, dtype=F32), torch.rand(groups, device=DEV), {BF16: 1, F16: 2}[xk]
    nb = max(16, dg.dg_lora_workspace(tokens, K, N, rank, groups))
    ws, out = _empty(nb, dtype=torch.uint8), _empty(tokens, N)
    say("adapters' race check %d tokens N %d K %d rank %d %s" % (tokens, N, K, rank, xk))
    _both(dg, (out,), lambda lib: lib.dg_lora(p(x), kind, K, tokens, K, p(a), p(b), p(scale), N, rank, groups, p(off), p(pos), p(slot),
                                              p(base), N, p(out), 0, p(ws), nb, st))


# ---- offsets past 32 bits ----------------------------------------------------------------


def test_products_past_32_bits(dg):
    """Weights of more than 2^32 codes and gradients of more than 2^32 elements: the last groups against the plain calls."""
    groups, N, K, g = 300, 4096, 4096, 128
    assert groups * N * K > 1 << 32
    b = torch.randint(0, 96, (groups, N, K), dtype=torch.uint8, device=DEV)
    sb = torch.rand(groups, N // g, K // g, device=DEV)
    off = torch.zeros(groups + 1, dtype=torch.int32, device=DEV)
    off[-2], off[-1] = 128, 384  # the last two groups' rows, the others have none
    q, s = dg.dg_quantize_fp8_blocks(normal(1, 384, K), gran=g)
    say("groups of %d codes" % b.numel())
    out = dg.dg_gemm_fp8_grouped(q, b, s, sb, off, gran=g)
    back = dg.dg_gemm_fp8_grouped(q, b, s, sb.transpose(1, 2).contiguous(), off, gran=g, layout=dg.DG_LAYOUT_NN)
    for e, lo, hi in ((groups - 2, 0, 128), (groups - 1, 128, 384)):
        at, sat = q[lo:hi], s[lo // g : hi // g]
        for got, want in ((out, dg.dg_gemm_fp8_layout(at, b[e], sat, sb[e], gran=g)),
                          (back, dg.dg_gemm_fp8_layout(at, b[e], sat, sb[e].t().contiguous(), gran=g, layout=dg.DG_LAYOUT_NN))):
            # the plain call may run another tile: the FP32 sums' order differs
            w = want.float()
            assert float((got[lo:hi].float() - w).norm() / w.norm()) <= 2.0 ** -8
    del b, sb
    d, sd = dg.dg_quantize_fp8_blocks(normal(2, 384, N), gran=g)
    dw = dg.dg_gemm_fp8_grouped_wgrad(d, q, sd, s, off, gran=g, fmt_a=0)
    assert not dw[: groups - 2].any()
    for e, lo, hi in ((groups - 2, 0, 128), (groups - 1, 128, 384)):
        want = dg.dg_gemm_fp8_layout(d[lo:hi], q[lo:hi], sd[lo // g : hi // g].t().contiguous(), s[lo // g : hi // g].t().contiguous(), gran=g,
                                     layout=dg.DG_LAYOUT_TN).float()
        assert float((dw[e].float() - want).norm() / want.norm()) <= 2.0 ** -8


def test_adapters_past_32_bits(dg):
    """A and B of more than 2^32 bytes, a base whose rows span more than 2^32 elements: the last rows."""
    groups, rank, K = 1024, 128, 18432
    a = torch.zeros(groups, rank, K, dtype=BF16, device=DEV)
    assert a.numel() * 2 > 1 << 32
    a[-1] = normal(1, rank, K, dtype=BF16)
    b = torch.zeros(groups, K, rank, dtype=BF16, device=DEV)
    b[-1] = normal(2, K, rank, dtype=BF16)
    tokens = 70000
    ids = torch.full((tokens, 1), -1, dtype=torch.int32, device=DEV)
    ids[:40], ids[-3:] = 5, groups - 1
    base = normal(3, tokens, 16, dtype=BF16).repeat(1, 4096)  # [tokens, 65536]
    off, pos, slot = dg.dg_route_sort(ids, groups)
    x = torch.zeros(tokens, K, dtype=BF16, device=DEV)
    x[-3:] = normal(4, 3, K, dtype=BF16)
    say("adapters of %d elements" % a.numel())
    out = dg.dg_lora(x, a, b, off, pos, slot, None, base[:, :K])
    v = x[-3:].double() @ a[-1].double().t()
    want = base[-3:, :K].double() + v @ b[-1].double().t()
    size = base[-3:, :K].double().abs() + x[-3:].double().abs() @ a[-1].double().abs().t() @ b[-1].double().abs().t()
    # FP32 sums of K and of rank terms, v as two BF16 numbers (2^-16 of it), one rounding
    room = (ref.half_step(BF16) * want.abs() + ((K + rank) * ref.U32 + 2.0 ** -16) * size) * 1.01
    assert ((out[-3:].double() - want).abs() <= room).all()
    assert torch.equal(out[:-3], base[:-3, :K])

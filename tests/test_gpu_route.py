"""The sort of rows by group and what moves rows there and back, on the GPU
against tests/_route_ref.py: indices exactly, FP8 rows to the bit against the
quantisers on the gathered matrix, sums within counted FP32 roundings."""

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


def close(got, want, bound, label):
    off = (got.cpu().double() - want).abs()
    bad = ~(off <= bound)
    assert not bad.any(), "%s: %d of %d outside, worst %g of the bound" % (
        label, int(bad.sum()), bad.numel(), float((off / bound.clamp(min=1e-300)).max()))


# one workgroup and several chunks, chunks of more than 4096 slots, waves with a last partial step, one slot, one group,
# a group count that is no power of two, the most groups
SORTS = [(1, 1, 1, 1, 0.0), (1, 8, 64, 1, 0.0), (64, 8, 64, 16, 0.1), (63, 1, 256, 1, 0.5), (1000, 8, 37, 128, 0.0),
         (1024, 8, 128, 1, 0.0), (8193, 1, 5, 64, 0.2), (8192, 8, 64, 128, 0.0), (3001, 6, 1024, 1, 0.3),
         (5000, 2, 1, 256, 0.0), (40000, 8, 160, 3, 0.05), (200003, 6, 1000, 1, 0.0)]


@pytest.mark.parametrize("dtype", [torch.int32, torch.int64])
@pytest.mark.parametrize("tokens,k,groups,align,idle", SORTS)
def test_sort(dg, tokens, k, groups, align, idle, dtype):
    ids = rr.routing(tokens + k, tokens, k, groups, idle, dtype=dtype)
    rows = rr.rows_of(tokens, k, groups, align)
    assert dg.dg_route_rows(tokens, k, groups, align) == rows
    say("sort %dx%d of %d align %d %s" % (tokens, k, groups, align, dtype))
    got = dg.dg_route_sort(ids.to(DEV), groups, align)
    for name, a, b in zip(("offsets", "position", "slot"), got, rr.sort(ids, groups, align, rows)):
        assert a.dtype == torch.int32 and torch.equal(a.cpu(), b), name
    # more rows than needed, outputs that hold other values
    slot = torch.full((rows + 777,), 12345, dtype=torch.int32, device=DEV)
    again = dg.dg_route_sort(ids.to(DEV), groups, align, offsets=torch.full_like(got[0], 9), position=torch.full_like(got[1], 9), slot=slot)
    assert torch.equal(again[0], got[0]) and torch.equal(again[1], got[1])
    assert again[2] is slot and torch.equal(slot[:rows], got[2]) and (slot[rows:] == -2).all()


@pytest.mark.parametrize("n", [5, 20000])
def test_sort_of_strange_indices(dg, n):
    """Values outside 0 .. groups - 1 take their slot out, those that only look inside in their low 32 bits too."""
    for groups in (3, 64):
        ids = torch.arange(n, dtype=torch.int64) % groups
        ids[::5] = torch.tensor([-1, groups, 1 << 32, -(1 << 32) + 1, (1 << 62) + 2]).repeat(n)[: ids[::5].numel()]
        say("strange indices %d of %d" % (n, groups))
        want = rr.sort(ids[:, None], groups, 1, n)
        for a, b in zip(dg.dg_route_sort(ids[:, None].to(DEV), groups), want):
            assert torch.equal(a.cpu(), b)
        small = torch.where((ids < -5) | (ids > 1000), -7, ids).int()
        for a, b in zip(dg.dg_route_sort(small[:, None].to(DEV), groups), want):
            assert torch.equal(a.cpu(), b)
    none = dg.dg_route_sort(torch.full((n, 2), -1, dtype=torch.int32, device=DEV), 7, 64)
    assert not none[0].any() and (none[1] == -1).all() and (none[2] == -2).all()
    one = dg.dg_route_sort(torch.full((n, 2), 6, dtype=torch.int32, device=DEV), 7, 1)
    assert torch.equal(one[1].reshape(-1).cpu(), torch.arange(2 * n, dtype=torch.int32))


QUANTS = [  # tokens, k, groups, align, cols, g, block_rows == g, weights, pitch
    (1, 8, 64, 1, 7168, 128, False, False, 0), (1, 1, 1, 64, 64, 64, True, True, 0), (70, 2, 9, 1, 320, 64, False, True, 8),
    (130, 4, 16, 128, 512, 128, True, False, 0), (130, 4, 16, 128, 512, 128, True, True, 64), (77, 3, 5, 256, 768, 256, True, True, 0),
    (500, 6, 33, 64, 1088, 64, True, False, 0), (300, 2, 8, 16, 1280, 256, False, True, 0), (2000, 2, 8, 64, 2048, 64, False, False, 0),
    (257, 9, 12, 100, 384, 128, False, True, 0), (1500, 8, 64, 128, 1024, 128, True, True, 0)]


@pytest.mark.parametrize("xk", [BF16, F16, F32])
@pytest.mark.parametrize("tokens,k,groups,align,cols,g,blocks,weighted,pad", QUANTS)
def test_rows(dg, tokens, k, groups, align, cols, g, blocks, weighted, pad, xk):
    """Codes and factors are the quantisers' on the gathered FP32 matrix, to the bit; rows behind the last group stay."""
    fmt = (tokens + cols // 64) % 2
    ids = rr.routing(tokens, tokens, k, groups, idle=0.15)
    rows = rr.rows_of(tokens, k, groups, align) + (g if tokens % 2 else 0)
    offsets, position, slot = rr.sort(ids, groups, align, rows)
    x = ref.stream(cols, tokens, cols, xk, zero_rows=(2,))
    w = torch.randn(tokens, k, generator=torch.Generator().manual_seed(3)) if weighted else None
    if weighted:
        w[0, 0] = 0.0
    br = g if blocks else 1
    end = int(offsets[-1])
    v = rr.gathered(x, slot, k, w)
    say("rows %dx%d of %d align %d cols %d g=%d blocks=%d weights=%d %s" % (tokens, k, groups, align, cols, g, blocks, weighted, xk))
    q = torch.full((rows, cols), 0xAB, dtype=torch.uint8, device=DEV)
    s = torch.full((-(-rows // br), cols // g), -5.0, device=DEV)
    dg.dg_route_quantize_fp8(ref.padded(x, pad), position.to(DEV), slot.to(DEV), None if w is None else w.to(DEV), gran=g, block_rows=br,
                             fmt=fmt, q=q, scales=s)
    torch.cuda.synchronize()
    assert (q[end:] == 0xAB).all() and (s[-(-end // br):] == -5.0).all()
    if end:
        wq, ws = (dg.dg_quantize_fp8_blocks if blocks else dg.dg_quantize_fp8_rows)(v[:end].to(DEV), gran=g, fmt=fmt)
        # a product with a weight of zero or a negative one may be a zero of either sign: as the gathered matrix has it
        assert torch.equal(q[:end], wq) and torch.equal(s[: -(-end // br)], ws)
        ref.check_codes(q[:end].cpu(), s[: -(-end // br)].cpu(), v[:end].double(), br, g, fmt, 2 * ref.U32)


def test_rows_with_no_slot_at_all(dg):
    x = torch.ones(4, 256, dtype=BF16, device=DEV)
    off, pos, slot = dg.dg_route_sort(torch.full((4, 2), -1, dtype=torch.int32, device=DEV), 3, 128)
    for br in (1, 128):
        q = torch.full((slot.shape[0], 256), 0xAB, dtype=torch.uint8, device=DEV)
        s = torch.full((-(-slot.shape[0] // br), 2), 3.0, device=DEV)
        say("rows without a slot, block rows %d" % br)
        dg.dg_route_quantize_fp8(x, pos, slot, block_rows=br, q=q, scales=s)
        assert (q == 0xAB).all() and (s == 3.0).all()


def test_indices_outside_are_not_followed(dg):
    """Positions and slots outside the arrays are as if they were not there."""
    x = ref.stream(1, 6, 256, BF16).to(DEV)
    ids = rr.routing(5, 6, 2, 3)
    off, pos, slot = (t.to(DEV) for t in rr.sort(ids, 3, 1, 12))
    bad_pos, bad_slot = pos.clone(), slot.clone()
    gone = int(bad_pos[2, 1])
    bad_pos[2, 1], bad_slot[gone] = 1 << 30, 1 << 30
    y = ref.stream(2, 12, 256, BF16).to(DEV)
    say("indices outside")
    for br in (1, 128):
        q = torch.zeros(12, 256, dtype=torch.uint8, device=DEV)
        s = torch.zeros(-(-12 // br), 2, device=DEV)
        dg.dg_route_quantize_fp8(x, bad_pos, bad_slot, block_rows=br, q=q, scales=s)
        torch.cuda.synchronize()
        assert not q[gone].any()
    want, bound = rr.combine(y.cpu(), torch.where(bad_pos.cpu() > 100, -1, bad_pos.cpu()), None, None)
    close(dg.dg_route_combine(y, bad_pos, out=torch.empty(6, 256, device=DEV)), want, bound + ref.U32 * want.abs(), "out")
    assert float(dg.dg_route_weight_grad(x, y, bad_pos)[2, 1]) == 0.0


COMBINES = [(1, 8, 64, 1, 4096, 0), (1, 1, 1, 1, 8, 0), (64, 8, 64, 1, 4096, 8), (333, 3, 7, 16, 1000, 0), (2000, 2, 8, 64, 7168, 0),
            (129, 13, 20, 1, 264, 16), (900, 8, 64, 128, 2048, 0)]


@pytest.mark.parametrize("yk,ok,weighted,with_res", [(BF16, BF16, True, True), (BF16, F32, True, False), (F32, BF16, False, True),
                                                     (F16, F16, False, False), (F32, F32, True, True), (F16, F32, True, True),
                                                     (BF16, F16, False, False)])
@pytest.mark.parametrize("tokens,k,groups,align,cols,pad", COMBINES)
def test_combine(dg, tokens, k, groups, align, cols, pad, yk, ok, weighted, with_res):
    ids = rr.routing(tokens + cols, tokens, k, groups, idle=0.2)
    ids[tokens // 2] = -1  # a token without any row
    rows = rr.rows_of(tokens, k, groups, align)
    offsets, position, slot = rr.sort(ids, groups, align, rows)
    y = ref.stream(7, rows, cols, F32) * 0.5
    y[slot < 0] = float("nan")  # rows that no slot names may hold anything
    y[int(offsets[-1]):] = float("inf")
    y = y.to(yk)
    w = torch.randn(tokens, k, generator=torch.Generator().manual_seed(4)) if weighted else None
    res = ref.stream(8, tokens, cols, ok) if with_res else None
    want, bound = rr.combine(y, position, w, res)
    say("combine %dx%d of %d cols %d %s -> %s w=%d res=%d" % (tokens, k, groups, cols, yk, ok, weighted, with_res))
    pad = pad * 2 if F32 not in (yk, ok) else pad
    gw = None if w is None else w.to(DEV)
    out = torch.empty(tokens, cols, dtype=ok, device=DEV)
    got = dg.dg_route_combine(ref.padded(y, pad), position.to(DEV), gw, None if res is None else ref.padded(res, pad), out)
    torch.cuda.synchronize()
    assert got is out
    tiny = 2.0 ** -25 if ok == F16 else 1e-37
    close(out, want, bound * 1.01 + (ref.U32 if ok == F32 else ref.half_step(ok)) * 1.01 * want.abs() + tiny, "out")
    if res is not None:
        over = res.to(DEV)
        assert dg.dg_route_combine(y.to(DEV), position.to(DEV), gw, over, over) is over and torch.equal(over, out)


@pytest.mark.parametrize("xk,yk", [(BF16, BF16), (F32, BF16), (F16, F16), (BF16, F32), (F32, F32), (F16, BF16)])
@pytest.mark.parametrize("tokens,k,groups,align,cols,pad", COMBINES)
def test_weight_grad(dg, tokens, k, groups, align, cols, pad, xk, yk):
    ids = rr.routing(tokens + cols + 1, tokens, k, groups, idle=0.2)
    rows = rr.rows_of(tokens, k, groups, align)
    offsets, position, slot = rr.sort(ids, groups, align, rows)
    x, y = ref.stream(1, tokens, cols, xk), ref.stream(2, rows, cols, F32)
    y[slot < 0] = float("nan")
    y = y.to(yk)
    want, bound = rr.weight_grad(x, y, position)
    say("weight gradient %dx%d cols %d %s %s" % (tokens, k, cols, xk, yk))
    dw = torch.full((tokens, k), 7.0, device=DEV)
    dg.dg_route_weight_grad(ref.padded(x, pad), ref.padded(y, pad), position.to(DEV), dw)
    torch.cuda.synchronize()
    close(dw, want, bound + ref.U32 * want.abs() + 1e-37, "dw")
    assert torch.equal(dg.dg_route_weight_grad(x.to(DEV), y.to(DEV), position.to(DEV)), dw)


def test_gradients_against_differences(dg):
    """L = sum(out * c) with out the combine of y: dw by the kernel against differences of the kernel's own L (L is linear in
    the weights, so a difference is exact but for the roundings), and dy = the weighted rows of c within the codes' steps."""
    tokens, k, groups, cols = 9, 3, 4, 512
    ids = rr.routing(3, tokens, k, groups)
    off, pos, slot = (t.to(DEV) for t in rr.sort(ids, groups, 1, tokens * k))
    y, c = ref.stream(1, tokens * k, cols, F32).to(DEV), ref.stream(2, tokens, cols, F32).to(DEV)
    w = torch.rand(tokens, k, generator=torch.Generator().manual_seed(1)).to(DEV)
    say("gradients against differences")
    loss = lambda w, y: float((dg.dg_route_combine(y, pos, w).double() * c.double()).sum())  # noqa: E731
    dw = dg.dg_route_weight_grad(c, y, pos)
    for t, j in [(0, 0), (4, 2), (8, 1)]:
        d = torch.zeros_like(w)
        d[t, j] = 0.5
        size = float((y[pos.long()].abs().sum(1) * c.abs()).sum())
        assert abs((loss(w + d, y) - loss(w - d, y)) - float(dw[t, j])) <= 32 * ref.U32 * size
    q, s = dg.dg_route_quantize_fp8(c, pos, slot, w, fmt=0)
    dy = q.view(torch.float8_e4m3fn).float() * s.repeat_interleave(128, 1)
    for r, col in [(0, 3), (11, 200), (26, 511)]:
        d = torch.zeros_like(y)
        d[r, col] = 64.0
        num = (loss(w, y + d) - loss(w, y - d)) / 128
        assert abs(num - float(dy[r, col])) <= 2.0 ** -4 * abs(num) + float(s[r, col // 128]) * 2.0 ** -10 + 1e-4


def test_dispatch_gradient(dg):
    """combine without weights is the transpose of the dispatch: <rows of x, y> = <x, combine(y)>."""
    tokens, k, groups, cols = 40, 4, 8, 256
    off, pos, slot = rr.sort(rr.routing(3, tokens, k, groups, idle=0.2), groups, 16, rr.rows_of(tokens, k, groups, 16))
    x, y = ref.stream(1, tokens, cols, F32), ref.stream(2, slot.shape[0], cols, F32)
    dx = dg.dg_route_combine(y.to(DEV), pos.to(DEV)).cpu().double()
    v = rr.gathered(x, slot, k, None)
    left = float((v.double() * y.double()).sum())
    assert abs(left - float((dx * x.double()).sum())) <= 8 * ref.U32 * float((v.double() * y.double()).abs().sum())


def test_offsets_past_32_bits(dg):
    """Sorted rows of more than 2^32 elements: the last rows."""
    tokens, k, cols = (1 << 18) + 3, 4, 4608
    rows = tokens * k
    ids = torch.zeros(tokens, k, dtype=torch.int32, device=DEV)
    x = torch.ones(tokens, cols, dtype=BF16, device=DEV)
    x[-2:] = ref.stream(1, 2, cols, BF16).to(DEV)
    say("rows of %d elements" % (rows * cols))
    off, pos, slot = dg.dg_route_sort(ids, 1)
    q, s = dg.dg_route_quantize_fp8(x, pos, slot)
    wq, ws = dg.dg_quantize_fp8_rows_typed(x[-2:].contiguous())
    assert torch.equal(q[-8:], wq.repeat_interleave(k, 0)) and torch.equal(s[-8:], ws.repeat_interleave(k, 0))
    bq, bs = dg.dg_route_quantize_fp8(x, pos, slot, block_rows=128)
    last = rows // 128 * 128
    wq, ws = dg.dg_quantize_fp8_blocks_typed(x[slot[last:].long() // k].contiguous())
    assert torch.equal(bq[last:], wq) and torch.equal(bs[-1:], ws)
    y = torch.zeros(rows, cols, dtype=BF16, device=DEV)
    y[-k:] = x[-1]
    got = dg.dg_route_combine(y, pos)
    assert torch.equal(got[-1], (x[-1].float() * k).to(BF16)) and not got[:-1].any()
    dw = dg.dg_route_weight_grad(x, y, pos)
    assert not dw[:-1].any() and (dw[-1] > 0).all() and torch.equal(dw[-1], dw[-1, :1].expand(k))

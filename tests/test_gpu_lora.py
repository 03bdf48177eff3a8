"""The low-rank adapters of many requests against 64 bits."""

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


def inputs(tokens, K, N, rank, groups, xk, ok, with_base, seed=0):
    gen = torch.Generator().manual_seed(seed + tokens + K)
    x = ref.stream(seed, tokens, K, xk)
    a = (torch.randn(groups, rank, K, generator=gen) / K ** 0.5).to(xk)
    b = (torch.randn(groups, N, rank, generator=gen) / rank ** 0.5).to(xk)
    scale = torch.rand(groups, generator=gen) * 2 - 0.5
    base = ref.stream(seed + 1, tokens, N, ok) if with_base else None
    return x, a, b, scale, base


def check(got, want, size, vsize, K, rank, xk, ok):
    # x A^T: FP32 sums of K products in chains of at most K / 32 matrix instructions of depth below 8, over waves and splits
    # (at most 64 + 8). v enters as two 16-bit numbers, each within half a step (2^-8 of BF16, 2^-11 of FP16): 2^-16 or 2^-22
    # of it is lost, or 2^-24 of the row's largest v where the second number is subnormal in FP16. The second sum has rank
    # terms, of two numbers each.
    first = (K / 32 * 8 + 80) * ref.U32
    second = (2 * rank + 16) * ref.U32 + (2.0 ** -16 if xk == BF16 else 2.0 ** -22)
    bound = (first + second) * size + (2.0 ** -24 * vsize if xk == F16 else 0.0) + 2 * ref.U32 * want.abs()
    bound = bound + (0 if ok == F32 else ref.half_step(ok)) * 1.01 * want.abs() + (2.0 ** -25 if ok == F16 else 1e-37)
    off = (got.cpu().double() - want).abs()
    bad = ~(off <= bound)
    assert not bad.any(), "%d of %d outside, worst %g of the bound" % (int(bad.sum()), bad.numel(), float((off / bound.clamp(min=1e-300)).max()))


CASES = [  # tokens, K, N, rank, adapters, idle: one token; decode; few rows per adapter and many; odd N; every rank class
    (1, 7168, 4096, 16, 4, 0.0), (1, 64, 17, 8, 1, 0.0), (64, 4096, 1024, 16, 64, 0.1), (37, 520, 523, 8, 5, 0.3),
    (200, 1024, 300, 32, 3, 0.0), (500, 776, 255, 64, 7, 0.1), (300, 512, 260, 128, 2, 0.0), (90, 2048, 1030, 104, 40, 0.2),
    (1000, 264, 64, 24, 6, 0.5), (130, 8, 1, 40, 2, 0.0), (33, 3000, 64, 72, 1000, 0.0)]


@pytest.mark.parametrize("xk,ok,with_base", [(BF16, BF16, True), (F16, F16, True), (BF16, F32, True), (BF16, BF16, False), (F16, F32, False), (F16, BF16, True)])
@pytest.mark.parametrize("tokens,K,N,rank,groups,idle", CASES)
def test_lora(dg, tokens, K, N, rank, groups, idle, xk, ok, with_base):
    x, a, b, scale, base = inputs(tokens, K, N, rank, groups, xk, ok, with_base)
    ids = rr.routing(tokens, tokens, 1, groups, idle)
    off, pos, slot = (t.to(DEV) for t in rr.sort(ids, groups, 1, tokens))
    use_scale = None if tokens % 2 else scale
    want, size, vsize = rr.lora(x, a, b, ids[:, 0], use_scale, base)
    say("lora %d tokens K=%d N=%d rank %d of %d %s %s base=%d" % (tokens, K, N, rank, groups, xk, ok, with_base))
    out = torch.full((tokens, N), -99.0, dtype=ok, device=DEV)
    gs = None if use_scale is None else scale.to(DEV)
    args = (a.to(DEV), b.to(DEV), off, pos, slot, gs)
    got = dg.dg_lora(ref.padded(x, 8), *args, None if base is None else ref.padded(base, 3), out)
    torch.cuda.synchronize()
    assert got is out
    check(out, want, size, vsize, K, rank, xk, ok)
    none = torch.nonzero(ids[:, 0] < 0)[:, 0]
    assert torch.equal(out.cpu()[none], torch.zeros(len(none), N, dtype=ok) if base is None else base[none])
    if base is not None:
        over = base.to(DEV)
        assert dg.dg_lora(x.to(DEV), *args, over, over) is over and torch.equal(over, out)  # in place
    ws = torch.full((dg.dg_lora_workspace(tokens, K, N, rank, groups),), 0xFF, dtype=torch.uint8, device=DEV)  # NaN patterns
    again = dg.dg_lora(x.to(DEV), *args, None if base is None else base.to(DEV), torch.empty_like(out), workspace=ws)
    assert torch.equal(again, out)


def test_a_row_does_not_depend_on_others(dg):
    """A token's output is the same bits whatever the other rows of its batch hold, NaN and infinity among them."""
    tokens, K, N, rank, groups = 50, 512, 96, 16, 5
    x, a, b, scale, base = inputs(tokens, K, N, rank, groups, BF16, BF16, True)
    ids = rr.routing(2, tokens, 1, groups)
    off, pos, slot = (t.to(DEV) for t in rr.sort(ids, groups, 1, tokens))
    args = (a.to(DEV), b.to(DEV), off, pos, slot, scale.to(DEV))
    say("rows of a batch")
    want = dg.dg_lora(x.to(DEV), *args, base.to(DEV))
    bad = x.clone()
    bad[::3], bad[1::3] = float("nan"), float("inf")
    got = dg.dg_lora(bad.to(DEV), *args, base.to(DEV))
    assert torch.equal(got[2::3], want[2::3])


def test_large_fp16_products(dg):
    """v beyond FP16's range (x A^T of 1e5 and more) and tiny ones."""
    tokens, K, N, rank = 24, 4096, 64, 16
    x = torch.full((tokens, K), 60.0)
    x[8:16] *= 1e-3
    x[16:] = 0.0
    a = torch.full((1, rank, K), 1.0)
    a[0, 1::2] = 2.0 ** -14
    b = torch.full((1, N, rank), 2.0 ** -12)
    x, a, b = x.to(F16), a.to(F16), b.to(F16)
    ids = torch.zeros(tokens, 1, dtype=torch.int32)
    off, pos, slot = (t.to(DEV) for t in rr.sort(ids, 1, 1, tokens))
    want, size, vsize = rr.lora(x, a, b, ids[:, 0], None, None)
    say("large products in FP16")
    got = dg.dg_lora(x.to(DEV), a.to(DEV), b.to(DEV), off, pos, slot, out=torch.empty(tokens, N, device=DEV))
    check(got, want, size, vsize, K, rank, F16, F32)


def test_indices_outside_are_not_followed(dg):
    tokens, K, N, rank, groups = 20, 128, 64, 8, 3
    x, a, b, scale, base = inputs(tokens, K, N, rank, groups, BF16, BF16, True)
    off, pos, slot = (t.to(DEV) for t in rr.sort(rr.routing(1, tokens, 1, groups), groups, 1, tokens))
    for wild in ([0, 5, 9, 1 << 30], [-9, 30, 2, 20], [(1 << 31) - 1, 0, -(1 << 31), 7]):
        guard = torch.full((tokens + 20, N), -9.0, dtype=BF16, device=DEV)
        bad = slot.clone()
        bad[::4], bad[1::4] = 1 << 30, -5
        say("lora offsets %s" % wild)
        dg.dg_lora(x.to(DEV), a.to(DEV), b.to(DEV), torch.tensor(wild, dtype=torch.int32, device=DEV), pos, bad, base=base.to(DEV), out=guard[10 : 10 + tokens])
        torch.cuda.synchronize()
        assert (guard[:10] == -9.0).all() and (guard[10 + tokens :] == -9.0).all()


@pytest.mark.parametrize("xk", [BF16, F16])
@pytest.mark.parametrize("tokens,K", [(6, 64), (300, 72)])
def test_infinities(dg, tokens, K, xk):
    """A row whose products with A overflow has the infinities of the formula, beside finite ones; other rows are untouched."""
    x, a, b = torch.ones(tokens, K, dtype=xk), torch.zeros(2, 16, K, dtype=xk), torch.ones(2, 40, 16, dtype=xk)
    a[0, 0, 0], a[0, 1, 1], a[1, 3, 2] = 2.0, -3.0, 1.0
    b[0, ::2, 0] = -1.0
    b[0, :, 1] = 0.5
    x[2, 0], x[2, 1] = float("inf"), 60000.0  # v: infinite at rank 0, large at rank 1
    x[3, 4] = float("nan")  # times zeros of A: NaN
    ids = (torch.arange(tokens) % 2).to(torch.int32)[:, None]
    ids[4] = -1
    x[4] = float("nan")  # without an adapter: not read
    base = torch.ones(tokens, 40, dtype=F32)
    off, pos, slot = dg.dg_route_sort(ids.to(DEV), 2)
    say("infinities %d %s" % (tokens, xk))
    out = dg.dg_lora(x.to(DEV), a.to(DEV), b.to(DEV), off, pos, slot, None, base.to(DEV)).cpu()
    want = base.double().clone()
    for t in range(tokens):
        if ids[t, 0] >= 0:
            e = int(ids[t, 0])
            # a rank's product is over the x that its row of A names, but for NaN and infinities times zero
            want[t] += b[e].double() @ (a[e].double() @ x[t].double())
    # an infinite x times the zeros of A's other rows makes those ranks NaN in the formula too
    assert torch.equal(torch.isnan(out), torch.isnan(want)) and torch.equal(torch.isinf(out), torch.isinf(want))
    fine = torch.isfinite(want)
    assert ((out.double() - want).abs()[fine] <= 2.0 ** -20 * want.abs()[fine]).all()


def test_products_past_fp32(dg):
    """v = x A^T past FP32's range without an infinite operand: infinities of the right sign in out."""
    x, a = torch.zeros(5, 64, dtype=BF16), torch.zeros(1, 8, 64, dtype=BF16)
    x[:, 0], x[:, 1], a[0, 0, 0], a[0, 1, 1] = 3e38, 2.0, 4.0, 1.0
    x[1, 0], x[2, 0] = 1.0, -3e38
    b = torch.ones(1, 24, 8, dtype=BF16)
    b[0, :, 1] = -1e30
    off, pos, slot = dg.dg_route_sort(torch.zeros(5, 1, dtype=torch.int32, device=DEV), 1)
    say("products past FP32")
    for ok in (BF16, F32):
        out = dg.dg_lora(x.to(DEV), a.to(DEV), b.to(DEV), off, pos, slot, None, torch.zeros(5, 24, dtype=ok, device=DEV)).cpu().float()
        assert (out[[0, 3, 4]] == float("inf")).all() and (out[2] == -float("inf")).all() and torch.isfinite(out[1]).all()

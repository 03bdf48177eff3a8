"""The adapters where their numbers end: elements of a row far below its largest,
products and scales near FP32's ends, positions outside the rows, infinities in B."""

import pytest
import torch

from tests import _layer_ref as ref
from tests._gpu import say

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def dg():
    import fp8_block_scaled_scales_amd as dg

    return dg


def mantissas(seed, *shape):
    """Numbers of 11 bits in [1, 2), exact in FP16."""
    return torch.randint(1024, 2048, shape, generator=torch.Generator().manual_seed(seed)).double() / 1024


def adapter(dg, x, a, b, scale=None, out=F32):
    """dg_lora of one adapter for all rows, without a base; x, a, b in 64 bits, exact in FP16."""
    x, a, b = (t.to(F16).to(DEV) for t in (x, a, b))
    off, pos, slot = dg.dg_route_sort(torch.zeros(x.shape[0], 1, dtype=torch.int32, device=DEV), 1)
    gs = None if scale is None else torch.tensor([scale], device=DEV)
    return dg.dg_lora(x, a[None], b[None], off, pos, slot, gs, out=torch.empty(x.shape[0], b.shape[0], dtype=out, device=DEV)).cpu().double()


@pytest.mark.parametrize("rank", [24, 32, 72])
@pytest.mark.parametrize("tokens", [5, 200])
def test_small_elements_of_an_fp16_row(dg, tokens, rank):
    """Every element of x A^T alone in an output, 22 bits each, from the row's largest to 2^-23 of it and below."""
    # v[t, r] = 2^(15 - r) (m0 + 2^-11 m1), the largest at rank 0; ranks from 30 on are zero
    live = 30 if rank > 30 else rank
    m = mantissas(rank + tokens, tokens, 2, live)
    down = 2.0 ** -torch.arange(live).double()
    x, a = torch.zeros(tokens, 2 * rank + 16, dtype=torch.float64), torch.zeros(rank, 2 * rank + 16, dtype=torch.float64)
    half = down.sqrt().log2().floor().exp2()  # the way down is shared by x and A
    x[:, 0 : 2 * live : 2], x[:, 1 : 2 * live : 2] = m[:, 0] * half * 2.0 ** 7, m[:, 1] * half * 2.0 ** 7
    rest = down / half * 2.0 ** 8
    for r in range(live):
        a[r, 2 * r], a[r, 2 * r + 1] = rest[r], rest[r] * 2.0 ** -11
    for t in (x, a):
        assert torch.equal(t.to(F16).double(), t)
    want = torch.zeros(tokens, rank, dtype=torch.float64)
    want[:, :live] = x @ a[:live].t()
    say("small elements of %d FP16 rows, rank %d" % (tokens, rank))
    got = adapter(dg, x, a, torch.eye(rank).double())
    # A row is scaled to a largest element in [2^14, 2^15). The first FP16 number is within 2^-11 of an element, the second
    # within 2^-11 of what is left or, where it is subnormal, half a step of 2^-24: 2^-25 / 2^14 of the largest. Both products
    # with one are exact, their FP32 sum rounds once.
    top = want.abs().amax(1, keepdim=True)
    bound = torch.maximum(2.0 ** -22 * want.abs(), 2.0 ** -39 * top) + ref.U32 * 1.01 * want.abs()
    assert ((got - want).abs() <= bound).all()
    # what dg_lora promises: 16 bits of every element of at least 2^-23 of its row's largest
    held = want.abs() >= 2.0 ** -23 * top
    assert int(held.sum()) >= 23 * tokens and ((got - want).abs() <= 2.0 ** -16 * 1.01 * want.abs())[held].all()


@pytest.mark.parametrize("tokens", [5, 200])
@pytest.mark.parametrize("xe,ae,se,be", [(-14, -10, -101, 0), (-14, -10, -102, 3), (14, 14, 90, -14), (14, 14, 95, -12), (0, 0, 0, 0)])
def test_scales_near_the_ends_of_fp32(dg, tokens, xe, ae, se, be):
    """x A^T times the adapter's scale is held where FP32 holds it, far outside FP16's range."""
    rank = 16
    m = mantissas(tokens, tokens, 2, rank)
    x, a = torch.zeros(tokens, 64, dtype=torch.float64), torch.zeros(rank, 64, dtype=torch.float64)
    x[:, 0:32:2], x[:, 1:32:2] = m[:, 0] * 2.0 ** xe, m[:, 1] * 2.0 ** xe
    for r in range(rank):
        a[r, 2 * r], a[r, 2 * r + 1] = 2.0 ** ae, 2.0 ** (ae - 11)
    b = torch.eye(rank).double() * 2.0 ** be
    want = 2.0 ** se * (x @ a.t()) * 2.0 ** be
    say("scale 2^%d of products 2^%d" % (se, xe + ae))
    got = adapter(dg, x, a, b, scale=2.0 ** se)
    # elements within a factor of two of the row's largest: both numbers normal, 2^-22; the sum rounds once, in FP32's normal
    # range (2^-126 and more)
    assert float(want.abs().min()) >= 2.0 ** -126 and ((got - want).abs() <= (2.0 ** -22 + ref.U32) * 1.01 * want.abs()).all()


@pytest.mark.parametrize("with_base", [True, False])
@pytest.mark.parametrize("tokens,groups", [(20, 3), (300, 2)])
def test_positions_outside_have_no_adapter(dg, tokens, groups, with_base):
    """A row whose position is not in 0 .. tokens - 1 is base alone, whatever the value."""
    K, N, rank = 128, 70, 16
    gen = torch.Generator().manual_seed(tokens)
    r = lambda *shape: torch.randn(*shape, generator=gen).to(BF16).to(DEV)  # noqa: E731
    x, a, b, base = r(tokens, K), r(groups, rank, K), r(groups, N, rank), r(tokens, N) if with_base else None
    ids = (torch.arange(tokens, dtype=torch.int32) % groups)[:, None]
    ids[::4] = -1
    off, pos, slot = dg.dg_route_sort(ids.to(DEV), groups)
    say("positions outside, %d tokens base=%d" % (tokens, with_base))
    want = dg.dg_lora(x, a, b, off, pos, slot, None, base, torch.full((tokens, N), -99.0, dtype=BF16, device=DEV))
    assert torch.equal(want[::4], torch.zeros_like(want[::4]) if base is None else base[::4])
    for value in (tokens, tokens + 1, 1 << 30, (1 << 31) - 1, -(1 << 31)):
        other = pos.clone()
        other[::4] = value
        out = torch.full((tokens, N), -99.0, dtype=BF16, device=DEV)
        assert torch.equal(dg.dg_lora(x, a, b, off, other, slot, None, base, out), want), value


@pytest.mark.parametrize("ok", [F32, BF16])
@pytest.mark.parametrize("tokens", [5, 200])
def test_products_between_the_largest_bf16_and_fp32(dg, tokens, ok):
    """Finite elements of x A^T that round to an infinity in BF16 stay finite in out where the formula's sum is."""
    x, a = torch.zeros(tokens, 64, dtype=BF16), torch.zeros(1, 8, 64, dtype=BF16)
    big = torch.finfo(BF16).max  # 3.39e38
    x[:, 0], x[:, 1], a[0, :, 0] = big, 1.0, 1.0
    for r, v in enumerate((1.0, 6e35, 7e35, 1e36, 1.2e36, 0.0, 1e30, 6.7e35)):  # half a step past the largest is 6.65e35
        a[0, r, 1] = v
    x[1::3] *= -1
    b = torch.zeros(1, 24, 8, dtype=BF16)
    b[0, :8], b[0, 8:16], b[0, 16:] = torch.eye(8) * 0.5, torch.eye(8) * -0.25, torch.eye(8) * 2.0 ** -100
    v = x.double() @ a[0].double().t()
    assert float(v.abs().max()) <= torch.finfo(F32).max
    off, pos, slot = dg.dg_route_sort(torch.zeros(tokens, 1, dtype=torch.int32, device=DEV), 1)
    say("products past the largest BF16, %d rows" % tokens)
    out = dg.dg_lora(x.to(DEV), a.to(DEV), b.to(DEV), off, pos, slot, out=torch.empty(tokens, 24, dtype=ok, device=DEV)).cpu().double()
    want = v @ b[0].double().t()
    # two BF16 numbers (2^-16), FP32 roundings of x A^T and of the sum, one of out
    room = (2.0 ** -16 + 3 * ref.U32 + (0.0 if ok == F32 else ref.half_step(BF16))) * 1.01 * want.abs()
    assert ((out - want).abs() <= room).all()


@pytest.mark.parametrize("xk", [BF16, F16])
@pytest.mark.parametrize("ok", [F32, BF16])
@pytest.mark.parametrize("tokens,rank", [(5, 8), (5, 32), (200, 16), (200, 72), (150, 128)])
def test_infinities_in_b(dg, tokens, rank, xk, ok):
    """An infinite or NaN element of B_l makes of its output what the formula does; other outputs keep their bits."""
    N, K = 203, 256
    gen = torch.Generator().manual_seed(rank)
    x, a = torch.zeros(tokens, K, dtype=xk), torch.zeros(1, rank, K, dtype=xk)
    whole = torch.randint(1, 200, (tokens, rank), generator=gen).double() * (1 - 2 * torch.randint(0, 2, (tokens, rank), generator=gen))
    x[:, :rank] = whole.to(xk)
    x[:, rank : 2 * rank] = (whole / 512).to(xk)
    x[3, :rank] = 0
    x[3, rank : 2 * rank] = 0  # no product but zero: an infinity times it is NaN
    x[2, 1] = x[2, rank + 1] = 0
    for r in range(rank):
        a[0, r, r] = a[0, r, rank + r] = 1.0  # 8 and more bits: the second numbers are zero for some, of either sign for others
    b = torch.randn(1, N, rank, generator=gen).to(xk)
    bad = b.clone()
    inf = float("inf")
    bad[0, 7, 0], bad[0, 64, rank - 1], bad[0, 65, 2], bad[0, 130, 1], bad[0, 202, 3] = inf, -inf, float("nan"), inf, -inf
    bad[0, 131, 4], bad[0, 131, 5] = inf, inf  # two of them: NaN where their products' signs differ
    base = torch.randn(tokens, N, generator=gen).to(ok)
    off, pos, slot = dg.dg_route_sort(torch.zeros(tokens, 1, dtype=torch.int32, device=DEV), 1)
    say("infinities in B, %d rows of rank %d %s %s" % (tokens, rank, xk, ok))
    clean, out = (dg.dg_lora(x.to(DEV), a.to(DEV), t.to(DEV), off, pos, slot, None, base.to(DEV)).cpu() for t in (b, bad))
    v = x.double() @ a[0].double().t()
    want = base.double() + (v[:, None] * bad[0].double()[None]).sum(2)
    finite = torch.isfinite(want)
    assert torch.isfinite(out[finite]).all() and torch.equal(out[finite], clean[finite])
    assert torch.equal(torch.isnan(out), torch.isnan(want))
    assert torch.equal(out.double()[torch.isinf(want)], want[torch.isinf(want)])
    over = base.to(DEV)
    dg.dg_lora(x.to(DEV), a.to(DEV), bad.to(DEV), off, pos, slot, None, over, over)  # in place
    bits = {F32: torch.int32, BF16: torch.int16}[ok]
    assert torch.equal(over.cpu().view(bits), out.view(bits))
    assert int(torch.isinf(want).sum()) > 2 * tokens and torch.isnan(want[3, 7])

"""Plain 64-bit forms of the operators around the product (norm, epilogue and
their gradients), on the CPU with torch, from their definitions; and the
bounds the tests hold the kernels to."""

from __future__ import annotations

import math

import torch

U32 = 2.0 ** -24  # half a step of FP32, relative
FMAX = {0: 448.0, 1: 57344.0}
F8 = {0: torch.float8_e4m3fn, 1: torch.float8_e5m2}
# half a step of the codes: relative for normal values, absolute (in units of the factor) for subnormal ones
CODE_REL = {0: 2.0 ** -4, 1: 2.0 ** -3}
CODE_ABS = {0: 2.0 ** -10, 1: 2.0 ** -17}


def half_step(dtype) -> float:
    return torch.finfo(dtype).eps / 2


def act(z, code):
    if code == 1:
        return torch.where(z > 0, z, torch.zeros_like(z))
    if code == 2:
        return 0.5 * z * torch.special.erfc(-z / math.sqrt(2))
    if code == 3:
        return z * torch.sigmoid(z)
    if code == 4:
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    return z


def act_grad(z, code):
    if code == 1:
        return (z > 0).to(z.dtype)
    if code == 2:
        return 0.5 * torch.special.erfc(-z / math.sqrt(2)) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if code == 3:
        p = torch.sigmoid(z)
        return p * (1 + z * (1 - p))
    if code == 4:
        z = z.clamp(-1e4, 1e4)  # both tails are constant far inside; keeps the cube finite
        k = math.sqrt(2 / math.pi)
        t = torch.tanh(k * (z + 0.044715 * z ** 3))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * k * (1 + 3 * 0.044715 * z * z)
    return torch.ones_like(z)


def norm(x, res, w, eps):
    """(h in its stored type, rstd, y) from CPU tensors; rstd and y in 64 bits."""
    h = x if res is None else (x.float() + res.float()).to(res.dtype)
    hd = h.double()
    rstd = 1.0 / torch.sqrt((hd * hd).mean(1) + eps)
    return h, rstd, hd * rstd[:, None] * w.double()


def norm_bwd(dy, h, rstd, w, dh):
    """(dx, dw, bound of dx, bound of dw but for the outputs' own rounding)."""
    n = h.double() * rstd.double()[:, None]
    g = dy.double()
    u = g * w.double()
    m = (u * n).mean(1, keepdim=True)
    k = rstd.double()[:, None]
    dx = k * (u - n * m)
    # FP32: a few roundings of each term, and a sum over the row of depth below
    # 96 (sequential inside a thread, then a tree) that errs by 96 U32 mean|u n|
    bx = 112 * U32 * k * (u.abs() + n.abs() * (u * n).abs().mean(1, keepdim=True))
    if dh is not None:
        dx = dx + dh.double()
        bx = bx + 2 * U32 * dh.double().abs()
    rows = dy.shape[0]
    return dx, (g * n).sum(0), bx, (rows + 8) * U32 * (g * n).abs().sum(0)


def factors(y, block_rows, g, fmt):
    """The factors of y's blocks in 64 bits (1.0 for blocks of zeros)."""
    rows, cols = y.shape
    n = -(-rows // block_rows)
    wide = torch.zeros(n * block_rows, cols, dtype=torch.float64)
    wide[:rows] = y
    s = wide.abs().reshape(n, block_rows, cols // g, g).amax((1, 3)) / FMAX[fmt]
    return torch.where(s > 0, s, torch.ones_like(s))


def check_codes(q, scales, y, block_rows, g, fmt, rel, absolute=0.0):
    """q, scales (CPU) against the 64-bit y, known to the kernel within rel * |y| + absolute."""
    s = factors(y, block_rows, g, fmt)
    got = scales.double()
    off = (rel + 2 * U32) * s + absolute / FMAX[fmt]
    assert got.shape == s.shape
    assert ((got - s).abs() <= off).all(), "factors off by up to %g" % ((got - s).abs() / s).max()
    by = got.repeat_interleave(block_rows, 0)[: y.shape[0]].repeat_interleave(g, 1)
    value = q.view(F8[fmt]).double() * by
    room = torch.maximum(CODE_REL[fmt] * y.abs(), CODE_ABS[fmt] * by) * (1 + 4 * rel + 8 * U32)
    bad = (value - y).abs() > room + (rel + 4 * U32) * y.abs() + absolute
    assert not bad.any(), "%d of %d codes off by more than half a step" % (int(bad.sum()), bad.numel())


def stream(seed, rows, cols, dtype, zero_rows=()):
    """Hidden states: rows of different size, a few large channels, some rows of zeros."""
    gen = torch.Generator().manual_seed(seed)
    v = torch.randn(rows, cols, generator=gen) * torch.exp(torch.rand(rows, 1, generator=gen) * 2 - 1)
    v = v * torch.where(torch.rand(1, cols, generator=gen) < 0.01, 20.0, 1.0)
    for r in zero_rows:
        if r < rows:
            v[r] = 0.0
    return v.to(dtype)


def padded(t, pad):
    """t on the GPU with `pad` further elements (of 7.0) between its rows."""
    if not pad:
        return t.to("cuda:0")
    wide = torch.full((t.shape[0], t.shape[1] + pad), 7.0, dtype=t.dtype, device="cuda:0")
    wide[:, : t.shape[1]] = t.to("cuda:0")
    return wide[:, : t.shape[1]]

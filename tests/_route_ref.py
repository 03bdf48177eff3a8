"""Plain forms of the calls of experts and adapters, on the CPU: the sort by
counting, the rest in 64 bits from the definitions; and routings for the tests."""

from __future__ import annotations

import numpy as np
import torch

from tests import _layer_ref as ref

U32 = ref.U32


def routing(seed, tokens, k, groups, idle=0.0, skew=1.0, dtype=torch.int32):
    """[tokens, k] groups, some liked more than others; a share of the slots -1. The same group may stand twice in a token."""
    rng = np.random.default_rng(seed)
    p = np.exp(skew * rng.standard_normal(groups))
    ids = rng.choice(groups, size=(tokens, k), p=p / p.sum())
    ids[rng.random((tokens, k)) < idle] = -1
    return torch.from_numpy(ids).to(dtype)


def rows_of(tokens, k, groups, align):
    n = tokens * k
    return (n + min(groups, n) * (align - 1)) // align * align


def sort(ids, groups, align, rows):
    """(offsets, position, slot) as int32 tensors, by numpy."""
    flat = ids.reshape(-1).numpy().astype(np.int64)
    ok = (flat >= 0) & (flat < groups)
    count = np.bincount(flat[ok], minlength=groups)
    start = np.concatenate([[0], np.cumsum(-(-count // align) * align)])
    slots = np.flatnonzero(ok)
    order = slots[np.argsort(flat[slots], kind="stable")]
    key = flat[order]
    at = start[key] + np.arange(order.size) - np.concatenate([[0], np.cumsum(count)])[key]
    position = np.full(flat.size, -1, np.int64)
    position[order] = at
    slot = np.full(rows, -2, np.int64)
    slot[: start[-1]] = -1
    slot[at] = order
    t = lambda v: torch.from_numpy(v.astype(np.int32))  # noqa: E731
    return t(start), t(position).reshape(ids.shape), t(slot)


def gathered(x, slot, k, weights):
    """The FP32 rows that are quantised: weights times x in sorted order, zeros in rows without a slot."""
    at = slot.long().clamp(min=0)
    v = x[at // k].float()
    if weights is not None:
        v = v * weights.reshape(-1)[at][:, None]
    v[slot < 0] = 0.0
    return v


def combine(y, position, weights, res):
    """(out, bound of the FP32 sum) in 64 bits; rows of y that no slot names are not touched."""
    tokens, k = position.shape
    out = torch.zeros(tokens, y.shape[1], dtype=torch.float64)
    size = torch.zeros_like(out)
    for j in range(k):
        t = torch.nonzero(position[:, j] >= 0)[:, 0]
        v = y[position[t, j].long()].double()
        if weights is not None:
            v = v * weights[t, j].double()[:, None]
        out[t] += v
        size[t] += v.abs()
    if res is not None:
        out, size = out + res.double(), size + res.double().abs()
    return out, (k + 1) * U32 * size  # k fused steps and the residual's addition


def weight_grad(x, y, position):
    """(dw, bound): chains of at most cols / 256 + 8 terms per thread, then trees of depth below 12."""
    tokens, k = position.shape
    dw = torch.zeros(tokens, k, dtype=torch.float64)
    size = torch.zeros_like(dw)
    for j in range(k):
        t = torch.nonzero(position[:, j] >= 0)[:, 0]
        p = x[t].double() * y[position[t, j].long()].double()
        dw[t, j], size[t, j] = p.sum(1), p.abs().sum(1)
    return dw, (x.shape[1] / 256 + 24) * U32 * size


def spread(s, rows, g, n):
    """Factors per block -> one per element, n rows, in 64 bits."""
    return s.double().repeat_interleave(rows, 0)[:n].repeat_interleave(g, 1)


def lora(x, a, b, ids, scale, base):
    """(out, the sizes of its terms) in 64 bits."""
    out = torch.zeros(x.shape[0], b.shape[1], dtype=torch.float64)
    size, vsize = torch.zeros_like(out), torch.zeros_like(out)
    for e in range(a.shape[0]):
        t = torch.nonzero(ids == e)[:, 0]
        if t.numel():
            s = 1.0 if scale is None else float(scale[e])
            ad, bd = a[e].double(), b[e].double()
            v = x[t].double() @ ad.t()
            out[t] = s * (v @ bd.t())
            size[t] = abs(s) * ((x[t].double().abs() @ ad.abs().t()) @ bd.abs().t())
            vsize[t] = abs(s) * (v.abs().amax(1, keepdim=True) * bd.abs().sum(1)[None])
    return (out if base is None else out + base.double()), size, vsize

"""The training step of examples/mlp_step.py, each result held to what its own products leave open: the shares that the
residual carries past them (h in out, dout in dx) are exact and taken off first.

Bounds, relative in the 2-norm, from the formats alone. An element's rounding error is spread evenly over a step, so an
operand's is at most its half step over sqrt(3) of it (E4M3 2^-4, E5M2 2^-3), and independent errors add in squares. The
activation: z is off by F of its size (about 1); GELU's slope is below 1.13 and its curvature below 0.8, GELU(z) has the
2-norm 0.65 and GELU'(z) 0.68 of a standard normal z. BF16 results add half a step over sqrt(3) of the stored value.

The gradient through an RMS norm has no part along the normed row: that holds whatever the products' errors are, and
shows the mean term that the other bounds would let pass."""

import math
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

E4, E5, B16 = (2.0 ** -n / math.sqrt(3) for n in (4, 3, 9))
F = math.hypot(E4, E4)  # pre: y and W1
A = math.hypot(1.13 / 0.65 * F, E4)  # the second product's quantised operand
DZ = math.sqrt(E5 ** 2 + E4 ** 2 + (0.8 / 0.68 * F) ** 2 + E5 ** 2)  # dout, W2, the derivative, the codes of dz
BOUNDS = dict(out=math.hypot(A, E4), dx=math.hypot(DZ, E4), dnorm=math.hypot(DZ, E4), dw1=math.hypot(DZ, E4), db1=DZ, dw2=math.hypot(E5, A))

NAMES = ("out", "dx", "dnorm", "dw1", "db1", "dw2", "db2")


def failures(got, want, x, residual, dout):
    """The names of what is outside its bound. got, want: out and the six gradients."""
    h = (x.float() + residual.float()).to(residual.dtype)
    bad = []
    for name, g, w in zip(NAMES, got, want):
        g, w = g.double(), w.double()
        past = h.double() if name == "out" else dout.double() if name == "dx" else 0.0
        # stored in BF16: out, and dx; every product's output too, in the chain (two more). db2 has FP32 sums alone
        stored = 0.0 if name == "db2" else 3 * B16
        room = BOUNDS.get(name, 0.0) * (w - past).norm() + (stored + 2.0 ** -20) * w.norm()
        if not (g - w).norm() <= room:
            bad.append(name)
        print("%s: off by %.4f of its bound" % (name, float((g - w).norm() / room)))
    # dx - dout is orthogonal to its row of h; dx's BF16 rounding leaves at most half a step of each term, each term's
    # error independent of the others', and FP32 sums a little
    d, hd = got[1].double() - dout.double(), h.double()
    along = (d * hd).sum(1)
    room = (2.0 ** -8 * got[1].double().abs() * hd.abs()).norm(dim=1) + 2.0 ** -18 * (d.abs() * hd.abs()).sum(1)
    if not along.norm() <= room.norm():
        bad.append("dx along h")
    print("dx along h: %.4f of its bound" % float(along.norm() / room.norm()))
    return bad


def _quantised(t, by_rows, fmax, dtype, g=128):
    """t as its FP8 codes and factors hold it."""
    rows, cols = t.shape
    b = t.double().reshape(rows, 1, cols // g, g) if by_rows else t.double().reshape(rows // g, g, cols // g, g)
    s = (b.abs().amax((1, 3), keepdim=True) / fmax).float().double().clamp(min=1e-30)
    return ((b / s).float().to(dtype).double() * s).reshape(rows, cols)


def step(weights, x, residual, dout, drop=None):
    """The step as its calls are defined, in 64 bits with their roundings, on the CPU. drop: a mistake planted here."""
    w1, b1, w2, b2, nw = (w.double() for w in weights)
    e4 = lambda t, rows=False: _quantised(t, rows, 448.0, torch.float8_e4m3fn)  # noqa: E731
    e5 = lambda t: _quantised(t, False, 57344.0, torch.float8_e5m2)  # noqa: E731
    h = (x.float() + residual.float()).to(residual.dtype).double()
    rstd = 1 / torch.sqrt(h.square().mean(1, keepdim=True) + 1e-6)
    y = h * rstd * nw
    pre = (e4(y, True) @ e4(w1).t() + b1).bfloat16().double()
    a = torch.nn.functional.gelu(pre).bfloat16().double()
    out = (e4(a, True) @ e4(w2).t() + b2 + h).bfloat16()
    d = dout.double()
    da = (e5(d) @ e4(w2)).bfloat16().double()
    slope = 0.5 * (1 + torch.erf(pre / math.sqrt(2))) + pre * torch.exp(-pre * pre / 2) / math.sqrt(2 * math.pi)
    dz = da * (1.0 if drop == "activation" else slope)
    dy = (e5(dz) @ e4(w1)).bfloat16().double()
    n, u = h * rstd, dy * nw
    mean = 0.0 if drop == "mean" else (u * n).mean(1, keepdim=True)
    dx = d + (0.0 if drop == "norm" else rstd * (u - n * mean))
    if drop == "residual":
        dx = dx - d
    if drop == "rstd":
        dx = d + (dx - d) / rstd
    return (out, dx.bfloat16(), (dy * n).sum(0), e5(dz).t() @ e4(y), dz.sum(0), e5(d).t() @ e4(a), d.sum(0))


@pytest.mark.parametrize("tokens,hidden,ffn", [(128, 256, 512), (384, 1024, 640)])
def test_bounds_find_planted_mistakes(tokens, hidden, ffn):
    import mlp_step

    weights, x, residual, dout = mlp_step.inputs(tokens, hidden, ffn, seed=tokens, device="cpu")
    ref, grads = mlp_step.reference(*weights, x, residual, dout)
    want = (ref,) + grads
    assert failures(step(weights, x, residual, dout), want, x, residual, dout) == []
    for drop, found in [("norm", "dx"), ("mean", "dx along h"), ("residual", "dx"), ("rstd", "dx"), ("activation", "db1")]:
        assert found in failures(step(weights, x, residual, dout, drop), want, x, residual, dout), drop
    for i, name in enumerate(NAMES[:-1]):  # a gradient of zeros, and one a quarter too large
        past = dout.double() if name == "dx" else 0.0
        for factor in (0.0, 1.25):
            if name != "out":
                got = list(want)
                got[i] = (past + factor * (want[i].double() - past)).to(want[i].dtype)
                assert name in failures(got, want, x, residual, dout), (name, factor)
    got = (x.float() + residual.float(),) + want[1:]
    assert "out" in failures(got, want, x, residual, dout)


def test_reference_leaves_its_arguments_alone():
    import mlp_step

    weights, x, residual, dout = mlp_step.inputs(8, 16, 24, device="cpu")
    mlp_step.reference(*weights, x, residual, dout)
    assert not any(t.requires_grad for t in weights + (x, residual, dout))


@pytest.mark.gpu
@pytest.mark.parametrize("tokens,hidden,ffn", [(128, 256, 512), (384, 1024, 640), (1024, 512, 2048), (2176, 768, 1920)])
def test_step(tokens, hidden, ffn):
    import mlp_step
    from tests._gpu import say

    say("mlp step, its own shares %d %d %d" % (tokens, hidden, ffn))
    weights, x, residual, dout = mlp_step.inputs(tokens, hidden, ffn, seed=tokens)
    mlp = mlp_step.MLP(*weights)
    out, kept = mlp.forward(x, residual)
    got = (out,) + mlp.backward(dout, kept)
    want, grads = mlp_step.reference(*weights, x, residual, dout)
    torch.cuda.synchronize()
    assert failures(got, (want,) + grads, x, residual, dout) == []

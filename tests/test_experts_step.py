"""The step of a layer of experts (examples/experts_step.py): each result against FP32 autograd on unquantised weights, the
shares that the residual carries past the experts (x in out, dout in dx) taken off first.

Bounds, relative in the 2-norm, from the formats alone, as for the dense step in test_mlp_step_gradients.py: an operand is
off by at most its half step over sqrt(3) of it, independent errors add in squares, and the activation passes an error F of
a standard normal z on as at most 1.13 F of 0.65, its derivative one of 0.8 F of 0.68. The choices' weights are exact. dw is
a row of dout (exact) times a row of y: y's error, as a share of y, along a direction that has nothing to do with it."""

import math
import os
import sys

import pytest
import torch

from tests.test_mlp_step_gradients import A, B16, DZ, E4, E5, _quantised

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

NAMES = ("out", "dx", "dw", "dw1", "dw2")
BOUNDS = dict(out=math.hypot(A, E4), dx=math.hypot(DZ, E4), dw=math.hypot(A, E4), dw1=math.hypot(DZ, E4), dw2=math.hypot(E5, A))


def failures(got, want, x, dout, names=NAMES):
    bad = []
    for name, g, w in zip(names, got, want):
        g, w = g.double(), w.double()
        past = x.double() if name == "out" else dout.double() if name == "dx" else 0.0
        # up to three BF16 tensors on the way, the last of the size of the whole result
        room = BOUNDS[name] * (w - past).norm() + (3 * B16 + 2.0 ** -20) * w.norm()
        if not (g - w).norm() <= room:
            bad.append(name)
        print("%s: off by %.4f of its bound" % (name, float((g - w).norm() / room)))
    return bad


def step(weights, x, ids, w, dout, drop=None):
    """The step as its calls are defined, in 64 bits with their roundings, expert by expert. drop: a mistake planted here."""
    e4 = lambda t: _quantised(t, False, 448.0, torch.float8_e4m3fn)  # noqa: E731
    e5 = lambda t: _quantised(t, False, 57344.0, torch.float8_e5m2)  # noqa: E731
    w1, w2 = weights
    out, dx, dw = x.double().clone(), dout.double().clone(), torch.zeros(w.shape, dtype=torch.float64)
    dw1, dw2 = torch.zeros(w1.shape, dtype=torch.float64), torch.zeros(w2.shape, dtype=torch.float64)
    for e in range(w1.shape[0]):
        token, choice = torch.nonzero(ids == (e + 1 if drop == "expert" else e), as_tuple=True)
        n = token.numel()
        if not n:
            continue

        def rows(t):  # padded with zeros to whole blocks, as the sort leaves them
            return torch.cat([t.double(), torch.zeros(-n % 128, t.shape[1], dtype=torch.float64)])

        u1, u2, weight = e4(w1[e]), e4(w2[e]), w[token, choice].double()[:, None]
        q = e4(rows(x[token]))
        pre = (q @ u1.t()).bfloat16().double()
        a = e4(torch.nn.functional.gelu(pre).bfloat16())
        y = (a @ u2.t()).bfloat16().double()[:n]
        out.index_add_(0, token, y * (1.0 if drop == "weights" else weight))
        d = e5(rows(dout[token].double() * (1.0 if drop == "gradient's weights" else weight)))
        dw[token, choice] = (dout[token].double() * y).sum(1)
        dw2[e] = (d.t() @ a).bfloat16()
        slope = 0.5 * (1 + torch.erf(pre / math.sqrt(2))) + pre * torch.exp(-pre * pre / 2) / math.sqrt(2 * math.pi)
        z = e5((d @ u2).bfloat16().double() * (1.0 if drop == "activation" else slope))
        dw1[e] = (z.t() @ q).bfloat16()
        back = (z @ u1).bfloat16().double()[:n]
        dx.index_add_(0, token, back.roll(1, 0) if drop == "order" else back)
    if drop == "residual":
        dx -= dout.double()
    return out.bfloat16(), dx.bfloat16(), dw, dw1, dw2


SIZES = [(300, 256, 384, 4, 2), (130, 512, 256, 5, 3)]


@pytest.mark.parametrize("tokens,hidden,ffn,experts,choices", SIZES)
def test_bounds_find_planted_mistakes(tokens, hidden, ffn, experts, choices):
    import experts_step

    weights, x, ids, w, dout = experts_step.inputs(tokens, hidden, ffn, experts, choices, seed=tokens, device="cpu")
    ref, grads = experts_step.reference(*weights, x, ids, w, dout)
    want = (ref,) + grads
    assert failures(step(weights, x, ids, w, dout), want, x, dout) == []
    for drop, found in [("expert", "out"), ("weights", "out"), ("gradient's weights", "dw2"), ("activation", "dw1"), ("order", "dx"),
                        ("residual", "dx")]:
        assert found in failures(step(weights, x, ids, w, dout, drop), want, x, dout), drop
    for i, name in list(enumerate(NAMES))[1:]:  # a gradient of zeros, and one half as large again
        past = dout.double() if name == "dx" else 0.0
        for factor in (0.0, 1.5):
            got = list(want)
            got[i] = (past + factor * (want[i].double() - past)).to(want[i].dtype)
            assert name in failures(got, want, x, dout), (name, factor)


@pytest.mark.gpu
@pytest.mark.parametrize("tokens,hidden,ffn,experts,choices", SIZES + [(1, 256, 256, 8, 8), (1000, 512, 1024, 64, 4), (2000, 768, 1920, 7, 2)])
def test_step(tokens, hidden, ffn, experts, choices):
    import experts_step
    from tests._gpu import say

    say("experts' step %d %d %d, %d of %d" % (tokens, hidden, ffn, choices, experts))
    weights, x, ids, w, dout = experts_step.inputs(tokens, hidden, ffn, experts, choices, seed=tokens)
    layer = experts_step.Experts(*weights)
    out, kept = layer.forward(x, ids, w)
    got = (out,) + layer.backward(dout, kept)
    one = layer.serve(x, ids, w)
    want, grads = experts_step.reference(*weights, x, ids, w, dout)
    torch.cuda.synchronize()
    many = tokens > 1  # of one token the sums have too few terms for errors to be independent
    assert failures(got if many else got[:1], ((want,) + grads) if many else (want,), x, dout) == []
    assert failures((one,), (want,), x, dout, ("out",)) == []


@pytest.mark.gpu
def test_step_in_a_graph():
    """Forward and backward captured once, replayed on other tokens, choices and gradients, with eager work and
    synchronisations between; every replay against the eager step to the bit."""
    import experts_step

    weights, x, ids, w, dout = experts_step.inputs(700, 512, 384, 12, 3)
    layer = experts_step.Experts(*weights)

    def both():
        out, kept = layer.forward(x, ids, w)
        return (out, layer.serve(x, ids, w)) + layer.backward(dout, kept)

    eager = both()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        both()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = both()
    for i in range(5):
        if i:
            _, x2, ids2, w2, d2 = experts_step.inputs(700, 512, 384, 12, 3, seed=i)
            x.copy_(x2), w.copy_(w2), dout.copy_(d2)
            ids.copy_(torch.zeros_like(ids2) + i if i == 2 else torch.where(ids2 < 3, -1, ids2) if i == 3 else ids2)
            eager = both()
            torch.cuda.synchronize()
        for t in held:
            t.fill_(float("nan"))
        graph.replay()
        if i % 2:
            both()
        torch.cuda.synchronize()
        for a, b in zip(held, eager):
            assert torch.equal(a, b)


@pytest.mark.gpu
def test_example_runs(capsys):
    import experts_step

    experts_step.main(256, 256, 256, 4, 2)
    assert "us a step" in capsys.readouterr().out

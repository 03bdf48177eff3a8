"""The training step of examples/mlp_step.py: its output and gradients against FP32 autograd on unquantised
weights. Every element of an operand is off by at most half a step of its format (2^-4 relative in E4M3, 2^-3 in
E5M2), so by at most 2^-4 and 2^-3 of it in the 2-norm; a product adds its operands' errors, and a chain of
products each one's. Then the biases, whose gradients pass through no quantised operand but those before them."""

import os
import sys

import pytest

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu

E4, E5 = 2.0 ** -4, 2.0 ** -3


@pytest.mark.parametrize("tokens,hidden,ffn", [(128, 256, 512), (384, 1024, 640), (1024, 512, 2048)])
def test_mlp_step(tokens, hidden, ffn):
    import torch

    import mlp_step
    from tests._gpu import say

    say("mlp step %d %d %d" % (tokens, hidden, ffn))
    weights, x, residual, dout = mlp_step.inputs(tokens, hidden, ffn, seed=tokens)
    mlp = mlp_step.MLP(*weights)
    out, kept = mlp.forward(x, residual)
    got = (out,) + mlp.backward(dout, kept)
    want, grads = mlp_step.reference(*weights, x, residual, dout)
    torch.cuda.synchronize()
    first = 2 * E4 * 1.13  # a: y and W1, through an activation of slope at most 1.13
    # the sums of independent errors stay below the sum of their bounds; the residual's share of out and dx has none
    bounds = dict(out=first + 2 * E4, dx=2 * (E5 + E4) + first, dnorm=2 * (E5 + E4) + first, dw1=2 * (E5 + E4) + first,
                  db1=E5 + E4 + first, dw2=E5 + E4 + first, db2=2.0 ** -20)
    for (name, bound), g, w in zip(bounds.items(), got, (want,) + grads):
        error = float((g.float() - w).norm() / w.norm())
        print("%s %.4f of %.4f" % (name, error, bound))
        assert error <= bound, name


def test_serving_forward_is_the_training_forward():
    import torch

    import mlp_step

    weights, x, residual, _ = mlp_step.inputs(77, 256, 384, seed=5)
    mlp = mlp_step.MLP(*weights)
    out, _ = mlp.forward(x, residual)
    one, _ = mlp.forward(x, residual, keep=False)
    torch.cuda.synchronize()
    assert torch.equal(out, one)

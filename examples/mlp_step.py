"""One training step of a pre-norm MLP block on the library's calls.

    h   = x + residual;  y = rmsnorm(h) * w
    out = gelu(y W1^T + b1) W2^T + b2 + h

Forward: the norm quantises its own output, the first product keeps its
pre-activation, the second adds the residual stream in its epilogue. Backward:
each epilogue's gradient is quantised once, in blocks that serve the gradient of
the activations and, read transposed, that of the weights; the norm's backward
pass adds the gradient that went past it. Serving runs the same forward calls
without y, rstd and pre.

Run on a GPU:  python examples/mlp_step.py [tokens hidden ffn]
prints the gradients' errors against FP32 autograd on the same weights, and the
time of a step.
"""

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import fp8_block_scaled_scales_amd as dg  # noqa: E402

G = 128  # block granularity of every quantised tensor
EPS = 1e-6


class MLP:
    """Weights [ffn, hidden] and [hidden, ffn], quantised once in G x G blocks, with their factors for both directions."""

    def __init__(self, w1, b1, w2, b2, norm_weight):
        self.b1, self.b2, self.norm_weight = b1, b2, norm_weight
        self.w1, self.s1 = dg.dg_quantize_fp8_blocks_typed(w1, gran=G)
        self.w2, self.s2 = dg.dg_quantize_fp8_blocks_typed(w2, gran=G)
        # the backward products read the same codes as [K, N]: only the factors are transposed
        self.s1t, self.s2t = self.s1.t().contiguous(), self.s2.t().contiguous()

    def forward(self, x, residual, keep=True):
        """(out, what backward needs): out is the new residual stream, of the type bfloat16."""
        rows, cols = x.shape
        y = torch.empty_like(x) if keep else None
        rstd = torch.empty(rows, dtype=torch.float32, device=x.device) if keep else None
        pre = torch.empty(rows, self.w1.shape[0], dtype=torch.bfloat16, device=x.device) if keep else None
        q, s, h = dg.dg_rmsnorm_quantize_fp8(x, residual, self.norm_weight, EPS, gran=G, y=y, rstd=rstd)
        a = dg.dg_gemm_fp8_residual(q, self.w1, s, self.s1, gran=G, sa_rows=1, bias=self.b1, act=dg.DG_ACT_GELU, pre=pre)
        aq, sa = dg.dg_quantize_fp8_rows_typed(a, gran=G)
        out = dg.dg_gemm_fp8_residual(aq, self.w2, sa, self.s2, res=h, gran=G, sa_rows=1, bias=self.b2)
        return out, (h, y, rstd, pre, a)

    def backward(self, dout, kept):
        """Gradients of (x and residual alike, norm weight, w1, b1, w2, b2) from that of out. Tokens in a multiple of G."""
        h, y, rstd, pre, a = kept
        e5 = dict(gran=G, fmt_a=dg.DG_FMT_E5M2)
        db1, db2 = torch.empty_like(self.b1), torch.empty_like(self.b2)
        # through "+ b2 + h": the codes of dout, and its column sums
        d, sd = dg.dg_epilogue_backward_fp8(dout, None, dg.DG_ACT_NONE, gran=G, dbias=db2)
        da = dg.dg_gemm_fp8_layout(d, self.w2, sd, self.s2t, layout=dg.DG_LAYOUT_NN, **e5)
        aq, sa = dg.dg_quantize_fp8_blocks_typed(a, gran=G)
        dw2 = dg.dg_gemm_fp8_layout(d, aq, sd.t().contiguous(), sa.t().contiguous(), layout=dg.DG_LAYOUT_TN, **e5)
        # through the activation
        z, sz = dg.dg_epilogue_backward_fp8(da, pre, dg.DG_ACT_GELU, gran=G, dbias=db1)
        dy = dg.dg_gemm_fp8_layout(z, self.w1, sz, self.s1t, layout=dg.DG_LAYOUT_NN, **e5)
        yq, sy = dg.dg_quantize_fp8_blocks_typed(y, gran=G)
        dw1 = dg.dg_gemm_fp8_layout(z, yq, sz.t().contiguous(), sy.t().contiguous(), layout=dg.DG_LAYOUT_TN, **e5)
        # through the norm, with the gradient that the residual carried past both products
        dx, dnorm = dg.dg_rmsnorm_backward(dy, h, rstd, self.norm_weight, dh=dout)
        return dx, dnorm, dw1, db1, dw2, db2


def reference(w1, b1, w2, b2, norm_weight, x, residual, dout):
    """The same step in FP32 on unquantised weights: out and the six gradients."""
    leaves = [t.detach().float().clone().requires_grad_() for t in (x, norm_weight, w1, b1, w2, b2)]
    xf, nw, w1f, b1f, w2f, b2f = leaves
    h = xf + residual.float()
    y = h * torch.rsqrt(h.square().mean(1, keepdim=True) + EPS) * nw
    out = torch.nn.functional.gelu(y @ w1f.t() + b1f) @ w2f.t() + b2f + h
    return out.detach(), torch.autograd.grad(out, leaves, dout.float())


def inputs(tokens, hidden, ffn, seed=0, device="cuda:0"):
    gen = torch.Generator(device=device).manual_seed(seed)
    r = lambda *shape: torch.randn(*shape, generator=gen, device=device)  # noqa: E731
    w1, w2 = (r(ffn, hidden) / hidden ** 0.5).bfloat16(), (r(hidden, ffn) / ffn ** 0.5).bfloat16()
    weights = (w1, 0.1 * r(ffn), w2, 0.1 * r(hidden), 1 + 0.1 * r(hidden))
    return weights, r(tokens, hidden).bfloat16(), r(tokens, hidden).bfloat16(), (r(tokens, hidden) * 1e-2).bfloat16()


def main(tokens=4096, hidden=2048, ffn=8192):
    weights, x, residual, dout = inputs(tokens, hidden, ffn)
    mlp = MLP(*weights)
    out, kept = mlp.forward(x, residual)
    grads = mlp.backward(dout, kept)
    want, want_grads = reference(*weights, x, residual, dout)
    for name, got, ref in zip(("out", "dx", "dnorm", "dw1", "db1", "dw2", "db2"), (out,) + grads, (want,) + want_grads):
        print("%-6s relative error %.4f" % (name, float((got.float() - ref).norm() / ref.norm())))
    start, stop = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    for _ in range(10):
        out, kept = mlp.forward(x, residual)
        mlp.backward(dout, kept)
    stop.record()
    torch.cuda.synchronize()
    us = start.elapsed_time(stop) * 100
    print("%d tokens, hidden %d, ffn %d: %.0f us a step, %.0f TFLOP/s in the six products" % (
        tokens, hidden, ffn, us, 12.0 * tokens * hidden * ffn / us * 1e-6))


if __name__ == "__main__":
    main(*map(int, sys.argv[1:4]))

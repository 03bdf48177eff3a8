"""One training step, and the serving forward pass, of a layer of experts on the library's calls.

    out = x + sum over j of w[t, j] * gelu(x W1_e^T) W2_e^T,  e = ids[t, j]

Forward: the choices are sorted by expert once; the tokens become FP8 rows in that
order, in blocks that the weights' gradient reads again; two products with each
expert's own weights, the first keeping its pre-activation; the outputs come back
weighted, with the residual stream. Backward: the gradient goes out to the experts as
weighted FP8 rows, once for the rows' and the weights' gradients. No number of rows
comes to the host. Serving sorts without padding and takes a factor per row.

Run on a GPU:  python examples/experts_step.py [tokens hidden ffn experts choices]
prints the gradients' errors against FP32 autograd on the same weights, and the
time of a step.
"""

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import fp8_block_scaled_scales_amd as dg  # noqa: E402

G = 128  # block granularity of every quantised tensor


def _weights(w):
    """[experts, N, K] as codes, factors, and the factors of the product that reads the same codes as [K, N]."""
    experts, n, k = w.shape
    q, s = dg.dg_quantize_fp8_blocks_typed(w.reshape(experts * n, k), gran=G)  # N in a multiple of G: no block has two experts
    s = s.reshape(experts, n // G, k // G)
    return q.reshape(w.shape), s, s.transpose(1, 2).contiguous()


class Experts:
    """Weights [experts, ffn, hidden] and [experts, hidden, ffn], quantised once in G x G blocks."""

    def __init__(self, w1, w2):
        self.experts = w1.shape[0]
        self.w1, self.s1, self.s1t = _weights(w1)
        self.w2, self.s2, self.s2t = _weights(w2)

    def forward(self, x, ids, w):
        """(out, what backward needs) for the tokens x, their choices ids [tokens, k] and those weights w (FP32)."""
        offsets, position, slot = dg.dg_route_sort(ids, self.experts, align=G)
        q, s = dg.dg_route_quantize_fp8(x, position, slot, gran=G, block_rows=G)
        pre = torch.empty(q.shape[0], self.w1.shape[1], dtype=torch.bfloat16, device=x.device)
        a = dg.dg_gemm_fp8_grouped(q, self.w1, s, self.s1, offsets, gran=G, act=dg.DG_ACT_GELU, pre=pre)
        # rows behind the last expert's hold anything, in blocks of their own, here and below: no later call uses them
        aq, sa = dg.dg_quantize_fp8_blocks_typed(a, gran=G)
        y = dg.dg_gemm_fp8_grouped(aq, self.w2, sa, self.s2, offsets, gran=G)
        out = dg.dg_route_combine(y, position, w, res=x)
        return out, (offsets, position, slot, w, q, s, pre, aq, sa, y)

    def serve(self, x, ids, w):
        """out alone: no padding, a factor per row."""
        offsets, position, slot = dg.dg_route_sort(ids, self.experts)
        q, s = dg.dg_route_quantize_fp8(x, position, slot, gran=G)
        a = dg.dg_gemm_fp8_grouped(q, self.w1, s, self.s1, offsets, gran=G, sa_rows=1, act=dg.DG_ACT_GELU)
        aq, sa = dg.dg_quantize_fp8_rows_typed(a, gran=G)
        y = dg.dg_gemm_fp8_grouped(aq, self.w2, sa, self.s2, offsets, gran=G, sa_rows=1)
        return dg.dg_route_combine(y, position, w, res=x)

    def backward(self, dout, kept):
        """Gradients of (x, the choices' weights, w1, w2) from that of out."""
        offsets, position, slot, w, q, s, pre, aq, sa, y = kept
        e5 = dict(gran=G, fmt_a=dg.DG_FMT_E5M2)
        d, sd = dg.dg_route_quantize_fp8(dout, position, slot, w, gran=G, block_rows=G, fmt=dg.DG_FMT_E5M2)
        dw = dg.dg_route_weight_grad(dout, y, position)
        da = dg.dg_gemm_fp8_grouped(d, self.w2, sd, self.s2t, offsets, layout=dg.DG_LAYOUT_NN, **e5)
        dw2 = dg.dg_gemm_fp8_grouped_wgrad(d, aq, sd, sa, offsets, **e5)
        z, sz = dg.dg_epilogue_backward_fp8(da, pre, dg.DG_ACT_GELU, gran=G)
        dx = dg.dg_gemm_fp8_grouped(z, self.w1, sz, self.s1t, offsets, layout=dg.DG_LAYOUT_NN, **e5)
        dw1 = dg.dg_gemm_fp8_grouped_wgrad(z, q, sz, s, offsets, **e5)
        return dg.dg_route_combine(dx, position, res=dout), dw, dw1, dw2


def reference(w1, w2, x, ids, w, dout):
    """The same step in FP32 on unquantised weights: out and the four gradients."""
    leaves = [t.detach().float().clone().requires_grad_() for t in (x, w, w1, w2)]
    xf, wf, w1f, w2f = leaves
    out = xf
    for e in range(w1.shape[0]):
        token, choice = torch.nonzero(ids == e, as_tuple=True)
        y = torch.nn.functional.gelu(xf[token] @ w1f[e].t()) @ w2f[e].t()
        out = out.index_add(0, token, wf[token, choice, None] * y)
    return out.detach(), torch.autograd.grad(out, leaves, dout.float())


def inputs(tokens, hidden, ffn, experts, choices, seed=0, device="cuda:0"):
    gen = torch.Generator(device=device).manual_seed(seed)
    r = lambda *shape: torch.randn(*shape, generator=gen, device=device)  # noqa: E731
    w1, w2 = (r(experts, ffn, hidden) / hidden ** 0.5).bfloat16(), (r(experts, hidden, ffn) / ffn ** 0.5).bfloat16()
    w, ids = torch.softmax(r(tokens, experts), 1).topk(choices, 1)
    return (w1, w2), r(tokens, hidden).bfloat16(), ids, w, (r(tokens, hidden) * 1e-2).bfloat16()


def main(tokens=8192, hidden=2048, ffn=4096, experts=16, choices=2):
    weights, x, ids, w, dout = inputs(tokens, hidden, ffn, experts, choices)
    layer = Experts(*weights)
    out, kept = layer.forward(x, ids, w)
    grads = layer.backward(dout, kept)
    want, want_grads = reference(*weights, x, ids, w, dout)
    for name, got, ref in zip(("out", "dx", "dw", "dw1", "dw2"), (out,) + grads, (want,) + want_grads):
        print("%-4s relative error %.4f" % (name, float((got.float() - ref).norm() / ref.norm())))
    start, stop = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    for _ in range(10):
        out, kept = layer.forward(x, ids, w)
        layer.backward(dout, kept)
    stop.record()
    torch.cuda.synchronize()
    us = start.elapsed_time(stop) * 100
    print("%d tokens to %d of %d experts, hidden %d, ffn %d: %.0f us a step, %.0f TFLOP/s in the six products" % (
        tokens, choices, experts, hidden, ffn, us, 12.0 * tokens * choices * hidden * ffn / us * 1e-6))


if __name__ == "__main__":
    main(*map(int, sys.argv[1:6]))

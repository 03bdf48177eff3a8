"""Cases for timing the operators that stand around the block-scaled FP8 product in a transformer layer.

Four operators, each in its plain form (elementary torch operations in 32 bits) and as the library's call:

  norm      h = x + residual, RMS norm of h, FP8 codes with one factor per row and g-wide segment
  norm_bwd  the gradient of h (for x and the residual alike) and of the norm's weight
  gemm      act(A B^T + bias) + residual on block-scaled FP8 operands, with the pre-activation where training keeps it
  epi_bwd   the gradient through that epilogue: FP8 codes with factors for the next products, and the bias gradient
"""

import math

import torch

own = False

F8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
FMAX = {"e4m3": 448.0, "e5m2": 57344.0}
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2, "none": 0}
ACTS = ("none", "relu", "gelu", "silu", "gelu_tanh")
EPS = 1e-6


def norm(name, rows, cols, g=128, fmt="e4m3", x="bf16", res="bf16", train=False, pad=0):
    """res: the residual's type or "none"; train: also y and 1/rms, as a backward pass needs; pad: elements between x's rows."""
    return dict(name=name, op="norm", rows=rows, cols=cols, g=g, fmt=fmt, x=x, res=res, train=train, pad=pad)


def norm_bwd(name, rows, cols, x="bf16", res="bf16", dh=True):
    """x: dy's type; res: the type of h, of its incoming gradient dh and of dx."""
    return dict(name=name, op="norm_bwd", rows=rows, cols=cols, x=x, res=res, dh=dh)


def gemm(name, M, N, K, g=128, layout="nt", rowa=False, fa="e4m3", fb="e4m3", bias=False, act="none", res="bf16", pre=False, pad=0):
    """layout: first letter t: A stored [K,M], second letter n: B stored [K,N]; rowa: A's factors per row."""
    return dict(name=name, op="gemm", M=M, N=N, K=K, g=g, layout=layout, rowa=rowa, fa=fa, fb=fb, bias=bias, act=act, res=res, pre=pre, pad=pad)


def epi_bwd(name, rows, cols, g=128, act="gelu", x="bf16", rowa=False, fmt="e5m2", dz=False, dbias=True):
    return dict(name=name, op="epi_bwd", rows=rows, cols=cols, g=g, act=act, x=x, rowa=rowa, fmt=fmt, dz=dz, dbias=dbias)


def listed():
    return [
        # one token being served, before the decode product (K = 7168): latency
        norm("norm_token_1x7168", 1, 7168),
        # a ragged batch with a residual stream kept in FP32, for a g = 64 product with a long K
        norm("norm_ragged_2000x16384_g64", 2000, 16384, g=64, res="f32"),
        # a training step over 8192 tokens: y for the weight gradient and 1/rms are kept too
        norm("norm_train_8192x8192", 8192, 8192, train=True),
        # the gradient for a small micro-batch
        norm_bwd("norm_bwd_64x7168", 64, 7168),
        # the ragged batch's gradient, with the FP32 stream
        norm_bwd("norm_bwd_ragged_2000x16384", 2000, 16384, res="f32"),
        # the training step's gradient
        norm_bwd("norm_bwd_8192x8192", 8192, 8192),
        # serving 64 tokens: an output projection whose result is added to the residual stream
        gemm("gemm_decode_64x4096x7168", 64, 4096, 7168, rowa=True),
        # a ragged batch with a long K at g = 64, bias, residual in FP32
        gemm("gemm_ragged_2000x4000x16384", 2000, 4000, 16384, g=64, bias=True, res="f32"),
        # a training forward pass: bias, GELU, residual, and the pre-activation kept
        gemm("gemm_train_8192x8192x8192", 8192, 8192, 8192, bias=True, act="gelu", pre=True),
        # the gradient through a served-size layer's GELU
        epi_bwd("epi_bwd_64x4096", 64, 4096),
        # ReLU, a ragged number of tokens, per-row factors, FP32 gradients in
        epi_bwd("epi_bwd_ragged_2000x7168_relu", 2000, 7168, act="relu", x="f32", rowa=True),
        # the training step's gradient: 128 x 128 blocks that serve both following products
        epi_bwd("epi_bwd_8192x8192", 8192, 8192),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("norm", "norm_bwd", "gemm", "epi_bwd"))
    g = rng.choice((64, 128, 128, 256))
    x = rng.choice(("bf16", "bf16", "f16", "f32"))
    if op == "gemm":
        K = g * _log(rng, max(1, 256 // g), 16384 // g)
        M = _log(rng, 1, 8192)
        N = _log(rng, 16, min(8192, max(16, 2 ** 38 // (M * K))))
        c = gemm("", M, N, K, g=g, layout=rng.choice(("nt", "nt", "nn", "tt", "tn")), rowa=rng.random() < 0.5, fa=rng.choice(("e4m3", "e4m3", "e5m2")),
                 fb=rng.choice(("e4m3", "e4m3", "e5m2")), bias=rng.random() < 0.5, act=rng.choice(ACTS), res=rng.choice(("bf16", "bf16", "f32", "f16", "none")),
                 pre=rng.random() < 0.3, pad=rng.choice((0, 0, 8, 5)))
    else:
        cols = g * _log(rng, max(1, 256 // g), 16384 // g)
        rows = _log(rng, 1, min(8192, 2 ** 26 // cols))
        res = rng.choice((x, x, "f32"))
        if op == "norm":
            res = rng.choice((res, res, "none"))
            c = norm("", rows, cols, g=g, fmt=rng.choice(("e4m3", "e4m3", "e5m2")), x=x, res=res, train=rng.random() < 0.5, pad=rng.choice((0, 0, 64)))
        elif op == "norm_bwd":
            c = norm_bwd("", rows, cols, x=x, res=res, dh=rng.random() < 0.8)
        else:
            c = epi_bwd("", rows, cols, g=g, act=rng.choice(ACTS), x=x, rowa=rng.random() < 0.5, fmt=rng.choice(("e5m2", "e4m3")), dz=rng.random() < 0.3,
                        dbias=rng.random() < 0.8)
    del c["name"]
    return c


def _cdiv(a, b):
    return -(-a // b)


class _Rand:
    """Seeded normal and uniform tensors on the GPU."""

    def __init__(self, seed):
        self.gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(self, *shape):
        return torch.randn(*shape, generator=self.gen, device="cuda")

    def uniform(self, *shape, lo=0.0, hi=1.0):
        return torch.rand(*shape, generator=self.gen, device="cuda") * (hi - lo) + lo


def _stream(r, rows, cols):
    """Hidden states as a layer meets them: rows of different size, and a few channels far larger than the rest."""
    v = r.normal(rows, cols) * torch.exp(r.uniform(rows, 1, lo=-1.0, hi=1.0))
    return v * torch.where(r.uniform(1, cols) < 0.002, 20.0, 1.0)


def _padded(v, pad):
    """v with `pad` unused elements between its rows."""
    if not pad:
        return v.contiguous()
    wide = torch.zeros(v.shape[0], v.shape[1] + pad, dtype=v.dtype, device=v.device)
    wide[:, : v.shape[1]] = v
    return wide[:, : v.shape[1]]


def _empty(shape, dtype):
    return torch.empty(shape, dtype=dtype, device="cuda")


def _codes(r, rows, cols, fmt, factor_rows, g):
    """FP8 codes of values whose blocks fill the format's range, and factors as a quantiser leaves them."""
    v = r.normal(rows, cols).clamp_(-4.5, 4.5) * (FMAX[fmt] / 4.5)
    s = torch.exp(r.uniform(_cdiv(rows, factor_rows), cols // g, lo=-1.0, hi=1.0)) / FMAX[fmt]
    return v.to(F8[fmt]), s


def prepare(case, seed):
    c, r = case, _Rand(seed)
    s = dict(case=c)
    if c["op"] == "gemm":
        M, N, K, g = c["M"], c["N"], c["K"], c["g"]
        a, s["sa"] = _codes(r, M, K, c["fa"], 1 if c["rowa"] else g, g)
        b, sb = _codes(r, N, K, c["fb"], g, g)
        s["sb"] = sb * (4.0 / math.sqrt(K))
        s["a"] = a.t().contiguous() if c["layout"][0] == "t" else a
        s["b"] = b.t().contiguous() if c["layout"][1] == "n" else b
        s["bias"] = r.normal(N) * 0.5 if c["bias"] else None
        s["res"] = _padded(_stream(r, M, N).to(TYPES[c["res"]]), c["pad"]) if c["res"] != "none" else None
        s["out"] = _empty((M, N), torch.bfloat16)
        s["pre"] = _empty((M, N), torch.bfloat16) if c["pre"] else None
        return s
    rows, cols = c["rows"], c["cols"]
    if c["op"] == "norm":
        x = _stream(r, rows, cols)
        x[rows // 2 + 1 :: 97] = 0.0  # padding tokens
        s["x"] = _padded(x.to(TYPES[c["x"]]), c["pad"])
        s["res"] = (_stream(r, rows, cols) * (x != 0)).to(TYPES[c["res"]]) if c["res"] != "none" else None
        s["w"] = 1.0 + 0.3 * r.normal(cols)
        s["h"] = _empty((rows, cols), s["res"].dtype) if s["res"] is not None else None
        s["q"], s["scales"] = _empty((rows, cols), F8[c["fmt"]]), _empty((rows, cols // c["g"]), torch.float32)
        s["y"] = _empty((rows, cols), TYPES[c["x"]]) if c["train"] else None
        s["rstd"] = _empty((rows,), torch.float32) if c["train"] else None
    elif c["op"] == "norm_bwd":
        h = _stream(r, rows, cols)
        s["h"] = h.to(TYPES[c["res"]])
        s["rstd"] = torch.rsqrt(s["h"].double().square().mean(-1) + EPS).float()
        s["dy"] = (r.normal(rows, cols) * 1e-2).to(TYPES[c["x"]])
        s["dh"] = (r.normal(rows, cols) * 1e-2).to(TYPES[c["res"]]) if c["dh"] else None
        s["w"] = 1.0 + 0.3 * r.normal(cols)
        s["dx"], s["dw"] = _empty((rows, cols), s["h"].dtype), _empty((cols,), torch.float32)
    else:
        s["dout"] = (r.normal(rows, cols) * torch.exp(r.uniform(rows, 1, lo=-2.0, hi=2.0)) * 1e-2).to(TYPES[c["x"]])
        s["pre"] = (r.normal(rows, cols) * 1.5).to(torch.bfloat16) if c["act"] != "none" else None
        s["q"] = _empty((rows, cols), F8[c["fmt"]])
        s["scales"] = _empty((rows if c["rowa"] else _cdiv(rows, c["g"]), cols // c["g"]), torch.float32)
        s["dz"] = _empty((rows, cols), TYPES[c["x"]]) if c["dz"] else None
        s["dbias"] = _empty((cols,), torch.float32) if c["dbias"] else None
    return s


# ---- the plain forms: 32 bits, rounded once at the end ------------------------


def _act(z, act):
    if act == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    if act == "silu":
        return z / (1 + torch.exp(-z))
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    return z


def _act_grad(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "gelu":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    if act == "silu":
        e = 1 / (1 + torch.exp(-z))
        return e * (1 + z * (1 - e))
    t = torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z))
    return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * z * z)


def _spread(s, factor_rows, g, rows):
    """Factors per block -> one per element."""
    return s.repeat_interleave(factor_rows, 0)[:rows].repeat_interleave(g, 1)


def _quantise(y, factor_rows, g, fmt):
    """(codes, factors) of y with one factor per factor_rows x g block."""
    rows, cols = y.shape
    n = _cdiv(rows, factor_rows)
    a = torch.zeros(n * factor_rows, cols, dtype=y.dtype, device=y.device) if n * factor_rows != rows else y
    if a is not y:
        a[:rows] = y
    s = a.abs().view(n, factor_rows, cols // g, g).amax((1, 3)) / FMAX[fmt]
    s = torch.where(s > 0, s, torch.ones_like(s))
    return (y / _spread(s, factor_rows, g, rows)).to(F8[fmt]), s


def _plain_norm(c, x, res, w):
    h = x if res is None else (x.float() + res.float()).to(res.dtype)
    hf = h.float()
    rstd = torch.rsqrt(hf.square().mean(-1) + EPS)
    y = hf * rstd[:, None] * w
    q, s = _quantise(y, 1, c["g"], c["fmt"])
    return dict(q=q, scales=s, h=None if res is None else h, y=y.to(x.dtype) if c["train"] else None, rstd=rstd if c["train"] else None)


def _plain_norm_bwd(dy, h, rstd, dh, w):
    hf, g = h.float(), dy.float()
    n = hf * rstd[:, None]
    u = g * w
    dx = rstd[:, None] * (u - n * (u * n).mean(-1, keepdim=True))
    if dh is not None:
        dx = dx + dh.float()
    return dict(dx=dx.to(h.dtype), dw=(g * n).double().sum(0).float())


def _plain_gemm(c, a, b, sa, sb, bias, res):
    g = c["g"]
    a = (a.t() if c["layout"][0] == "t" else a).float() * _spread(sa, 1 if c["rowa"] else g, g, c["M"])
    b = (b.t() if c["layout"][1] == "n" else b).float() * _spread(sb, g, g, c["N"])
    z = a @ b.t()
    if bias is not None:
        z = z + bias
    out = _act(z, c["act"])
    if res is not None:
        out = out + res.float()
    return dict(out=out.bfloat16(), pre=z.bfloat16() if c["pre"] else None)


def _plain_epi_bwd(c, dout, pre):
    dz = dout.float()
    if pre is not None:
        dz = dz * _act_grad(pre.float(), c["act"])
    q, s = _quantise(dz, 1 if c["rowa"] else c["g"], c["g"], c["fmt"])
    return dict(q=q, scales=s, dz=dz.to(dout.dtype) if c["dz"] else None, dbias=dz.double().sum(0).float() if c["dbias"] else None)


def _own(s):
    import fp8_block_scaled_scales_amd as dg

    c = s["case"]
    fmt = dict(e4m3=dg.DG_FMT_E4M3, e5m2=dg.DG_FMT_E5M2)
    act = dict(none=dg.DG_ACT_NONE, relu=dg.DG_ACT_RELU, gelu=dg.DG_ACT_GELU, silu=dg.DG_ACT_SILU, gelu_tanh=dg.DG_ACT_GELU_TANH)
    if c["op"] == "norm":
        q, scales, h = dg.dg_rmsnorm_quantize_fp8(s["x"], s["res"], s["w"], EPS, gran=c["g"], fmt=fmt[c["fmt"]], h=s["h"], y=s["y"], rstd=s["rstd"], q=s["q"],
                                                  scales=s["scales"])
        return dict(q=q, scales=scales, h=h if s["res"] is not None else None, y=s["y"], rstd=s["rstd"])
    if c["op"] == "norm_bwd":
        dx, dw = dg.dg_rmsnorm_backward(s["dy"], s["h"], s["rstd"], s["w"], dh=s["dh"], dx=s["dx"], dweight=s["dw"])
        return dict(dx=dx, dw=dw)
    if c["op"] == "gemm":
        layout = dict(nt=dg.DG_LAYOUT_NT, nn=dg.DG_LAYOUT_NN, tt=dg.DG_LAYOUT_TT, tn=dg.DG_LAYOUT_TN)
        out = dg.dg_gemm_fp8_residual(s["a"], s["b"], s["sa"], s["sb"], s["res"], s["out"], gran=c["g"], layout=layout[c["layout"]], sa_rows=1 if c["rowa"] else c["g"],
                                      fmt_a=fmt[c["fa"]], fmt_b=fmt[c["fb"]], bias=s["bias"], act=act[c["act"]], pre=s["pre"])
        return dict(out=out, pre=s["pre"])
    q, scales = dg.dg_epilogue_backward_fp8(s["dout"], s["pre"], act[c["act"]], gran=c["g"], block_rows=1 if c["rowa"] else c["g"], fmt=fmt[c["fmt"]], dz=s["dz"],
                                            dbias=s["dbias"], q=s["q"], scales=s["scales"])
    return dict(q=q, scales=scales, dz=s["dz"], dbias=s["dbias"])


def run(state):
    s, c = state, state["case"]
    if own:
        return _own(s)
    if c["op"] == "norm":
        return _plain_norm(c, s["x"], s["res"], s["w"])
    if c["op"] == "norm_bwd":
        return _plain_norm_bwd(s["dy"], s["h"], s["rstd"], s["dh"], s["w"])
    if c["op"] == "gemm":
        return _plain_gemm(c, s["a"], s["b"], s["sa"], s["sb"], s["bias"], s["res"])
    return _plain_epi_bwd(c, s["dout"], s["pre"])


def work(case):
    """Each input read once and each output written once; 2 M N K for the product."""
    c = case
    if c["op"] == "gemm":
        M, N, K, g = c["M"], c["N"], c["K"], c["g"]
        factors = (M if c["rowa"] else _cdiv(M, g)) + _cdiv(N, g)
        return dict(bytes=M * K + N * K + 4 * factors * (K // g) + M * N * (2 + SIZE[c["res"]] + 2 * c["pre"]) + 4 * N * c["bias"], flops=2.0 * M * N * K)
    rows, cols = c["rows"], c["cols"]
    n = rows * cols
    if c["op"] == "norm":
        segments = rows * (cols // c["g"])
        return dict(bytes=n * (SIZE[c["x"]] * (1 + c["train"]) + 2 * SIZE[c["res"]] + 1) + 4 * (segments + cols + rows * c["train"]), flops=8.0 * n)
    if c["op"] == "norm_bwd":
        return dict(bytes=n * (SIZE[c["x"]] + SIZE[c["res"]] * (2 + c["dh"])) + 4 * (rows + 2 * cols), flops=12.0 * n)
    factors = (rows if c["rowa"] else _cdiv(rows, c["g"])) * (cols // c["g"])
    return dict(bytes=n * (SIZE[c["x"]] * (1 + c["dz"]) + 2 * (c["act"] != "none") + 1) + 4 * (factors + cols * c["dbias"]), flops=8.0 * n)


# ---- the definitions in 64 bits -----------------------------------------------


def _cdf(z):
    return 0.5 * torch.special.erfc(-z / math.sqrt(2.0))


def _exact_act(z, act):
    """(act(z), act'(z))."""
    if act == "relu":
        return z.clamp(min=0), torch.heaviside(z, torch.zeros_like(z))
    if act == "gelu":
        return z * _cdf(z), _cdf(z) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if act in ("silu", "gelu_tanh"):
        k = 2 * math.sqrt(2 / math.pi)
        v, dv = (z, torch.ones_like(z)) if act == "silu" else (k * (z + 0.044715 * z ** 3), k * (1 + 0.134145 * z ** 2))
        p = torch.sigmoid(v)
        return z * p, p + z * p * (1 - p) * dv
    return z, torch.ones_like(z)


def _exact_codes(y, block, g, fmt):
    """FP8 codes and factors of y: the blocks by padding with zeros and pooling."""
    rows, cols = y.shape
    wide = torch.nn.functional.pad(y, (0, 0, 0, -rows % block))
    top = wide.abs().reshape(-1, block, cols // g, g).amax(3).amax(1)
    s = (top / FMAX[fmt]).float().double()  # a factor is an FP32 number
    s[s == 0] = 1.0
    by = s[torch.arange(rows, device=y.device) // block][:, torch.arange(cols, device=y.device) // g]
    return (y / by).float().to(F8[fmt]), s


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "norm":
        h = s["x"].double()
        if s["res"] is not None:
            h = (h + s["res"].double()).to(s["res"].dtype).double()  # the norm is of the stream as it is stored
        rms = (h.pow(2).sum(1) / c["cols"] + EPS).sqrt()
        y = h / rms[:, None] * s["w"].double()
        q, scales = _exact_codes(y, 1, c["g"], c["fmt"])
        return dict(q=q, scales=scales, h=h if s["res"] is not None else None, y=y if c["train"] else None, rstd=1 / rms if c["train"] else None)
    if c["op"] == "norm_bwd":
        h, dy, k = s["h"].double(), s["dy"].double(), s["rstd"].double()[:, None]
        u = dy * s["w"].double()
        dx = k * u - h * k ** 3 * ((u * h).sum(1, keepdim=True) / c["cols"])
        return dict(dx=dx + s["dh"].double() if c["dh"] else dx, dw=(dy * h * k).sum(0))
    if c["op"] == "gemm":
        g = c["g"]
        a = s["a"].double() if c["layout"][0] == "n" else s["a"].double().t()
        b = s["b"].double() if c["layout"][1] == "t" else s["b"].double().t()
        row = torch.arange(c["M"], device="cuda") // (1 if c["rowa"] else g)
        col = torch.arange(c["N"], device="cuda") // g
        z = torch.zeros(c["M"], c["N"], dtype=torch.float64, device="cuda")
        for kb in range(c["K"] // g):  # segment by segment, each restored by its factors
            p = a[:, kb * g : (kb + 1) * g] @ b[:, kb * g : (kb + 1) * g].t()
            z += p * s["sa"].double()[row, kb][:, None] * s["sb"].double()[col, kb]
        if c["bias"]:
            z += s["bias"].double()
        out = _exact_act(z, c["act"])[0]
        return dict(out=out if s["res"] is None else out + s["res"].double(), pre=z if c["pre"] else None)
    dz = s["dout"].double()
    if s["pre"] is not None:
        dz = dz * _exact_act(s["pre"].double(), c["act"])[1]
    q, scales = _exact_codes(dz, 1 if c["rowa"] else c["g"], c["g"], c["fmt"])
    return dict(q=q, scales=scales, dz=dz if c["dz"] else None, dbias=dz.sum(0) if c["dbias"] else None)

"""Cases for timing the operators of layers whose weights each row chooses: experts and low-rank adapters.

Six operators, each in its plain form (elementary torch operations in 32 bits) and as the library's calls:

  dispatch     tokens sorted by expert, and their rows as FP8 codes in that order
  combine      every token's expert outputs brought back, weighted and added (with the residual stream where there is one)
  combine_bwd  its gradient: weighted FP8 rows in expert order for the next products, and the gradient of the weights
  grouped      the experts' products on the sorted rows, with the activation (and the pre-activation where training keeps it)
  wgrad        the gradient of the experts' weights: one product over each expert's rows
  lora         the low-rank adapters of many requests at once, added to a shared projection's output
"""

import math

import torch

own = False

F8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
FMAX = {"e4m3": 448.0, "e5m2": 57344.0}
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2, "none": 0}
ACTS = ("none", "relu", "gelu", "silu", "gelu_tanh")


def dispatch(name, tokens, k, experts, cols, g=128, blocks=False, align=1, fmt="e4m3", x="bf16", idle=0.0):
    """blocks: g x g blocks of the sorted rows (else 1 x g); align: rows an expert's range is a multiple of; idle: share of the
    tokens that no expert here takes (padding, or experts on another GPU)."""
    return dict(name=name, op="dispatch", tokens=tokens, k=k, experts=experts, cols=cols, g=g, blocks=blocks, align=align, fmt=fmt, x=x, idle=idle)


def combine(name, tokens, k, experts, cols, align=1, y="bf16", res="none", weighted=True, idle=0.0):
    return dict(name=name, op="combine", tokens=tokens, k=k, experts=experts, cols=cols, align=align, y=y, res=res, weighted=weighted, idle=idle)


def combine_bwd(name, tokens, k, experts, cols, g=128, blocks=True, align=128, fmt="e5m2", x="bf16", y="bf16", idle=0.0):
    return dict(name=name, op="combine_bwd", tokens=tokens, k=k, experts=experts, cols=cols, g=g, blocks=blocks, align=align, fmt=fmt, x=x, y=y, idle=idle)


def grouped(name, tokens, k, experts, N, K, g=128, layout="nt", blocks=False, align=1, fa="e4m3", fb="e4m3", act="none", pre=False):
    """layout: second letter n: the weights are stored [K,N]; blocks: g x g factors for the rows (else one per row)."""
    return dict(name=name, op="grouped", tokens=tokens, k=k, experts=experts, N=N, K=K, g=g, layout=layout, blocks=blocks, align=align, fa=fa, fb=fb, act=act, pre=pre)


def wgrad(name, tokens, k, experts, M, N, g=128, align=128, fa="e5m2", fb="e4m3"):
    return dict(name=name, op="wgrad", tokens=tokens, k=k, experts=experts, M=M, N=N, g=g, align=align, fa=fa, fb=fb)


def lora(name, tokens, adapters, N, K, rank, x="bf16", base="bf16", idle=0.0):
    """base: the type of the shared projection's output, or "none"; idle: share of the tokens whose request has no adapter."""
    return dict(name=name, op="lora", tokens=tokens, adapters=adapters, N=N, K=K, rank=rank, x=x, base=base, idle=idle)


def listed():
    return [
        # one token being served: latency
        dispatch("dispatch_token_1x7168", 1, 8, 64, 7168),
        # a training step: every token to eight of 64 experts, in the blocks that serve the weight gradient too
        dispatch("dispatch_train_8192x4096", 8192, 8, 64, 4096, blocks=True, align=128),
        # 64 tokens being served, some of whose experts are elsewhere, added to the residual stream
        combine("combine_decode_64x4096", 64, 8, 64, 4096, res="bf16", idle=0.1),
        # the training step's outputs
        combine("combine_train_8192x4096", 8192, 8, 64, 4096, align=128),
        # the gradient of a ragged batch over few experts, FP32 gradients in, one factor per row
        combine_bwd("combine_bwd_ragged_2000x7168", 2000, 2, 8, 7168, g=64, blocks=False, align=64, x="f32"),
        # the training step's gradient
        combine_bwd("combine_bwd_8192x4096", 8192, 8, 64, 4096),
        # 64 tokens being served: a few rows for each of 64 experts, whose weights are read once
        grouped("grouped_decode_64x8_4096x2048", 64, 8, 64, 4096, 2048, act="silu"),
        # a training forward pass: unequal numbers of rows per expert, pre-activation kept
        grouped("grouped_train_8192x4_8192x2048", 8192, 4, 32, 8192, 2048, blocks=True, align=128, act="gelu", pre=True),
        # a ragged batch's weight gradient at g = 64
        wgrad("wgrad_ragged_2000x2_4096x2048", 2000, 2, 8, 4096, 2048, g=64, align=64),
        # the training step's weight gradient
        wgrad("wgrad_train_8192x4_8192x2048", 8192, 4, 32, 8192, 2048),
        # 64 requests being served, a token each, most with an adapter of their own
        lora("lora_decode_64x4096x7168_r16", 64, 128, 4096, 7168, 16, idle=0.1),
        # prompts of a few requests
        lora("lora_prompt_8192x4096x4096_r64", 8192, 8, 4096, 4096, 64),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))


def draw(rng):
    op = rng.choice(("dispatch", "combine", "combine_bwd", "grouped", "wgrad", "lora"))
    g = rng.choice((64, 128, 128, 256))
    x = rng.choice(("bf16", "bf16", "f16", "f32"))
    fa, fb = rng.choice(("e4m3", "e4m3", "e5m2")), rng.choice(("e4m3", "e4m3", "e5m2"))
    idle = rng.choice((0.0, 0.0, 0.1, 0.6))
    if op == "lora":
        N, K = _log(rng, 17, 8192), 8 * _log(rng, 8, 1024)
        tokens = _log(rng, 1, min(8192, 2 ** 25 // max(N, K)))
        c = lora("", tokens, _log(rng, 1, 256), N, K, 8 * _log(rng, 1, 16), x=rng.choice(("bf16", "bf16", "f16")), base=rng.choice(("bf16", "bf16", "f16", "f32", "none")),
                 idle=idle)
    else:
        experts = _log(rng, 1, 128)
        k = min(experts, rng.choice((1, 2, 4, 6, 8)))
        tokens = _log(rng, 1, 8192)
        blocks = rng.random() < 0.5
        align = g if blocks else rng.choice((1, 1, 16, 128))
        if op in ("grouped", "wgrad"):
            g = min(g, 128) if op == "wgrad" else g
            tokens = _log(rng, 1, 8192 * 4 // k)
            K = g * _log(rng, max(1, 256 // g), 8192 // g)
            N = _log(rng, 16, min(8192, 2 ** 29 // (experts * K), max(16, 2 ** 38 // (tokens * k * K))))
            if op == "grouped":
                c = grouped("", tokens, k, experts, N, K, g=g, layout=rng.choice(("nt", "nt", "nn")), blocks=blocks, align=align, fa=fa, fb=fb, act=rng.choice(ACTS),
                            pre=rng.random() < 0.3)
            else:
                c = wgrad("", tokens, k, experts, K, max(g, N // g * g), g=g, align=g * rng.choice((1, 1, 2)), fa=fa, fb=fb)
        else:
            cols = g * _log(rng, max(1, 256 // g), 8192 // g)
            tokens = _log(rng, 1, min(8192, 2 ** 27 // (cols * k)))
            if op == "dispatch":
                c = dispatch("", tokens, k, experts, cols, g=g, blocks=blocks, align=align, fmt=fa, x=x, idle=idle)
            elif op == "combine":
                c = combine("", tokens, k, experts, cols, align=align, y=x, res=rng.choice(("none", x, "f32")), weighted=rng.random() < 0.7, idle=idle)
            else:
                c = combine_bwd("", tokens, k, experts, cols, g=g, blocks=blocks, align=align, fmt=fb, x=x, y=rng.choice(("bf16", x)), idle=idle)
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


def _routing(r, tokens, k, experts, idle):
    """(ids [tokens,k], weights): each token's k best of experts some of which are liked more than others; -1: no expert here."""
    liked = r.normal(1, experts) * 0.7
    score, ids = torch.topk(r.normal(tokens, experts) + liked, k, dim=1)
    away = r.uniform(tokens, 1) < idle
    return torch.where(away, -1, ids).int(), torch.softmax(score, 1)


def _rows(tokens, k, groups, align):
    """Rows that hold any routing of tokens * k slots."""
    n = tokens * k
    return (n + min(groups, n) * (align - 1)) // align * align


def _empty(shape, dtype):
    return torch.empty(shape, dtype=dtype, device="cuda")


def _zeros(shape, dtype):
    return torch.zeros(shape, dtype=torch.uint8 if "float8" in str(dtype) else dtype, device="cuda").view(dtype)


def _codes(r, rows, cols, fmt, factor_rows, g):
    """FP8 codes of values whose blocks fill the format's range, and factors as a quantiser leaves them."""
    v = r.normal(rows, cols).clamp_(-4.5, 4.5) * (FMAX[fmt] / 4.5)
    s = torch.exp(r.uniform(_cdiv(rows, factor_rows), cols // g, lo=-1.0, hi=1.0)) / FMAX[fmt]
    return v.to(F8[fmt]), s


def _row_codes(r, live, cols, fmt, factor_rows, g):
    """The same for sorted rows, of which those between the groups hold zeros."""
    q, s = _codes(r, live.numel(), cols, fmt, factor_rows, g)
    return torch.where(live[:, None], q.view(torch.uint8), 0).view(q.dtype), s


def prepare(case, seed):
    c, r = case, _Rand(seed)
    s = dict(case=c)
    if c["op"] == "lora":
        T, G, N, K, rank = c["tokens"], c["adapters"], c["N"], c["K"], c["rank"]
        ids, _ = _routing(r, T, 1, G, c["idle"])
        s["offsets"], s["position"], s["slot"] = _plain_sort(ids, G, 1, T)  # kept for all projections of a step
        s["top"] = _largest(s["offsets"])
        s["x"] = _stream(r, T, K).to(TYPES[c["x"]])
        s["a"] = (r.normal(G, rank, K) / math.sqrt(K)).to(TYPES[c["x"]])
        s["b"] = (r.normal(G, N, rank) / math.sqrt(rank)).to(TYPES[c["x"]])
        s["scale"] = r.uniform(G, lo=0.25, hi=2.0)
        kind = TYPES[c["x"] if c["base"] == "none" else c["base"]]
        s["base"] = _stream(r, T, N).to(kind) if c["base"] != "none" else None
        s["out"] = _empty((T, N), kind)
        return s
    T, k, E = c["tokens"], c["k"], c["experts"]
    ids, weights = _routing(r, T, k, E, c.get("idle", 0.0))
    R = _rows(T, k, E, c["align"])
    offsets, position, slot = _plain_sort(ids, E, c["align"], R)
    live = slot >= 0
    if c["op"] == "dispatch":
        g, cols = c["g"], c["cols"]
        s["ids"], s["x"] = ids, _stream(r, T, cols).to(TYPES[c["x"]])
        s["offsets"], s["position"], s["slot"] = _empty((E + 1,), torch.int32), _empty((T, k), torch.int32), _empty((R,), torch.int32)
        # rows past the last expert's stay as they were
        s["q"], s["scales"] = _zeros((R, cols), F8[c["fmt"]]), _zeros((_cdiv(R, g if c["blocks"] else 1), cols // g), torch.float32)
        return s
    s["offsets"], s["position"], s["slot"] = offsets, position, slot
    if c["op"] == "combine":
        cols = c["cols"]
        s["y"] = torch.where(live[:, None], r.normal(R, cols), 0.0).to(TYPES[c["y"]])
        s["res"] = _stream(r, T, cols).to(TYPES[c["res"]]) if c["res"] != "none" else None
        s["weights"] = weights if c["weighted"] else None
        s["out"] = _empty((T, cols), TYPES[c["y"] if c["res"] == "none" else c["res"]])
    elif c["op"] == "combine_bwd":
        g, cols = c["g"], c["cols"]
        s["weights"] = weights
        s["dout"] = (r.normal(T, cols) * torch.exp(r.uniform(T, 1, lo=-2.0, hi=2.0)) * 1e-2).to(TYPES[c["x"]])
        s["y"] = torch.where(live[:, None], r.normal(R, cols), 0.0).to(TYPES[c["y"]])
        s["q"], s["scales"] = _zeros((R, cols), F8[c["fmt"]]), _zeros((_cdiv(R, g if c["blocks"] else 1), cols // g), torch.float32)
        s["dweights"] = _empty((T, k), torch.float32)
    elif c["op"] == "grouped":
        N, K, g = c["N"], c["K"], c["g"]
        s["top"] = _largest(offsets)
        s["a"], s["sa"] = _row_codes(r, live, K, c["fa"], g if c["blocks"] else 1, g)
        b, sb = _codes(r, E * N, K, c["fb"], E * N, g)
        b = b.view(E, N, K)
        s["b"] = b.transpose(1, 2).contiguous() if c["layout"][1] == "n" else b
        s["sb"] = torch.exp(r.uniform(E, _cdiv(N, g), K // g, lo=-1.0, hi=1.0)) * (4.0 / math.sqrt(K) / FMAX[c["fb"]])
        s["out"] = _zeros((R, N), torch.bfloat16)
        s["pre"] = _zeros((R, N), torch.bfloat16) if c["pre"] else None
    else:
        M, N, g = c["M"], c["N"], c["g"]
        s["top"] = _largest(offsets)
        s["a"], s["sa"] = _row_codes(r, live, M, c["fa"], g, g)
        s["b"], s["sb"] = _row_codes(r, live, N, c["fb"], g, g)
        s["out"] = _empty((E, M, N), torch.bfloat16)
    return s


# ---- the plain forms: 32 bits, rounded once at the end ------------------------


def _largest(offsets):
    """Rows of the largest group, as the host knows them."""
    return max(1, int((offsets[1:] - offsets[:-1]).max()))


def _plain_sort(ids, groups, align, rows):
    """(offsets, position, slot): a stable sort by group, each group from a multiple of align rows on."""
    T, k = ids.shape
    flat = ids.reshape(-1)
    key = torch.where((flat >= 0) & (flat < groups), flat, groups).long()
    count = (key[:, None] == torch.arange(groups + 1, device=key.device)).sum(0)
    wide = torch.div(count + align - 1, align, rounding_mode="floor") * align
    zero = torch.zeros(1, dtype=torch.int64, device=key.device)
    start, first = torch.cat([zero, wide.cumsum(0)]), torch.cat([zero, count.cumsum(0)])
    kept, order = torch.sort(key, stable=True)
    at = torch.arange(T * k, device=key.device) - first[kept] + start[kept]
    position = torch.empty_like(key)
    position[order] = torch.where(kept < groups, at, -1)
    row = torch.arange(rows, device=key.device)
    slot = torch.cat([torch.where(row < start[groups], -1, -2), zero])  # the last entry takes what is dropped
    slot[torch.where(kept < groups, at, rows)] = order
    return start[: groups + 1].int(), position.view(T, k).int(), slot[:rows].int()


def _spread(s, factor_rows, g, rows):
    """Factors per block -> one per element."""
    return s.repeat_interleave(factor_rows, 0)[:rows].repeat_interleave(g, 1)


def _quantise(y, factor_rows, g, fmt):
    """(codes, factors) of y with one factor per factor_rows x g block."""
    rows, cols = y.shape
    s = y.abs().view(rows // factor_rows, factor_rows, cols // g, g).amax((1, 3)) / FMAX[fmt]
    s = torch.where(s > 0, s, torch.ones_like(s))
    return (y / _spread(s, factor_rows, g, rows)).to(F8[fmt]), s


def _gather(x, slot, k, weights):
    """Rows of x in sorted order, weighted; zeros where there is none."""
    at = slot.long().clamp(min=0)
    v = x[torch.div(at, k, rounding_mode="floor")].float()
    if weights is not None:
        v = v * weights.reshape(-1)[at][:, None]
    return torch.where((slot >= 0)[:, None], v, torch.zeros_like(v))


def _plain_rows(c, x, slot, offsets, weights):
    """The sorted rows' codes and factors; rows past the last group's are zeros, with factors of zero."""
    rows = 1 if not c["blocks"] else c["g"]
    q, s = _quantise(_gather(x, slot, c["k"], weights), rows, c["g"], c["fmt"])
    first = torch.arange(s.shape[0], device=s.device) * rows
    return q, torch.where((first < offsets[-1])[:, None], s, torch.zeros_like(s))


def _plain_combine(y, position, weights, res, kind):
    at = position.long().clamp(min=0)
    v = y[at].float()
    if weights is not None:
        v = v * weights[:, :, None]
    out = torch.where((position >= 0)[:, :, None], v, torch.zeros_like(v)).sum(1)
    return (out if res is None else out + res.float()).to(kind)


def _plain_weight_grad(dout, y, position):
    v = (dout.float()[:, None, :] * y[position.long().clamp(min=0)].float()).double().sum(2).float()
    return torch.where(position >= 0, v, torch.zeros_like(v))


def _grid(offsets, top):
    """(row of every group's i-th row, whether it has one)."""
    at = offsets[:-1, None].long() + torch.arange(top, device=offsets.device)
    return at, at < offsets[1:, None]


def _by_group(v, offsets, top):
    """Rows by group, [groups, top, cols], zeros past a group's end."""
    at, has = _grid(offsets, top)
    return torch.where(has[:, :, None], v[at.clamp(max=v.shape[0] - 1)], torch.zeros((), dtype=v.dtype, device=v.device))


def _back(v, offsets, top, rows):
    """The reverse: [groups, top, cols] to [rows, cols], zeros where no group has the row."""
    at, has = _grid(offsets, top)
    out = torch.zeros(rows + 1, v.shape[2], dtype=v.dtype, device=v.device)
    out[torch.where(has, at, rows).reshape(-1)] = v.reshape(-1, v.shape[2])
    return out[:rows]


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


def _plain_grouped(c, a, b, sa, sb, offsets, top):
    g, R = c["g"], a.shape[0]
    af = a.float() * _spread(sa, g if c["blocks"] else 1, g, R)
    bf = b.float() if c["layout"][1] == "t" else b.float().transpose(1, 2)
    bf = bf * sb.repeat_interleave(g, 1)[:, : c["N"]].repeat_interleave(g, 2)
    z = _back(torch.bmm(_by_group(af, offsets, top), bf.transpose(1, 2).contiguous()), offsets, top, R)
    return dict(out=_act(z, c["act"]).bfloat16(), pre=z.bfloat16() if c["pre"] else None)


def _plain_wgrad(c, a, b, sa, sb, offsets, top):
    g, R = c["g"], a.shape[0]
    af = _by_group(a.float() * _spread(sa, g, g, R), offsets, top)
    bf = _by_group(b.float() * _spread(sb, g, g, R), offsets, top)
    return dict(out=torch.bmm(af.transpose(1, 2).contiguous(), bf).bfloat16())


def _plain_lora(c, x, a, b, scale, base, offsets, slot, top, kind):
    T = x.shape[0]
    live = slot >= 0
    v = torch.bmm(_by_group(x[slot.long().clamp(min=0)].float(), offsets, top), a.float().transpose(1, 2).contiguous())
    d = _back(torch.bmm(v * scale[:, None, None], b.float().transpose(1, 2).contiguous()), offsets, top, T)
    out = torch.zeros(T + 1, d.shape[1], device=d.device)
    out[torch.where(live, slot.long(), T)] = d
    return dict(out=(out[:T] if base is None else base.float() + out[:T]).to(kind))


def _own(s):
    import fp8_block_scaled_scales_amd as dg

    c = s["case"]
    fmt = dict(e4m3=dg.DG_FMT_E4M3, e5m2=dg.DG_FMT_E5M2)
    if c["op"] == "dispatch":
        dg.dg_route_sort(s["ids"], c["experts"], align=c["align"], offsets=s["offsets"], position=s["position"], slot=s["slot"])
        q, scales = dg.dg_route_quantize_fp8(s["x"], s["position"], s["slot"], gran=c["g"], block_rows=c["g"] if c["blocks"] else 1, fmt=fmt[c["fmt"]], q=s["q"],
                                             scales=s["scales"])
        return dict(offsets=s["offsets"], position=s["position"], slot=s["slot"], q=q, scales=scales)
    if c["op"] == "combine":
        return dict(out=dg.dg_route_combine(s["y"], s["position"], weights=s["weights"], res=s["res"], out=s["out"]))
    if c["op"] == "combine_bwd":
        q, scales = dg.dg_route_quantize_fp8(s["dout"], s["position"], s["slot"], weights=s["weights"], gran=c["g"], block_rows=c["g"] if c["blocks"] else 1,
                                             fmt=fmt[c["fmt"]], q=s["q"], scales=s["scales"])
        return dict(q=q, scales=scales, dweights=dg.dg_route_weight_grad(s["dout"], s["y"], s["position"], dweights=s["dweights"]))
    if c["op"] == "grouped":
        act = dict(none=dg.DG_ACT_NONE, relu=dg.DG_ACT_RELU, gelu=dg.DG_ACT_GELU, silu=dg.DG_ACT_SILU, gelu_tanh=dg.DG_ACT_GELU_TANH)
        out = dg.dg_gemm_fp8_grouped(s["a"], s["b"], s["sa"], s["sb"], s["offsets"], out=s["out"], gran=c["g"], layout=dict(nt=dg.DG_LAYOUT_NT, nn=dg.DG_LAYOUT_NN)[c["layout"]],
                                     sa_rows=c["g"] if c["blocks"] else 1, fmt_a=fmt[c["fa"]], fmt_b=fmt[c["fb"]], act=act[c["act"]], pre=s["pre"])
        return dict(out=out, pre=s["pre"])
    if c["op"] == "wgrad":
        return dict(out=dg.dg_gemm_fp8_grouped_wgrad(s["a"], s["b"], s["sa"], s["sb"], s["offsets"], out=s["out"], gran=c["g"], fmt_a=fmt[c["fa"]], fmt_b=fmt[c["fb"]]))
    return dict(out=dg.dg_lora(s["x"], s["a"], s["b"], s["offsets"], s["position"], s["slot"], scale=s["scale"], base=s["base"], out=s["out"]))


def run(state):
    s, c = state, state["case"]
    if own:
        return _own(s)
    if c["op"] == "dispatch":
        offsets, position, slot = _plain_sort(s["ids"], c["experts"], c["align"], s["slot"].shape[0])
        q, scales = _plain_rows(c, s["x"], slot, offsets, None)
        return dict(offsets=offsets, position=position, slot=slot, q=q, scales=scales)
    if c["op"] == "combine":
        return dict(out=_plain_combine(s["y"], s["position"], s["weights"], s["res"], s["out"].dtype))
    if c["op"] == "combine_bwd":
        q, scales = _plain_rows(c, s["dout"], s["slot"], s["offsets"], s["weights"])
        return dict(q=q, scales=scales, dweights=_plain_weight_grad(s["dout"], s["y"], s["position"]))
    if c["op"] == "grouped":
        return _plain_grouped(c, s["a"], s["b"], s["sa"], s["sb"], s["offsets"], s["top"])
    if c["op"] == "wgrad":
        return _plain_wgrad(c, s["a"], s["b"], s["sa"], s["sb"], s["offsets"], s["top"])
    return _plain_lora(c, s["x"], s["a"], s["b"], s["scale"], s["base"], s["offsets"], s["slot"], s["top"], s["out"].dtype)


def work(case):
    """Each input read once and each output written once. Rows and experts as they are expected: all tokens that are not idle, experts
    that some row takes."""
    c = case
    live = 1.0 - c.get("idle", 0.0)
    if c["op"] == "lora":
        T, N, K, r = c["tokens"], c["N"], c["K"], c["rank"]
        used = c["adapters"] * (1 - (1 - 1 / c["adapters"]) ** (live * T))
        e, o = SIZE[c["x"]], SIZE[c["x"] if c["base"] == "none" else c["base"]]
        return dict(bytes=int(live * T * K * e + used * r * (K + N) * e + T * N * (o + SIZE[c["base"]]) + 12 * T), flops=2.0 * live * T * r * (K + N))
    T, k, E = c["tokens"], c["k"], c["experts"]
    n = live * T * k
    if c["op"] in ("dispatch", "combine_bwd"):
        cols, e = c["cols"], SIZE[c["x"]]
        factors = n / (c["g"] if c["blocks"] else 1) * (cols // c["g"])
        moved = live * T * cols * e + n * cols + 4 * factors + 4 * (2 * T * k + _rows(T, k, E, c["align"]))
        if c["op"] == "combine_bwd":
            moved += n * cols * SIZE[c["y"]] + 8 * T * k
        return dict(bytes=int(moved), flops=(4.0 if c["op"] == "dispatch" else 7.0) * n * cols)
    if c["op"] == "combine":
        cols = c["cols"]
        return dict(bytes=int(n * cols * SIZE[c["y"]] + T * cols * (SIZE[c["res"]] + SIZE[c["y"] if c["res"] == "none" else c["res"]]) + 4 * T * k * (1 + c["weighted"])),
                    flops=2.0 * n * cols)
    used = E * (1 - (1 - 1 / E) ** n)
    if c["op"] == "grouped":
        N, K, g = c["N"], c["K"], c["g"]
        return dict(bytes=int(n * K + used * N * K + 4 * (n / (g if c["blocks"] else 1) * (K // g) + used * _cdiv(N, g) * (K // g)) + 2 * n * N * (1 + c["pre"])), flops=2.0 * n * N * K)
    M, N, g = c["M"], c["N"], c["g"]
    return dict(bytes=int(n * (M + N) + 4 * n / g * (M + N) // g + 2 * E * M * N), flops=2.0 * n * M * N)


# ---- the definitions in 64 bits -----------------------------------------------


def _exact_sort(ids, groups, align, rows):
    """By counting: a slot's row is its group's start and the number of its group's slots before it."""
    T, k = ids.shape
    flat = ids.reshape(-1).cpu().tolist()
    filled = [0] * groups
    rank = []
    for e in flat:
        ok = 0 <= e < groups
        rank.append(filled[e] if ok else -1)
        if ok:
            filled[e] += 1
    starts = [0]
    for n in filled:
        starts.append(starts[-1] + -(-n // align) * align)
    slot = [-1] * starts[-1] + [-2] * (rows - starts[-1])
    position = [-1 if r < 0 else starts[e] + r for e, r in zip(flat, rank)]
    for i, p in enumerate(position):
        if p >= 0:
            slot[p] = i
    t = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    return t(starts), t(position).view(T, k), t(slot)


def _exact_codes(y, block, g, fmt, end):
    """FP8 codes and factors of the sorted rows y, zeros from row `end` on."""
    rows, cols = y.shape
    top = y.abs().reshape(rows // block, block, cols // g, g).amax(3).amax(1)
    s = (top / FMAX[fmt]).float().double()  # a factor is an FP32 number
    s[s == 0] = 1.0
    by = s[torch.arange(rows, device=y.device) // block][:, torch.arange(cols, device=y.device) // g]
    q = (y / by).float().to(F8[fmt])
    s[-(-end // block):] = 0.0
    return q, s


def _exact_rows(c, x, slot, end, weights):
    y = torch.zeros(slot.numel(), c["cols"], dtype=torch.float64, device="cuda")
    r = torch.nonzero(slot >= 0)[:, 0]
    i = slot[r].long()
    y[r] = x.double()[i // c["k"]]
    if weights is not None:
        y[r] = (y[r] * weights.double().reshape(-1)[i][:, None]).float().double()  # the codes are of an FP32 number
    return _exact_codes(y, c["g"] if c["blocks"] else 1, c["g"], c["fmt"], end)


def _exact_act(z, act):
    if act == "relu":
        return z.clamp(min=0)
    if act == "gelu":
        return z * 0.5 * torch.special.erfc(-z / math.sqrt(2.0))
    if act == "silu":
        return z * torch.sigmoid(z)
    if act == "gelu_tanh":
        return z * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))
    return z


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "dispatch":
        offsets, position, slot = _exact_sort(s["ids"], c["experts"], c["align"], s["slot"].shape[0])
        q, scales = _exact_rows(c, s["x"], slot, int(offsets[-1]), None)
        return dict(offsets=offsets, position=position, slot=slot, q=q, scales=scales)
    ends = s["offsets"].cpu().tolist()
    if c["op"] == "combine":
        out = torch.zeros(c["tokens"], c["cols"], dtype=torch.float64, device="cuda")
        if s["res"] is not None:
            out += s["res"].double()
        for j in range(c["k"]):
            t = torch.nonzero(s["position"][:, j] >= 0)[:, 0]
            v = s["y"][s["position"][t, j].long()].double()
            out[t] += v if s["weights"] is None else v * s["weights"][t, j].double()[:, None]
        return dict(out=out)
    if c["op"] == "combine_bwd":
        q, scales = _exact_rows(c, s["dout"], s["slot"], ends[-1], s["weights"])
        dw = torch.zeros(c["tokens"], c["k"], dtype=torch.float64, device="cuda")
        for j in range(c["k"]):
            t = torch.nonzero(s["position"][:, j] >= 0)[:, 0]
            dw[t, j] = (s["dout"][t].double() * s["y"][s["position"][t, j].long()].double()).sum(1)
        return dict(q=q, scales=scales, dweights=dw)
    if c["op"] == "grouped":
        g, N, K = c["g"], c["N"], c["K"]
        z = torch.zeros(s["a"].shape[0], N, dtype=torch.float64, device="cuda")
        col = torch.arange(N, device="cuda") // g
        for e, (lo, hi) in enumerate(zip(ends, ends[1:])):
            if hi == lo:
                continue
            b = s["b"][e].double() if c["layout"][1] == "t" else s["b"][e].double().t()
            row = torch.arange(lo, hi, device="cuda") // (g if c["blocks"] else 1)
            by_a = s["sa"].double()[row].repeat_interleave(g, 1)
            by_b = s["sb"][e].double()[col].repeat_interleave(g, 1)
            z[lo:hi] = (s["a"][lo:hi].double() * by_a) @ (b * by_b).t()
        return dict(out=_exact_act(z, c["act"]), pre=z if c["pre"] else None)
    if c["op"] == "wgrad":
        g = c["g"]
        out = torch.zeros(c["experts"], c["M"], c["N"], dtype=torch.float64, device="cuda")
        for e, (lo, hi) in enumerate(zip(ends, ends[1:])):
            if hi > lo:
                row = torch.arange(lo, hi, device="cuda") // g
                a, b = (s[n][lo:hi].double() * s["s" + n].double()[row].repeat_interleave(g, 1) for n in "ab")
                out[e] = a.t() @ b
        return dict(out=out)
    out = torch.zeros(c["tokens"], c["N"], dtype=torch.float64, device="cuda")
    for e, (lo, hi) in enumerate(zip(ends, ends[1:])):
        if hi > lo:
            t = s["slot"][lo:hi].long()
            out[t] = s["scale"][e].double() * ((s["x"][t].double() @ s["a"][e].double().t()) @ s["b"][e].double().t())
    return dict(out=out if s["base"] is None else out + s["base"].double())

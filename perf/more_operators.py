"""Measured cases of the mixture-of-experts layer around the grouped GEMM.

Seven passes: the router (``route``) and its gradient (``route_bwd``); the pairs sorted by expert
and the tokens' rows laid out in that order (``dispatch``); the experts' rows back to their tokens
with the router's weights (``combine``, also the dispatch's gradient, without weights) and its
gradient (``combine_bwd``); the gated product of two projections with an 8-bit checkpoint of its
pre-activations (``ckpt``), and its gradient from that checkpoint (``ckpt_bwd``).

``run`` computes each in plain torch where ``own`` is false, and calls the library where it is
true. ``exact`` gives the same outputs from the definitions in 64 bits.

Shapes are those of the benchmark's expert workload: 256 experts, 8 a token, K = 7168 channels,
F = 2048 feed-forward columns of an expert; odd ones beside them.
"""
import math

import torch

own = False

DEV = "cuda"
QMAX = 448.0           # largest finite e4m3fn value
Q_EPS = 1e-10          # floor of a group's largest magnitude
RENORM_EPS = 1e-20     # added to the sum that router weights are divided by


# ------------------------------------------------------------------------------ cases

def listed():
    return [
        # one decode step's router: sigmoid scores, a bias that balances the load, expert groups
        dict(name="route_decode_8", op="route", T=8, E=256, topk=8, score="sigmoid", bias=True,
             groups=8, topk_groups=4, renorm=True, x="fp32", mask=False),
        # a prompt's: the plain form of most models, 16-bit logits with experts masked out
        dict(name="route_prefill_4096", op="route", T=4096, E=256, topk=8, score="softmax",
             bias=False, groups=1, topk_groups=1, renorm=False, x="bf16", mask=True),
        # a training batch's router gradient
        dict(name="route_bwd_4096", op="route_bwd", T=4096, E=256, topk=8, score="sigmoid",
             renorm=True, x="fp32", mask=False),
        # a prompt's tokens, quantized on the way into expert order
        dict(name="dispatch_prefill_4096", op="dispatch", T=4096, K=7168, E=256, topk=8,
             drop=False, inp="bf16", out="codes", layout="row", scales="fp32"),
        # one of eight GPUs that share the experts: codes from the norm step, most pairs elsewhere
        dict(name="dispatch_shard_777", op="dispatch", T=777, K=7168, E=32, topk=8, drop=True,
             inp="codes", out="codes", layout="col", scales="fp32"),
        # a decode step's experts back to their token, beside a shared expert's output
        dict(name="combine_decode_1", op="combine", T=1, K=7168, E=256, topk=8, drop=False,
             order="pair", rows="bf16", weights=True, base=True, out="bf16", ckpt=False),
        # a training batch's, keeping the rows in 8 bits for the weights' gradient; the largest
        dict(name="combine_train_4096", op="combine", T=4096, K=7168, E=256, topk=8, drop=False,
             order="expert", rows="bf16", weights=True, base=True, out="bf16", ckpt=True),
        # its gradient from those 8 bits, as codes for the next grouped GEMM
        dict(name="combine_bwd_4096", op="combine_bwd", T=4096, K=7168, E=256, topk=8, drop=False,
             order="expert", rows="codes", dout="bf16", out="codes", layout="row", scales="fp32"),
        # an odd batch on some of the experts, 16-bit rows in pair order, a gradient in 32 bits
        dict(name="combine_bwd_odd_333", op="combine_bwd", T=333, K=1544, E=24, topk=6, drop=True,
             order="pair", rows="bf16", dout="fp32", out="bf16", layout="row", scales="fp32"),
        # the product between an expert's two GEMMs, its pre-activations kept in 8 bits
        dict(name="ckpt_train_32768", op="ckpt", M=32768, F=2048, act="silu", h="codes",
             layout="row", scales="fp32"),
        # a few rows, powers of two
        dict(name="ckpt_small_52", op="ckpt", M=52, F=1536, act="gelu_tanh", h="codes",
             layout="col", scales="ue8m0"),
        # the gradient from the 8 bits, as codes for the next grouped GEMM
        dict(name="ckpt_bwd_32768", op="ckpt_bwd", M=32768, F=2048, act="silu", out="codes",
             layout="row", scales="fp32"),
    ]


def draw(rng):
    def log(lo, hi, step=1):
        return max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step)) * step)

    op = rng.choice(["route", "route_bwd", "dispatch", "combine", "combine", "combine_bwd",
                     "ckpt", "ckpt_bwd"])
    layout, scales = rng.choice(["row", "col"]), rng.choice(["fp32", "ue8m0"])
    if op in ("ckpt", "ckpt_bwd"):
        F = log(256, 8192, 128)
        M = log(1, max(2, min(32768, 32768 * 2048 // F)))
        c = dict(op=op, M=M, F=F, act=rng.choice(["silu", "gelu_tanh"]), layout=layout,
                 scales=scales)
        if op == "ckpt":
            c["h"] = rng.choice(["codes", "bf16"])
        else:
            c["out"] = rng.choice(["codes", "bf16", "bf16_h"])
        return c
    T, topk = log(1, 4096), rng.choice([1, 2, 3, 4, 6, 8])
    if op in ("route", "route_bwd"):
        score, groups = rng.choice(["softmax", "sigmoid"]), rng.choice([1, 1, 4, 8])
        E = groups * log(16, 512 // groups) if groups > 1 else log(16, 512)
        c = dict(op=op, T=T, E=E, topk=topk, score=score, x=rng.choice(["fp32", "bf16"]),
                 renorm=rng.random() < 0.5 and topk > 1, mask=rng.random() < 0.3)
        if op == "route":
            c.update(bias=rng.random() < 0.5, groups=groups, topk_groups=max(1, groups // 2))
        return c
    E, drop = log(8, 256), rng.random() < 0.4
    if op == "dispatch":
        inp = rng.choice(["bf16", "codes"])
        out = "codes" if inp == "codes" else rng.choice(["codes", "bf16"])
        K = log(512, 7168, 128) if out == "codes" else log(256, 7168, 8)
        return dict(op=op, T=T, K=K, E=E, topk=topk, drop=drop, inp=inp, out=out, layout=layout,
                    scales=scales)
    order, weights = rng.choice(["pair", "expert"]), rng.random() < 0.7
    if op == "combine":
        ckpt = rng.random() < 0.3
        rows = rng.choice(["bf16", "bf16", "fp32"])
        if rows == "fp32":             # twice the bytes a row
            T = min(T, 2048)
        return dict(op=op, T=T, K=log(512, 7168, 128) if ckpt else log(256, 7168, 8), E=E,
                    topk=topk, drop=drop, order=order, rows=rows, weights=weights,
                    base=rng.random() < 0.5, out=rng.choice(["bf16", "fp32"]), ckpt=ckpt)
    rows, out = rng.choice(["bf16", "codes"]), rng.choice(["bf16", "codes"])
    eights = rows == "bf16" and out == "bf16"
    return dict(op=op, T=T, K=log(256, 7168, 8) if eights else log(512, 7168, 128), E=E, topk=topk,
                drop=drop, order=order, rows=rows, dout=rng.choice(["bf16", "fp32"]), out=out,
                layout=layout, scales=scales)


_BYTES = {"bf16": 2, "fp32": 4, "codes": 1}


def work(c):
    if c["op"] in ("ckpt", "ckpt_bwd"):
        M, F = c["M"], c["F"]
        kept = 2 * M * F + 8 * M * (F // 128)          # codes and scales of both halves
        if c["op"] == "ckpt":
            out = M * F + 4 * M * (F // 128) if c["h"] == "codes" else 2 * M * F
            return {"bytes": float(4 * M * F + kept + out), "flops": 14.0 * M * F}
        out = {"codes": kept, "bf16": 4 * M * F, "bf16_h": 6 * M * F}[c["out"]]
        return {"bytes": float(kept + 2 * M * F + out), "flops": 20.0 * M * F}
    T, topk = c["T"], c["topk"]
    P = T * topk
    if c["op"] == "route":
        return {"bytes": float(T * c["E"] * _BYTES[c["x"]] + 8 * P + 4 * c["E"] * c["bias"]),
                "flops": 8.0 * T * c["E"]}
    if c["op"] == "route_bwd":
        return {"bytes": float(2 * T * c["E"] * _BYTES[c["x"]] + 8 * P),
                "flops": 8.0 * T * c["E"]}
    K = c["K"]
    live = P * (c["E"] / (4 * c["E"])) if c["drop"] else P    # a quarter of the experts is here

    def row(kind):
        return _BYTES[kind] * K + (4 * (K // 128) if kind == "codes" else 0)

    if c["op"] == "dispatch":
        return {"bytes": float(T * row(c["inp"]) + live * row(c["out"]) + 8 * P + 4 * c["E"]),
                "flops": 4.0 * T * K}
    if c["op"] == "combine":
        b = live * row(c["rows"]) + T * K * _BYTES[c["out"]] * (2 if c["base"] else 1)
        b += live * row("codes") if c["ckpt"] else 0
        return {"bytes": float(b + 8 * P), "flops": 2.0 * live * K}
    b = T * K * _BYTES[c["dout"]] + live * (row(c["rows"]) + row(c["out"]))
    return {"bytes": float(b + 12 * P), "flops": 3.0 * live * K}


# ------------------------------------------------------------------- formats, plain form

def _pow2_ceil(s):
    """The smallest power of two >= s (s positive)."""
    m, e = torch.frexp(s)
    return torch.ldexp(torch.ones_like(s), torch.where(m == 0.5, e - 1, e))


def _quant_groups(x, ue8m0):
    """fp32 [M, K] -> e4m3fn codes [M, K] and one scale per 128 columns [M, K/128]."""
    M, K = x.shape
    g = x.view(M, K // 128, 128)
    s = torch.clamp(g.abs().amax(dim=2), min=Q_EPS) / QMAX
    if ue8m0:
        s = _pow2_ceil(s)
    return (g / s.unsqueeze(2)).to(torch.float8_e4m3fn).view(M, K), s


def _rows_value(codes, s):
    """The values of codes with one scale per 128 columns (s in [M, K/128])."""
    M, K = codes.shape
    return (codes.float().view(M, K // 128, 128) * s.unsqueeze(2)).view(M, K)


def _laid_out(s, layout):
    return s if layout == "row" else s.t().contiguous()


_GELU_A, _GELU_B = math.sqrt(2.0 / math.pi), 0.044715


def _act_and_slope(g, act):
    if act == "silu":
        p = 1 / (1 + torch.exp(-g))
        return g * p, p * (1 + g * (1 - p))
    t = _GELU_A * (g + _GELU_B * g * g * g)
    p = 1 / (1 + torch.exp(-2 * t))              # 0.5 (1 + tanh t) = 1 / (1 + exp(-2t))
    return g * p, p + g * p * (1 - p) * 2 * _GELU_A * (1 + 3 * _GELU_B * g * g)


# ------------------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32)


def _dtype(name):
    return {"bf16": torch.bfloat16, "fp32": torch.float32}[name]


def _codes_buffer(*shape):
    return torch.zeros(shape, device=DEV, dtype=torch.uint8).view(torch.float8_e4m3fn)


def _scales_buffer(M, G, layout):
    return torch.zeros((M, G) if layout == "row" else (G, M), device=DEV, dtype=torch.float32)


def _logits(g, c):
    """Router logits; some experts are more popular than others. With a mask a tenth of the
    experts is out of reach of a token, and of every 17th token all but three are."""
    T, E = c["T"], c["E"]
    x = _randn(g, T, E) * 1.5 + 0.5 * _randn(g, E)
    if c["mask"]:
        out = torch.rand((T, E), generator=g, device=DEV) < 0.1
        out[::17, 3:] = True
        out[:, 0] = False
        x[out] = -math.inf
    return x.to(_dtype(c["x"]))


def _expert_ids(g, c):
    """Distinct experts of each token, some more popular. With drop the experts are a quarter of
    all, the second one, and the ids are relative to it: the others lie outside [0, E)."""
    T, E, topk = c["T"], c["E"], c["topk"]
    every = 4 * E if c["drop"] else E
    score = _randn(g, T, every) + 0.5 * _randn(g, every)
    ids = torch.argsort(score, dim=1, descending=True)[:, :topk]
    return (ids - (E if c["drop"] else 0)).to(torch.int32).contiguous()


def _places(ids, E):
    """(first row of each expert and the count of all, place of each pair in expert order or -1)."""
    flat = ids.reshape(-1).long()
    bucket = torch.where((flat >= 0) & (flat < E), flat, E)
    order = torch.argsort(bucket, stable=True)
    at = torch.empty_like(order)
    at[order] = torch.arange(order.numel(), device=DEV)
    ends = torch.cumsum(torch.bincount(bucket, minlength=E + 1), 0)[:E]
    offsets = torch.cat([torch.zeros(1, device=DEV, dtype=ends.dtype), ends])
    return offsets.int(), torch.where(bucket < E, at, -1).int().view_as(ids)


def prepare(c, seed):
    g = _gen(seed)
    s = dict(c)
    if c["op"] in ("ckpt", "ckpt_bwd"):
        M, F, ue = c["M"], c["F"], c["scales"] == "ue8m0"
        pre = (_randn(g, M, 2 * F) * 1.5 * torch.exp(0.5 * _randn(g, M, 1))).bfloat16()
        if c["op"] == "ckpt":
            s["pre"] = pre
            s["kept"] = _codes_buffer(M, 2 * F)
            s["kept_scales"] = _scales_buffer(M, 2 * F // 128, "row")
            if c["h"] == "codes":
                s["q"] = _codes_buffer(M, F)
                s["q_scales"] = _scales_buffer(M, F // 128, c["layout"])
            else:
                s["h_out"] = torch.zeros((M, F), device=DEV, dtype=torch.bfloat16)
            return s
        s["kept"], s["kept_scales"] = _quant_groups(pre.float(), False)
        s["dh"] = (_randn(g, M, F) * torch.exp(_randn(g, M, 1))).mul_(1e-3).bfloat16()
        if c["out"] == "codes":
            s["q"] = _codes_buffer(M, 2 * F)
            s["q_scales"] = _scales_buffer(M, 2 * F // 128, c["layout"])
        else:
            s["dpre"] = torch.zeros((M, 2 * F), device=DEV, dtype=torch.bfloat16)
            if c["out"] == "bf16_h":
                s["h_out"] = torch.zeros((M, F), device=DEV, dtype=torch.bfloat16)
        return s
    T, E, topk = c["T"], c["E"], c["topk"]
    P = T * topk
    if c["op"] in ("route", "route_bwd"):
        s["logits"] = _logits(g, c)
        s["weight_scale"] = 2.5 if c["score"] == "sigmoid" else 1.0
        if c["op"] == "route":
            s["bias_values"] = 0.1 * _randn(g, E) if c["bias"] else None
            s["ids"] = torch.empty((T, topk), device=DEV, dtype=torch.int32)
            s["w"] = torch.empty((T, topk), device=DEV, dtype=torch.float32)
        else:
            key = s["logits"].float()
            ids = torch.sort(key, dim=1, descending=True, stable=True).indices[:, :topk]
            s["ids"] = torch.where(torch.isinf(key.gather(1, ids)), -1, ids).int().contiguous()
            s["d_w"] = _randn(g, T, topk) * 1e-2
            s["d_logits"] = torch.empty_like(s["logits"])
        return s
    K, ue = c["K"], c.get("scales") == "ue8m0"
    s["ids"] = _expert_ids(g, c)
    if c["op"] == "dispatch":
        x = _randn(g, T, K) * torch.exp(0.5 * _randn(g, T, 1))
        s["x"] = x.bfloat16()
        if c["inp"] == "codes":
            s["x"], xs = _quant_groups(s["x"].float(), ue)
            s["x_scales"] = _laid_out(xs, c["layout"])
        s["offsets"] = torch.zeros(E + 1, device=DEV, dtype=torch.int32)
        s["sorted"] = torch.zeros(P, device=DEV, dtype=torch.int32)
        s["pair_rows"] = torch.zeros((T, topk), device=DEV, dtype=torch.int32)
        if c["out"] == "codes":
            s["q"] = _codes_buffer(P, K)
            s["q_scales"] = _scales_buffer(P, K // 128, c["layout"])
        else:
            s["rows_out"] = torch.zeros((P, K), device=DEV, dtype=torch.bfloat16)
        return s
    _, pair_rows = _places(s["ids"], E)
    live = pair_rows.reshape(-1) >= 0
    pairs = torch.arange(P, device=DEV)
    s["pair_rows"] = pair_rows if c["order"] == "expert" else None
    w = torch.rand((T, topk), generator=g, device=DEV) + 0.05
    s["w"] = w / w.sum(dim=1, keepdim=True) * 2.5
    rows = _randn(g, P, K) * torch.exp(0.5 * _randn(g, P, 1))
    if c["op"] == "combine_bwd":
        # an expert's output and the gradient that reaches it have something in common
        d = _randn(g, T, K)
        of = d.repeat_interleave(topk, dim=0)
        if c["order"] == "expert":
            rows[pair_rows.reshape(-1)[live].long()] += 0.25 * of[live]
        else:
            rows += 0.25 * of
    # rows that no expert wrote hold anything
    used = torch.zeros(P, device=DEV, dtype=torch.bool)
    used[torch.where(live, pair_rows.reshape(-1).long() if c["order"] == "expert" else pairs,
                     0)[live]] = True
    if c["op"] == "combine":
        rows[~used] = math.nan
        s["rows_in"] = rows.to(_dtype(c["rows"]))
        s["w"] = s["w"] if c["weights"] else None
        ot = _dtype(c["out"])
        s["base_in"] = _randn(g, T, K).to(ot) if c["base"] else None
        s["out_rows"] = torch.empty((T, K), device=DEV, dtype=ot)
        if c["ckpt"]:
            s["kept"] = _codes_buffer(P, K)
            s["kept_scales"] = _scales_buffer(P, K // 128, "row")
        return s
    if c["rows"] == "codes":
        s["rows_in"], s["rows_scales"] = _quant_groups(rows, False)
        s["rows_scales"][~used] = math.nan
    else:
        rows[~used] = math.nan
        s["rows_in"], s["rows_scales"] = rows.bfloat16(), None
    s["d_out"] = (d * 1e-2 * torch.exp(_randn(g, T, 1))).to(_dtype(c["dout"]))
    s["d_w"] = torch.empty((T, topk), device=DEV, dtype=torch.float32)
    if c["out"] == "codes":
        s["q"] = _codes_buffer(P, K)
        s["q_scales"] = _scales_buffer(P, K // 128, c["layout"])
    else:
        s["d_rows"] = torch.zeros((P, K), device=DEV, dtype=torch.bfloat16)
    return s


# ------------------------------------------------------------------------- plain forms

def _plain_route(s):
    x, topk, E, T = s["logits"].float(), s["topk"], s["E"], s["T"]
    x64 = x.double()              # keys of neighbouring experts lie next to each other
    if s["score"] == "softmax":
        e = torch.exp(x64 - x64.amax(dim=1, keepdim=True))
        scores = e / e.sum(dim=1, keepdim=True)
    else:
        scores = 1 / (1 + torch.exp(-x64))
    key = x64
    if s["bias"] or s["groups"] > 1:
        key = scores + (s["bias_values"].double() if s["bias"] else 0.0)
        key = torch.where(torch.isinf(x64), -math.inf, key)
    if s["groups"] > 1:
        per = key.view(T, s["groups"], E // s["groups"])
        two = torch.sort(per, dim=2, descending=True).values[:, :, :2]
        total = torch.where(torch.isinf(two), 0.0, two).sum(dim=2)
        total = torch.where(torch.isinf(two[:, :, 0]), -math.inf, total)
        best = torch.sort(total, dim=1, descending=True, stable=True).indices[:, :s["topk_groups"]]
        kept = torch.zeros_like(total, dtype=torch.bool).scatter_(1, best, True)
        key = torch.where(kept.unsqueeze(2), per, -math.inf).reshape(T, E)
    order = torch.sort(key, dim=1, descending=True, stable=True)
    ids, taken = order.indices[:, :topk], ~torch.isinf(order.values[:, :topk])
    w = torch.where(taken, scores.gather(1, ids), 0.0)
    if s["renorm"]:
        w = w / (w.sum(dim=1, keepdim=True) + RENORM_EPS)
    return {"ids": torch.where(taken, ids, -1).int(), "weights": (w * s["weight_scale"]).float()}


def _plain_route_bwd(s):
    x, g = s["logits"].double(), s["d_w"].double()     # the renormed gradient is a small difference
    if s["score"] == "softmax":
        e = torch.exp(x - x.amax(dim=1, keepdim=True))
        p = e / e.sum(dim=1, keepdim=True)
    else:
        p = 1 / (1 + torch.exp(-x))
    taken = s["ids"] >= 0
    ids = s["ids"].long().clamp(min=0)
    sj = torch.where(taken, p.gather(1, ids), 0.0)
    if s["renorm"]:
        D = sj.sum(dim=1, keepdim=True) + RENORM_EPS
        g = (g - (g * sj).sum(dim=1, keepdim=True) / D) / D
    ds = torch.where(taken, g * s["weight_scale"], 0.0)
    d = torch.zeros_like(p).scatter_add_(1, ids, ds)
    if s["score"] == "softmax":
        d = p * (d - (ds * sj).sum(dim=1, keepdim=True))
    else:
        d = d * p * (1 - p)
    return {"d_logits": d.to(s["logits"].dtype)}


def _plain_dispatch(s):
    offsets, pair_rows = _places(s["ids"], s["E"])
    flat = pair_rows.reshape(-1).long()
    pairs = torch.nonzero(flat >= 0).reshape(-1)
    to, frm = flat[pairs], pairs // s["topk"]
    out = {"offsets": offsets, "pair_rows": pair_rows}
    if s["out"] == "bf16":
        out["rows"] = torch.zeros_like(s["rows_out"])
        out["rows"][to] = s["x"][frm]
        return out
    if s["inp"] == "codes":
        q, qs = s["x"], s["x_scales"] if s["layout"] == "row" else s["x_scales"].t()
    else:
        q, qs = _quant_groups(s["x"].float(), s["scales"] == "ue8m0")
    rows = torch.zeros(s["q"].shape, device=DEV, dtype=torch.uint8)
    rows[to] = q.view(torch.uint8)[frm]
    scales = torch.zeros((s["q"].shape[0], qs.shape[1]), device=DEV)
    scales[to] = qs[frm]
    out.update(q=rows.view(torch.float8_e4m3fn), scales=_laid_out(scales, s["layout"]))
    return out


def _pair_places(s):
    """Rows of the pairs [T, topk] and which of them exist."""
    if s["order"] == "expert":
        r = s["pair_rows"].long()
        return r.clamp(min=0), r >= 0
    r = torch.arange(s["T"] * s["topk"], device=DEV).view(s["T"], s["topk"])
    return r, (s["ids"] >= 0) & (s["ids"] < s["E"])


def _plain_combine(s):
    at, live = _pair_places(s)
    rows = s["rows_in"][at].float()
    if s["w"] is not None:
        rows = rows * s["w"].unsqueeze(2)
    y = torch.where(live.unsqueeze(2), rows, 0.0).sum(dim=1)
    if s["base_in"] is not None:
        y = s["base_in"].float() + y
    out = {"out": y.to(s["out_rows"].dtype)}
    if s["ckpt"]:
        q, qs = _quant_groups(s["rows_in"].float(), False)
        used = torch.zeros(q.shape[0], device=DEV, dtype=torch.bool)
        used[at[live]] = True
        out["kept"] = torch.where(used.unsqueeze(1), q.view(torch.uint8), 0).view(torch.float8_e4m3fn)
        out["kept_scales"] = torch.where(used.unsqueeze(1), qs, 0.0)
    return out


def _plain_combine_bwd(s):
    at, live = _pair_places(s)
    rows = s["rows_in"].float() if s["rows"] == "bf16" else _rows_value(s["rows_in"], s["rows_scales"])
    d = s["d_out"].float()
    dw = (rows[at] * d.unsqueeze(1)).sum(dim=2)
    out = {"d_weights": torch.where(live, dw, 0.0)}
    dr = torch.zeros((rows.shape[0], rows.shape[1]), device=DEV)
    dr[at[live]] = (s["w"].unsqueeze(2) * d.unsqueeze(1))[live]
    if s["out"] == "bf16":
        out["d_rows"] = dr.bfloat16()
        return out
    q, qs = _quant_groups(dr, s["scales"] == "ue8m0")
    used = torch.zeros(rows.shape[0], device=DEV, dtype=torch.bool)
    used[at[live]] = True
    out.update(q=q, scales=_laid_out(torch.where(used.unsqueeze(1), qs, 0.0), s["layout"]))
    return out


def _plain_ckpt(s):
    F, pre = s["F"], s["pre"].float()
    h = _act_and_slope(pre[:, :F], s["act"])[0] * pre[:, F:]
    q, qs = _quant_groups(pre, False)
    out = {"kept": q, "kept_scales": qs}
    if s["h"] == "bf16":
        out["h"] = h.bfloat16()
    else:
        q, qs = _quant_groups(h, s["scales"] == "ue8m0")
        out.update(q=q, scales=_laid_out(qs, s["layout"]))
    return out


def _plain_ckpt_bwd(s):
    F, dh = s["F"], s["dh"].float()
    pre = _rows_value(s["kept"], s["kept_scales"])
    g, u = pre[:, :F], pre[:, F:]
    a, slope = _act_and_slope(g, s["act"])
    dpre = torch.cat([dh * u * slope, dh * a], dim=1)
    if s["out"] == "codes":
        q, qs = _quant_groups(dpre, s["scales"] == "ue8m0")
        return {"q": q, "scales": _laid_out(qs, s["layout"])}
    out = {"dpre": dpre.bfloat16()}
    if s["out"] == "bf16_h":
        out["h"] = (a * u).bfloat16()
    return out


# ----------------------------------------------------------------------------- library

def _score_kind(s, bfq):
    return bfq.BFQ_SCORE_SOFTMAX if s["score"] == "softmax" else bfq.BFQ_SCORE_SIGMOID


def _scale_form(s, bfq):
    return dict(layout=bfq.BFQ_SCALES_ROW_MAJOR if s["layout"] == "row" else bfq.BFQ_SCALES_COL_MAJOR,
                scale_fmt=bfq.BFQ_SCALE_UE8M0 if s["scales"] == "ue8m0" else bfq.BFQ_SCALE_FP32)


def _own_route(s):
    from block_scaled_w8a8_amd import bfq
    bfq.bfq_moe_route(s["logits"], s["ids"], s["w"], bias=s["bias_values"],
                      score=_score_kind(s, bfq), n_groups=s["groups"],
                      topk_groups=s["topk_groups"], renorm=s["renorm"],
                      weight_scale=s["weight_scale"])
    return {"ids": s["ids"], "weights": s["w"]}


def _own_route_bwd(s):
    from block_scaled_w8a8_amd import bfq
    bfq.bfq_moe_route_backward(s["logits"], s["ids"], s["d_w"], s["d_logits"],
                               score=_score_kind(s, bfq), renorm=s["renorm"],
                               weight_scale=s["weight_scale"])
    return {"d_logits": s["d_logits"]}


def _own_dispatch(s):
    from block_scaled_w8a8_amd import bfq
    if "ws" not in s:                    # a workspace that the program keeps
        n = bfq.bfq_moe_sort_workspace_bytes(s["T"], s["topk"], s["E"])
        s["ws"] = torch.empty(n, device=DEV, dtype=torch.uint8) if n else None
    bfq.bfq_moe_sort(s["ids"], s["E"], s["offsets"], s["sorted"], s["pair_rows"],
                     workspace=s["ws"])
    out = {"offsets": s["offsets"], "pair_rows": s["pair_rows"]}
    if s["out"] == "bf16":
        bfq.bfq_moe_dispatch(s["x"], s["pair_rows"], rows=s["rows_out"])
        out["rows"] = s["rows_out"]
        return out
    form = _scale_form(s, bfq)
    if s["inp"] == "codes":
        form.update(x_scales=s["x_scales"], x_layout=form["layout"])
    bfq.bfq_moe_dispatch(s["x"], s["pair_rows"], q=s["q"], scales=s["q_scales"], **form)
    out.update(q=s["q"], scales=s["q_scales"])
    return out


def _own_places(s):
    """The arguments that say where a pair's row is."""
    if s["order"] == "expert":
        return dict(pair_rows=s["pair_rows"])
    return dict(topk_ids=s["ids"], E=s["E"])


def _own_combine(s):
    from block_scaled_w8a8_amd import bfq
    kept = dict(ckpt=s["kept"], ckpt_scales=s["kept_scales"]) if s["ckpt"] else {}
    bfq.bfq_moe_combine(s["rows_in"], s["out_rows"], s["topk"], weights=s["w"],
                        base=s["base_in"], **_own_places(s), **kept)
    out = {"out": s["out_rows"]}
    if s["ckpt"]:
        out.update(kept=s["kept"], kept_scales=s["kept_scales"])
    return out


def _own_combine_bwd(s):
    from block_scaled_w8a8_amd import bfq
    out = {"d_weights": s["d_w"]}
    if s["out"] == "bf16":
        form = dict(d_rows=s["d_rows"])
        out["d_rows"] = s["d_rows"]
    else:
        form = dict(q=s["q"], scales=s["q_scales"], **_scale_form(s, bfq))
        out.update(q=s["q"], scales=s["q_scales"])
    bfq.bfq_moe_combine_backward(s["d_out"], s["topk"], weights=s["w"], rows=s["rows_in"],
                                 rows_scales=s["rows_scales"], d_weights=s["d_w"],
                                 **_own_places(s), **form)
    return out


def _own_ckpt(s):
    from block_scaled_w8a8_amd import bfq
    act = bfq.BFQ_ACT_SILU if s["act"] == "silu" else bfq.BFQ_ACT_GELU_TANH
    out = {"kept": s["kept"], "kept_scales": s["kept_scales"]}
    if s["h"] == "bf16":
        form = dict(h=s["h_out"])
        out["h"] = s["h_out"]
    else:
        form = dict(q=s["q"], scales=s["q_scales"], **_scale_form(s, bfq))
        out.update(q=s["q"], scales=s["q_scales"])
    bfq.bfq_gated_checkpoint(s["pre"], act=act, ckpt=s["kept"], ckpt_scales=s["kept_scales"], **form)
    return out


def _own_ckpt_bwd(s):
    from block_scaled_w8a8_amd import bfq
    act = bfq.BFQ_ACT_SILU if s["act"] == "silu" else bfq.BFQ_ACT_GELU_TANH
    if s["out"] == "codes":
        form = dict(q=s["q"], scales=s["q_scales"], **_scale_form(s, bfq))
        out = {"q": s["q"], "scales": s["q_scales"]}
    else:
        form = dict(dpre=s["dpre"])
        out = {"dpre": s["dpre"]}
        if s["out"] == "bf16_h":
            form["h"] = out["h"] = s["h_out"]
    bfq.bfq_gated_checkpoint_backward(s["kept"], s["kept_scales"], s["dh"], act=act, **form)
    return out


def run(s):
    if own:
        return {"route": _own_route, "route_bwd": _own_route_bwd, "dispatch": _own_dispatch,
                "combine": _own_combine, "combine_bwd": _own_combine_bwd, "ckpt": _own_ckpt,
                "ckpt_bwd": _own_ckpt_bwd}[s["op"]](s)
    return {"route": _plain_route, "route_bwd": _plain_route_bwd, "dispatch": _plain_dispatch,
            "combine": _plain_combine, "combine_bwd": _plain_combine_bwd, "ckpt": _plain_ckpt,
            "ckpt_bwd": _plain_ckpt_bwd}[s["op"]](s)


# ------------------------------------------------------------------------- in 64 bits

def _exact_values(codes, s):
    return codes.double() * s.double().repeat_interleave(128, dim=1)


def _exact_codes(x, ue):
    """The e4m3fn values (as 64-bit numbers) that x stands for after group quantization."""
    M, K = x.shape
    groups = x.reshape(M * K // 128, 128)
    s = groups.abs().max(dim=1).values.clamp(min=Q_EPS) / QMAX
    if ue:
        s = 2.0 ** torch.ceil(torch.log2(s))
    v = groups / s[:, None]
    # round half to even on the grid of three mantissa bits (2^-9 steps below 2^-6)
    step = 2.0 ** (torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
    v = (torch.round(v / step) * step).clamp(-QMAX, QMAX)
    return v.reshape(M, K), s.reshape(M, K // 128)


def _exact_act(g, act):
    """The activation and its slope."""
    if act == "silu":
        p = torch.sigmoid(g)
        return g * p, p + g * p * (1 - p)
    c = math.sqrt(2.0 / math.pi)
    th = torch.tanh(c * (g + 0.044715 * g ** 3))
    return 0.5 * g * (1 + th), 0.5 * (1 + th) + 0.5 * g * (1 - th ** 2) * c * (1 + 3 * 0.044715 * g ** 2)


def _exact_rows(s):
    """One row index a pair, -1 where it has none."""
    if s["order"] == "expert":
        return s["pair_rows"].long()
    at = torch.arange(s["ids"].numel(), device=DEV).view_as(s["ids"])
    return torch.where((s["ids"] < 0) | (s["ids"] >= s["E"]), -1, at)


def _exact_scales(v, layout):
    return v if layout == "row" else v.t().contiguous()


def exact(c, seed):
    s = prepare(c, seed)
    if c["op"] == "ckpt":
        pre = s["pre"].double()
        g, u = pre.split(c["F"], dim=1)
        h = _exact_act(g, c["act"])[0] * u
        out = dict(zip(("kept", "kept_scales"), _exact_codes(pre, False)))
        if c["h"] == "bf16":
            out["h"] = h
        else:
            out["q"], sc = _exact_codes(h, c["scales"] == "ue8m0")
            out["scales"] = _exact_scales(sc, c["layout"])
        return out
    if c["op"] == "ckpt_bwd":
        g, u = _exact_values(s["kept"], s["kept_scales"]).split(c["F"], dim=1)
        a, slope = _exact_act(g, c["act"])
        dh = s["dh"].double()
        d = torch.cat([dh * u * slope, dh * a], dim=1)
        if c["out"] == "codes":
            q, sc = _exact_codes(d, c["scales"] == "ue8m0")
            return {"q": q, "scales": _exact_scales(sc, c["layout"])}
        return {"dpre": d, "h": a * u} if c["out"] == "bf16_h" else {"dpre": d}
    if c["op"] in ("route", "route_bwd"):
        x = s["logits"].double()
        score = torch.softmax(x, dim=1) if c["score"] == "softmax" else torch.sigmoid(x)
        if c["op"] == "route":
            # the ids are whole numbers; the weights follow from them
            ids = _plain_route(s)["ids"].long()
        else:
            ids = s["ids"].long()
        chosen = torch.zeros_like(score).scatter_add_(1, ids.clamp(min=0), (ids >= 0).double())
        picked = score.gather(1, ids.clamp(min=0)) * (ids >= 0)
        total = (score * chosen).sum(dim=1, keepdim=True) + RENORM_EPS
        if c["op"] == "route":
            if c["renorm"]:
                picked = picked / total
            return {"ids": None, "weights": picked * s["weight_scale"]}
        x = x.clone().requires_grad_()
        with torch.enable_grad():
            score = torch.softmax(x, dim=1) if c["score"] == "softmax" else torch.sigmoid(x)
            picked = score.gather(1, ids.clamp(min=0)) * (ids >= 0)
            if c["renorm"]:
                picked = picked / (picked.sum(dim=1, keepdim=True) + RENORM_EPS)
            (picked * s["d_w"].double()).sum().mul(s["weight_scale"]).backward()
        return {"d_logits": x.grad}
    if c["op"] == "dispatch":
        out = {"offsets": None, "pair_rows": None}
        rows = _places(s["ids"], c["E"])[1].long().reshape(-1)
        pairs = (rows >= 0).nonzero()[:, 0]

        def spread(v):
            r = torch.zeros((rows.numel(), v.shape[1]), device=DEV, dtype=torch.float64)
            return r.index_copy_(0, rows[pairs], v.double()[pairs // c["topk"]])

        if c["out"] == "bf16":
            out["rows"] = spread(s["x"])
            return out
        if c["inp"] == "codes":
            q, sc = s["x"], s["x_scales"] if c["layout"] == "row" else s["x_scales"].t()
        else:
            q, sc = _exact_codes(s["x"].double(), c["scales"] == "ue8m0")
        out["q"], out["scales"] = spread(q), _exact_scales(spread(sc), c["layout"])
        return out
    at = _exact_rows(s)
    if c["op"] == "combine":
        y = torch.zeros((c["T"], c["K"]), device=DEV, dtype=torch.float64)
        if c["base"]:
            y += s["base_in"].double()
        for j in range(c["topk"]):
            t = (at[:, j] >= 0).nonzero()[:, 0]
            r = s["rows_in"][at[t, j]].double()
            y[t] += r * s["w"][t, j].double()[:, None] if c["weights"] else r
        out = {"out": y}
        if c["ckpt"]:
            r = at[at >= 0]
            q, sc = _exact_codes(s["rows_in"][r].double(), False)
            out["kept"] = torch.zeros(s["kept"].shape, device=DEV, dtype=torch.float64)
            out["kept"][r] = q
            out["kept_scales"] = torch.zeros(s["kept_scales"].shape, device=DEV, dtype=torch.float64)
            out["kept_scales"][r] = sc
        return out
    P = c["T"] * c["topk"]
    d = s["d_out"].double()
    dw = torch.zeros((c["T"], c["topk"]), device=DEV, dtype=torch.float64)
    dr = torch.zeros((P, c["K"]), device=DEV, dtype=torch.float64)
    for j in range(c["topk"]):
        t = (at[:, j] >= 0).nonzero()[:, 0]
        r = at[t, j]
        rows = s["rows_in"][r].double() if c["rows"] == "bf16" else \
            _exact_values(s["rows_in"][r], s["rows_scales"][r])
        dw[t, j] = (rows * d[t]).sum(dim=1)
        dr[r] = d[t] * s["w"][t, j].double()[:, None]
    out = {"d_weights": dw}
    if c["out"] == "bf16":
        out["d_rows"] = dr
        return out
    q, sc = _exact_codes(dr, c["scales"] == "ue8m0")
    here = torch.zeros(P, device=DEV, dtype=torch.bool)
    here[at[at >= 0]] = True
    out["q"], out["scales"] = q, _exact_scales(sc * here[:, None], c["layout"])
    return out

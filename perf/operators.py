"""Measured cases of the feed-forward operators around the block-scaled W8A8 linear.

Four operators: the gated projection pair of a feed-forward block with its activation and
product (``gated``), the backward pass of that block down to its input's gradient
(``gated_bwd``), the norms before and after a block fused with the block's gate, residual scale
and the token quantization (``norm``), and the backward pass of those norms (``norm_bwd``).

``run`` computes each in plain torch where ``own`` is false, and calls the library where it is
true. ``exact`` gives the same outputs from the definitions in 64 bits.

Shapes are the projection shapes of the benchmark: K = 7168 features, F = 18432 feed-forward
columns of a dense layer, 2048 of a routed expert, 2304 of one GPU's eighth of a dense layer.
"""
import math

import torch

own = False

DEV = "cuda"
QMAX = 448.0           # largest finite e4m3fn value
Q_EPS = 1e-10          # floor of a group's largest magnitude
NORM_EPS = 1e-6


# ------------------------------------------------------------------------------ cases

def listed():
    return [
        # one token through the wide pair of projections: the decode step, a stream of weights
        dict(name="gated_decode_1", op="gated", M=1, K=7168, F=18432, act="silu", scales="fp32",
             layout="packed", out="bf16", keep=False),
        # a small decode batch on one GPU's eighth of the layer: launch and latency
        dict(name="gated_shard_16", op="gated", M=16, K=7168, F=2304, act="silu", scales="fp32",
             layout="row", out="fp16", keep=False),
        # prompt processing that keeps the pre-activations for a backward pass; the largest
        dict(name="gated_prefill_4096", op="gated", M=4096, K=7168, F=18432, act="silu",
             scales="fp32", layout="packed", out="bf16", keep=True),
        # a whole feed-forward block at an odd batch: codes out, then the down projection
        dict(name="ffn_expert_333", op="gated", M=333, K=7168, F=2048, act="gelu_tanh",
             scales="ue8m0", layout="packed", out="down", keep=False),
        # a training step's gradient at the pre-activations, 16 bits, and the product again
        dict(name="gated_bwd_elementwise", op="gated_bwd", M=4096, K=0, F=18432, act="silu",
             scales="fp32", layout="packed", out="dpre"),
        # the gradient at the block's input, through quantized gradients and weights
        dict(name="gated_bwd_input_1024", op="gated_bwd", M=1024, K=7168, F=18432, act="silu",
             scales="fp32", layout="packed", out="dx"),
        # the same for a few tokens of a small layer
        dict(name="gated_bwd_input_24", op="gated_bwd", M=24, K=1536, F=1536, act="gelu_tanh",
             scales="ue8m0", layout="row", out="dx"),
        # one token: residual add, the next block's norm, its input codes
        dict(name="norm_decode_1", op="norm", M=1, K=7168, post=False, gate="none", res="bf16",
             out="codes", scales="fp32", layout="row"),
        # a prompt: norm after the block, channel gate, residual scale, norm before, codes
        dict(name="norm_prefill_4096", op="norm", M=4096, K=7168, post=True, gate="channel",
             res="bf16", out="codes", scales="fp32", layout="col"),
        # a residual stream in 32 bits, a full gate, a row that is no multiple of 128, 16 bits out
        dict(name="norm_odd_1003", op="norm", M=1003, K=1544, post=True, gate="full", res="fp32",
             out="bf16", scales="fp32", layout="row"),
        # the norms' gradients of a training batch
        dict(name="norm_bwd_4096", op="norm_bwd", M=4096, K=7168, post=True, gate="channel",
             res="bf16"),
        # and of a small odd one with a gate value per token
        dict(name="norm_bwd_257", op="norm_bwd", M=257, K=1544, post=True, gate="token",
             res="fp32"),
    ]


def draw(rng):
    def log(lo, hi, step=1):
        return max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step)) * step)

    op = rng.choice(["gated", "gated", "gated_bwd", "norm", "norm_bwd"])
    act = rng.choice(["silu", "gelu_tanh"])
    scales = rng.choice(["fp32", "ue8m0"])
    layout = rng.choice(["packed", "row"])
    M = log(1, 4096)
    if op == "gated":
        out = rng.choice(["bf16", "fp16", "down"])
        # a block with its down projection has half as many operations again
        return dict(op=op, M=M, K=log(512, 7168, 128),
                    F=log(512, 12288 if out == "down" else 18432, 128), act=act, scales=scales,
                    layout=layout, out=out, keep=rng.random() < 0.3)
    if op == "gated_bwd":
        out = rng.choice(["dpre", "dx", "dx"])
        return dict(op=op, M=M, K=0 if out == "dpre" else log(512, 7168, 128),
                    F=log(512, 18432, 128), act=act, scales=scales, layout=layout, out=out)
    post = rng.random() < 0.6
    gate = rng.choice(["none", "channel", "token", "full"])
    res = rng.choice(["bf16", "fp32"])
    if op == "norm":
        out = rng.choice(["codes", "codes", "bf16"])
        K = log(512, 8192, 128) if out == "codes" else log(256, 8192, 8)
        return dict(op=op, M=M, K=K, post=post, gate=gate, res=res, out=out, scales="fp32",
                    layout=rng.choice(["row", "col"]))
    return dict(op=op, M=M, K=log(256, 8192, 8), post=post, gate=gate, res=res)


def work(c):
    M, K = c["M"], c["K"]
    if c["op"] == "gated":
        F = c["F"]
        b = M * K + 4 * M * (K // 128) + 2 * F * K + 4 * (2 * F // 128) * (K // 128)
        f = 4.0 * M * F * K + 8.0 * M * F
        if c["out"] == "down":       # the down projection's weights and the block's output
            b += F * K + 4 * (F // 128) * (K // 128) + 2 * M * K
            f += 2.0 * M * F * K
        else:
            b += 2 * M * F
        b += 4 * M * F if c["keep"] else 0
        return {"bytes": float(b), "flops": f}
    if c["op"] == "gated_bwd":
        F = c["F"]
        b, f = 6 * M * F, 16.0 * M * F
        if c["out"] == "dpre":
            b += 6 * M * F
        else:
            b += 2 * F * K + 4 * (2 * F // 128) * (K // 128) + 2 * M * K
            f += 4.0 * M * F * K
        return {"bytes": float(b), "flops": f}
    r = 2 if c["res"] == "bf16" else 4
    gate = {"none": 0, "channel": 2 * K, "token": 2 * M, "full": 2 * M * K}[c["gate"]]
    vecs = 2 * K * (2 if c["post"] else 1)
    if c["op"] == "norm":
        b = M * K * (2 + 2 * r) + gate + vecs
        b += M * K + 4 * M * (K // 128) if c["out"] == "codes" else 2 * M * K
        return {"bytes": float(b), "flops": 12.0 * M * K}
    # y, the stored sum, both gradients in; both gradients out; the vectors' gradients
    b = M * K * (2 + r + 2 + r + 2 + r) + gate + vecs + 4 * K * (2 if c["post"] else 1)
    b += {"none": 0, "channel": 4 * K, "token": 4 * M, "full": 2 * M * K}[c["gate"]]
    return {"bytes": float(b), "flops": 30.0 * M * K}


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


def _quant_blocks(w, ue8m0):
    """fp32 [N, K] -> e4m3fn codes and one scale per 128 x 128 block."""
    N, K = w.shape
    b = w.view(N // 128, 128, K // 128, 128)
    s = torch.clamp(b.abs().amax(dim=(1, 3)), min=Q_EPS) / QMAX
    if ue8m0:
        s = _pow2_ceil(s)
    return (b / s[:, None, :, None]).to(torch.float8_e4m3fn).view(N, K), s


def _packed(codes):
    """Row-major codes [N, K] in the order of 16-row fragments that the GEMMs stream: per 16
    rows and 128 columns, byte h*1024 + 16*(16*c + r) + b holds row r, column 64h + 16c + b."""
    N, K = codes.shape
    v = codes.view(torch.uint8).view(N // 16, 16, K // 128, 2, 4, 16)
    return v.permute(0, 2, 3, 4, 1, 5).contiguous().view(N, K)


def _rows_value(codes, s):
    """The values of codes with one scale per 128 columns (s in [M, K/128])."""
    M, K = codes.shape
    return (codes.float().view(M, K // 128, 128) * s.unsqueeze(2)).view(M, K)


def _blocks_value(codes, s):
    N, K = codes.shape
    return (codes.float().view(N // 128, 128, K // 128, 128) * s[:, None, :, None]).view(N, K)


_GELU_A, _GELU_B = math.sqrt(2.0 / math.pi), 0.044715


def _act(g, act):
    if act == "silu":
        return g / (1 + torch.exp(-g))
    t = _GELU_A * (g + _GELU_B * g * g * g)
    return g / (1 + torch.exp(-2 * t))           # 0.5 (1 + tanh t) = 1 / (1 + exp(-2t))


def _act_and_slope(g, act):
    if act == "silu":
        p = 1 / (1 + torch.exp(-g))
        return g * p, p * (1 + g * (1 - p))
    t = _GELU_A * (g + _GELU_B * g * g * g)
    p = 1 / (1 + torch.exp(-2 * t))
    return g * p, p + g * p * (1 - p) * 2 * _GELU_A * (1 + 3 * _GELU_B * g * g)


# ------------------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32)


def _activations(g, M, K):
    """N(0, 1) with 2 % outlier columns of 20 times the size."""
    x = _randn(g, M, K)
    cols = torch.randperm(K, generator=g, device=DEV)[: int(round(0.02 * K))]
    x[:, cols] *= 20.0
    return x


def _dtype(name):
    return {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}[name]


def prepare(c, seed):
    g = _gen(seed)
    M, K = c["M"], c["K"]
    s = dict(c)
    if c["op"] in ("gated", "gated_bwd"):
        F, ue = c["F"], c["scales"] == "ue8m0"
    if c["op"] == "gated":
        # activation codes as the token quantizer leaves them (column-major scales), weights
        # as the offline step leaves them
        a, sa = _quant_groups(_activations(g, M, K).bfloat16().float(), ue)
        w, sw = _quant_blocks(_randn(g, 2 * F, K) * 0.02, ue)
        s.update(a=a, sa=sa.t().contiguous(), w=w, sw=sw)
        s["w_own"] = _packed(w) if c["layout"] == "packed" else w.view(torch.uint8)
        if c["out"] == "down":
            wd, swd = _quant_blocks(_randn(g, K, F) * 0.02, ue)
            s.update(wd=wd, swd=swd)
            s["wd_own"] = _packed(wd) if c["layout"] == "packed" else wd.view(torch.uint8)
            s["h"] = torch.empty((M, F), device=DEV, dtype=torch.float8_e4m3fn)
            s["h_scales"] = torch.empty((F // 128, M), device=DEV, dtype=torch.float32)
        else:
            s["h"] = torch.empty((M, F), device=DEV, dtype=_dtype(c["out"]))
        s["pre"] = torch.empty((M, 2 * F), device=DEV, dtype=torch.bfloat16) if c["keep"] else None
    elif c["op"] == "gated_bwd":
        s["pre"] = (_randn(g, M, 2 * F) * 1.5).bfloat16()
        s["dh"] = (_randn(g, M, F) * torch.exp(_randn(g, M, 1))).mul_(1e-3).bfloat16()
        if c["out"] == "dx":
            # the transposed weights, laid out once: row k holds column k of the pair [2F, K]
            w, sw = _quant_blocks(_randn(g, K, 2 * F) * 0.02, ue)
            s.update(w=w, sw=sw)
            s["w_own"] = _packed(w) if c["layout"] == "packed" else w.view(torch.uint8)
            s["q"] = torch.empty((M, 2 * F), device=DEV, dtype=torch.float8_e4m3fn)
            s["q_scales"] = torch.empty((2 * F // 128, M), device=DEV, dtype=torch.float32)
        else:
            s["dpre"] = torch.empty((M, 2 * F), device=DEV, dtype=torch.bfloat16)
            s["h"] = torch.empty((M, F), device=DEV, dtype=torch.bfloat16)
    else:
        rt = _dtype(c["res"])
        s["y"] = (_randn(g, M, K) * 0.7).bfloat16()
        s["w_pre"] = (1 + 0.2 * _randn(g, K)).bfloat16()
        s["w_post"] = (1 + 0.2 * _randn(g, K)).bfloat16() if c["post"] else None
        shape = {"channel": (K,), "token": (M,), "full": (M, K)}.get(c["gate"])
        s["gate"] = (0.5 + 0.5 * _randn(g, *shape)).bfloat16() if shape else None
        s["gate_kind"], s["res_scale"] = c["gate"], 0.75
        s["r"] = _activations(g, M, K).to(rt)       # bwd: the stored sum
        if c["op"] == "norm":
            s["res_out"] = torch.empty((M, K), device=DEV, dtype=rt)
            if c["out"] == "codes":
                s["q"] = torch.empty((M, K), device=DEV, dtype=torch.float8_e4m3fn)
                sh = (M, K // 128) if c["layout"] == "row" else (K // 128, M)
                s["q_scales"] = torch.empty(sh, device=DEV, dtype=torch.float32)
            else:
                s["normed"] = torch.empty((M, K), device=DEV, dtype=torch.bfloat16)
        else:
            s["d_normed"] = (_randn(g, M, K) * 1e-2).bfloat16()
            s["d_res_out"] = (_randn(g, M, K) * 1e-2).to(rt)
            s["d_res"] = torch.empty((M, K), device=DEV, dtype=rt)
            s["d_y"] = torch.empty((M, K), device=DEV, dtype=torch.bfloat16)
            s["d_w_pre"] = torch.empty(K, device=DEV, dtype=torch.float32)
            s["d_w_post"] = torch.empty(K, device=DEV, dtype=torch.float32) if c["post"] else None
            s["d_gate"] = None
            if shape:
                gt = torch.bfloat16 if c["gate"] == "full" else torch.float32
                s["d_gate"] = torch.empty(shape, device=DEV, dtype=gt)
    return s


# ------------------------------------------------------------------------- plain forms

def _plain_gated(s):
    ue, F = s["scales"] == "ue8m0", s["F"]
    a = _rows_value(s["a"], s["sa"].t())
    pre = a @ _blocks_value(s["w"], s["sw"]).t()
    h = _act(pre[:, :F], s["act"]) * pre[:, F:]
    if s["out"] == "down":
        q, qs = _quant_groups(h, ue)
        out = {"y": (_rows_value(q, qs) @ _blocks_value(s["wd"], s["swd"]).t()).bfloat16()}
    else:
        out = {"h": h.to(_dtype(s["out"]))}
    if s["keep"]:
        out["pre"] = pre.bfloat16()
    return out


def _plain_gated_bwd(s):
    F, dh = s["F"], s["dh"].float()
    g, u = s["pre"][:, :F].float(), s["pre"][:, F:].float()
    a, slope = _act_and_slope(g, s["act"])
    dpre = torch.cat([dh * u * slope, dh * a], dim=1)
    if s["out"] == "dpre":
        return {"dpre": dpre.bfloat16(), "h": (a * u).bfloat16()}
    q, qs = _quant_groups(dpre, s["scales"] == "ue8m0")
    return {"dx": (_rows_value(q, qs) @ _blocks_value(s["w"], s["sw"]).t()).bfloat16()}


def _rms(x):
    return 1 / torch.sqrt((x * x).mean(dim=1, keepdim=True) + NORM_EPS)


def _gate_rows(s):
    """The gate as something that broadcasts over [M, K], in 32 bits."""
    if s["gate"] is None:
        return 1.0
    return s["gate"].float()[:, None] if s["gate_kind"] == "token" else s["gate"].float()


def _plain_norm(s):
    y = s["y"].float()
    z = y * _rms(y) * s["w_post"].float() if s["post"] else y
    r = s["r"].float() + s["res_scale"] * _gate_rows(s) * z
    n = r * _rms(r) * s["w_pre"].float()
    out = {"res": r.to(s["r"].dtype)}
    if s["out"] == "codes":
        q, qs = _quant_groups(n, False)
        out.update(q=q, scales=qs if s["layout"] == "row" else qs.t().contiguous())
    else:
        out["normed"] = n.bfloat16()
    return out


def _plain_norm_bwd(s):
    r, y, dn = s["r"].float(), s["y"].float(), s["d_normed"].float()
    ir = _rms(r)
    xr = r * ir
    t = dn * s["w_pre"].float()
    dr = s["d_res_out"].float() + ir * (t - xr * (t * xr).mean(dim=1, keepdim=True))
    out = {"d_res": dr.to(s["r"].dtype), "d_w_pre": (dn * xr).sum(dim=0)}
    gate = _gate_rows(s)
    if s["post"]:
        iy = _rms(y)
        xy, w = y * iy, s["w_post"].float()
        z = xy * w
        dz = s["res_scale"] * gate * dr
        out["d_w_post"] = (dz * xy).sum(dim=0)
        t = dz * w
        dy = iy * (t - xy * (t * xy).mean(dim=1, keepdim=True))
    else:
        z = y
        dy = s["res_scale"] * gate * dr
    out["d_y"] = dy.bfloat16()
    dg = s["res_scale"] * dr * z
    if s["gate_kind"] == "channel":
        out["d_gate"] = dg.sum(dim=0)
    elif s["gate_kind"] == "token":
        out["d_gate"] = dg.sum(dim=1)
    elif s["gate_kind"] == "full":
        out["d_gate"] = dg.bfloat16()
    return out


# ----------------------------------------------------------------------------- library

def _own_gated(s):
    from block_scaled_w8a8_amd import bfq
    sf = bfq.BFQ_SCALE_UE8M0 if s["scales"] == "ue8m0" else bfq.BFQ_SCALE_FP32
    wl = bfq.BFQ_W_PACKED16 if s["layout"] == "packed" else bfq.BFQ_W_ROW_MAJOR
    act = bfq.BFQ_ACT_SILU if s["act"] == "silu" else bfq.BFQ_ACT_GELU_TANH
    down = s["out"] == "down"
    if "ws" not in s:                    # a workspace that the program keeps
        n = bfq.bfq_gated_gemm_workspace_bytes(
            s["M"], s["F"], s["K"], w_layout=wl, scale_fmt=sf,
            out_dtype=bfq.BFQ_E4M3FN if down else bfq.BFQ_BF16)
        s["ws"] = torch.empty(n, device=DEV, dtype=torch.uint8) if n else None
    bfq.bfq_gated_gemm(s["a"], s["sa"], s["w_own"], s["sw"], s["h"], act=act,
                       a_layout=bfq.BFQ_SCALES_COL_MAJOR, w_layout=wl, scale_fmt=sf,
                       out_scales=s["h_scales"] if down else None,
                       out_layout=bfq.BFQ_SCALES_COL_MAJOR, preact=s["pre"], workspace=s["ws"])
    if down:
        out = {"y": bfq.block_gemm(s["h"], s["h_scales"], s["wd_own"], s["swd"],
                                   a_layout=bfq.BFQ_SCALES_COL_MAJOR, w_layout=wl, scale_fmt=sf)}
    else:
        out = {"h": s["h"]}
    if s["keep"]:
        out["pre"] = s["pre"]
    return out


def _own_gated_bwd(s):
    from block_scaled_w8a8_amd import bfq
    sf = bfq.BFQ_SCALE_UE8M0 if s["scales"] == "ue8m0" else bfq.BFQ_SCALE_FP32
    wl = bfq.BFQ_W_PACKED16 if s["layout"] == "packed" else bfq.BFQ_W_ROW_MAJOR
    act = bfq.BFQ_ACT_SILU if s["act"] == "silu" else bfq.BFQ_ACT_GELU_TANH
    if s["out"] == "dpre":
        bfq.bfq_gated_backward(s["pre"], s["dh"], act=act, dpre=s["dpre"], h=s["h"])
        return {"dpre": s["dpre"], "h": s["h"]}
    bfq.bfq_gated_backward(s["pre"], s["dh"], act=act, q=s["q"], scales=s["q_scales"],
                           layout=bfq.BFQ_SCALES_COL_MAJOR, scale_fmt=sf)
    return {"dx": bfq.block_gemm(s["q"], s["q_scales"], s["w_own"], s["sw"],
                                 a_layout=bfq.BFQ_SCALES_COL_MAJOR, w_layout=wl, scale_fmt=sf)}


def _own_kind(s, bfq):
    return {"none": bfq.BFQ_GATE_NONE, "channel": bfq.BFQ_GATE_CHANNEL,
            "token": bfq.BFQ_GATE_TOKEN, "full": bfq.BFQ_GATE_FULL}[s["gate_kind"]]


def _own_norm(s):
    from block_scaled_w8a8_amd import bfq
    out = {"res": s["res_out"]}
    if s["out"] == "codes":
        lay = bfq.BFQ_SCALES_ROW_MAJOR if s["layout"] == "row" else bfq.BFQ_SCALES_COL_MAJOR
        form = dict(q=s["q"], scales=s["q_scales"], layout=lay)
        out.update(q=s["q"], scales=s["q_scales"])
    else:
        form = dict(normed=s["normed"])
        out["normed"] = s["normed"]
    bfq.bfq_norm_residual(s["r"], y=s["y"], w_post=s["w_post"], gate=s["gate"],
                          gate_kind=_own_kind(s, bfq), res_scale=s["res_scale"],
                          w_pre=s["w_pre"], norm_eps=NORM_EPS, res_out=s["res_out"], **form)
    return out


def _own_norm_bwd(s):
    from block_scaled_w8a8_amd import bfq
    if "ws" not in s:
        n = bfq.bfq_norm_residual_backward_workspace_bytes(s["M"], s["K"])
        s["ws"] = torch.empty(n, device=DEV, dtype=torch.uint8) if n else None
    bfq.bfq_norm_residual_backward(
        s["r"], y=s["y"], w_post=s["w_post"], gate=s["gate"], gate_kind=_own_kind(s, bfq),
        res_scale=s["res_scale"], w_pre=s["w_pre"], norm_eps=NORM_EPS, d_normed=s["d_normed"],
        d_res_out=s["d_res_out"], d_res=s["d_res"], d_y=s["d_y"], d_w_pre=s["d_w_pre"],
        d_w_post=s["d_w_post"], d_gate=s["d_gate"], workspace=s["ws"])
    out = {"d_res": s["d_res"], "d_w_pre": s["d_w_pre"], "d_y": s["d_y"]}
    if s["post"]:
        out["d_w_post"] = s["d_w_post"]
    if s["gate"] is not None:
        out["d_gate"] = s["d_gate"]
    return out


def run(s):
    if own:
        return {"gated": _own_gated, "gated_bwd": _own_gated_bwd, "norm": _own_norm,
                "norm_bwd": _own_norm_bwd}[s["op"]](s)
    return {"gated": _plain_gated, "gated_bwd": _plain_gated_bwd, "norm": _plain_norm,
            "norm_bwd": _plain_norm_bwd}[s["op"]](s)


# ------------------------------------------------------------------------- in 64 bits

def _exact_values(codes, s, rows):
    """Codes times scales in 64 bits; one scale covers `rows` rows and 128 columns."""
    full = s.double().repeat_interleave(128, dim=1)
    if rows > 1:
        full = full.repeat_interleave(rows, dim=0)
    return codes.double() * full


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


def _exact_gate(s):
    if s["gate"] is None:
        return torch.ones((), device=DEV, dtype=torch.float64)
    g = s["gate"].double()
    return g.reshape(-1, 1) if s["gate_kind"] == "token" else g


def exact(c, seed):
    s = prepare(c, seed)
    if c["op"] == "gated":
        F, ue = c["F"], c["scales"] == "ue8m0"
        x = _exact_values(s["a"], s["sa"].t().contiguous(), 1)
        gate = torch.mm(x, _exact_values(s["w"][:F], s["sw"][: F // 128], 128).t())
        up = torch.mm(x, _exact_values(s["w"][F:], s["sw"][F // 128:], 128).t())
        h = _exact_act(gate, c["act"])[0] * up
        if c["out"] == "down":
            v, vs = _exact_codes(h, ue)
            out = {"y": torch.mm(v * vs.repeat_interleave(128, dim=1),
                                 _exact_values(s["wd"], s["swd"], 128).t())}
        else:
            out = {"h": h}
        if c["keep"]:
            out["pre"] = torch.cat([gate, up], dim=1)
        return out
    if c["op"] == "gated_bwd":
        F, dh = c["F"], s["dh"].double()
        g, u = s["pre"].double().split(F, dim=1)
        a, slope = _exact_act(g, c["act"])
        d = torch.cat([dh * u * slope, dh * a], dim=1)
        if c["out"] == "dpre":
            return {"dpre": d, "h": a * u}
        v, vs = _exact_codes(d, c["scales"] == "ue8m0")
        return {"dx": torch.mm(v * vs.repeat_interleave(128, dim=1),
                               _exact_values(s["w"], s["sw"], 128).t())}
    y, r, gate, alpha = s["y"].double(), s["r"].double(), _exact_gate(s), s["res_scale"]
    root = lambda x: torch.sqrt(x.square().mean(dim=1, keepdim=True) + NORM_EPS)  # noqa: E731
    z = y / root(y) * s["w_post"].double() if c["post"] else y
    if c["op"] == "norm":
        r = r + alpha * gate * z
        n = r / root(r) * s["w_pre"].double()
        out = {"res": r}
        if c["out"] == "codes":
            out["q"], sc = _exact_codes(n, False)
            out["scales"] = sc if c["layout"] == "row" else sc.t().contiguous()
        else:
            out["normed"] = n
        return out

    def norm_grad(x, w, d):
        """Gradients of x / root(x) * w at x and at w, for the gradient d of its output."""
        rt, K = root(x), x.shape[1]
        t = w * d
        return t / rt - x * (t * x).sum(dim=1, keepdim=True) / (K * rt ** 3), (d * x / rt).sum(dim=0)

    dr, dw = norm_grad(r, s["w_pre"].double(), s["d_normed"].double())
    dr = dr + s["d_res_out"].double()
    out = {"d_res": dr, "d_w_pre": dw}
    dz = alpha * gate * dr
    if c["post"]:
        out["d_y"], out["d_w_post"] = norm_grad(y, s["w_post"].double(), dz)
    else:
        out["d_y"] = dz.expand_as(y).contiguous()
    dg = alpha * dr * z
    if c["gate"] == "channel":
        out["d_gate"] = dg.sum(dim=0)
    elif c["gate"] == "token":
        out["d_gate"] = dg.sum(dim=1)
    elif c["gate"] == "full":
        out["d_gate"] = dg
    return out

"""GPU tests of the feed-forward operators: the gated product, its gradient, the weight transpose,
the norms around a block with gate and residual scale, and their gradients.

References are the formulas in 64 bits. Tolerances count roundings: u = 2^-24 is half a step of
fp32, H[t] half a step of an output type relative to the value.
  * Gated product: its two sums are the block GEMM's, so they are compared through it. For every
    compiled gated tile there is a block-GEMM tile that runs the same MFMA and scale steps in the
    same order; on the 2F-row weights that tile's fp32 output is the pair (g, u) bit for bit, and
    the reference act(g) * u is formed from it in 64 bits. What is left is the activation: the
    exponential, 1 + e, the reciprocal and two products, each within a step (2u), 16u in all with
    the capped argument's own roundings, plus the argument's relative error (at most 4u, none for
    SILU) times |z| in the exponential.
  * Norms: a row's sum of squares adds at most 64 terms in a thread, 6 in a wave and 16 across
    waves, each addition and product within u of a sum of positive terms: 90u, 45u on its root.
"""
import math

import numpy as np
import pytest
import torch

from block_scaled_w8a8_amd import synth

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U = 2.0 ** -24
H = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
TINY = {torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -149}


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _randn(seed, *shape):
    return torch.randn(shape, generator=_gen(seed), device=DEV, dtype=torch.float32)


def _within(got, ref, tol, what):
    got, ref = got.double(), ref.double()
    assert torch.equal(torch.isnan(got), torch.isnan(ref)), what
    bad = ((got - ref).abs() > tol) & ~torch.isnan(ref)
    if bool(bad.any()):
        i = tuple(int(x[0]) for x in torch.nonzero(bad, as_tuple=True))
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} outside; first at {i}: "
                             f"{float(got[i])} against {float(ref[i])}, "
                             f"tolerance {float(torch.as_tensor(tol).expand(got.shape)[i])}")


def _act(g, act):
    """act(g), its slope and the argument z of the sigmoid, in 64 bits."""
    if act == 0:
        p = torch.sigmoid(g)
        return g * p, p + g * p * (1 - p), g
    c = 2 * math.sqrt(2 / math.pi)
    z = c * (g + 0.044715 * g ** 3)
    p = torch.sigmoid(z)
    return g * p, p + g * p * (1 - p) * c * (1 + 3 * 0.044715 * g * g), z


# ---------------------------------------------------------------------- quantized outputs

def _check_codes(codes, scales, x, xtol, ue8m0, what, int8=False, group=128):
    """codes / scales [M, G] (fp32) of x, known to xtol per element (64-bit tensors)."""
    M, N = x.shape
    qmax = 127.0 if int8 else 448.0
    xg, tg = x.view(M, N // group, group), xtol.view(M, N // group, group)
    amax, i = xg.abs().max(dim=2)
    dt = tg.max(dim=2).values                       # how far the largest magnitude may be off
    s = scales.double()
    lo, hi = [(torch.clamp(a, min=1e-10) / qmax) for a in (amax - dt, amax + dt)]
    if ue8m0:
        assert torch.equal(torch.frexp(scales)[0], torch.full_like(scales, 0.5)), what
        lo, hi = (torch.exp2(torch.ceil(torch.log2(v * (1 + e)))) for v, e in ((lo, -U), (hi, U)))
        assert bool(((s >= lo) & (s <= hi)).all()), what
    else:
        _within(scales, (lo + hi) / 2, (hi - lo) / 2 + 2 * U * hi, what + " scales")
    v = xg / s.unsqueeze(2)
    got = (codes.view(torch.int8).double() if int8
           else codes.view(torch.float8_e4m3fn).double()).view_as(v)
    # half a step of the code: 2^-4 relative (int8: 1/2), 2^-10 where e4m3 is subnormal
    half = torch.full_like(v, 0.5) if int8 else torch.clamp(v.abs() * 2.0 ** -4, min=2.0 ** -10)
    _within(got, v, half * (1 + 4 * U) + tg / s.unsqueeze(2) + 4 * U * v.abs(), what + " codes")


def _unpack_scales(bfq, scales, layout, M, G):
    """Scales [M, G] fp32 from any layout; packed words also have their padding checked."""
    if layout == bfq.BFQ_SCALES_ROW_MAJOR:
        return scales[:M, :G]
    if layout == bfq.BFQ_SCALES_COL_MAJOR:
        return scales[:G, :M].t()
    b = scales.contiguous().view(torch.uint8).view(scales.shape[0], scales.shape[1], 4)
    m4 = (M + 3) // 4 * 4
    assert not bool(b[:, M:m4].any()), "padding rows of packed words"
    flat = b[:, :M].permute(1, 0, 2).reshape(M, -1)
    assert not bool(flat[:, G:].any()), "padding bytes of packed words"
    return torch.exp2(flat[:, :G].float() - 127)


# ------------------------------------------------------------------------- gated product

def _pair(bfq, M, F, K, seed, sfmt, wl):
    """Token codes (row-major scales) and the weight pair, quantized on the device."""
    x = synth.activations(M, K, seed=seed).to(DEV)
    w = _randn(seed + 1, 2 * F, K) * 0.02
    qa, sa = bfq.quant_tokens(x, scale_fmt=sfmt)
    qw, sw = bfq.quant_weight_blocks(w, scale_fmt=sfmt)
    return qa, sa, bfq.pack_weights(qw) if wl else qw, sw, qw


def _twin(bfq, t, wl):
    """The block-GEMM tile that forms the same sums in the same order as gated tile t."""
    d = {"variant": 0, "bm": 128, "bn": 128, "waves_m": 2, "waves_n": 2, "stages": 2, "group_m": 8,
         "sched": 3 if t.sched == 3 and t.variant == 0 else 0, "split_k": t.split_k}
    if t.variant == 1 and t.waves_m >= 4 and t.sched != 2:
        d.update(variant=1, bm=16, bn=16, waves_m=t.waves_m, waves_n=1, stages=4, sched=0, group_m=1)
    return bfq.bfq_tile.from_dict(d)


def _gu_interleaved(bfq, qa, sa, qw, sw, t, wl, sfmt):
    """The ring strips' sums: the waves of a workgroup take every waves_m-th K block of a part, each
    in ascending order; their sums are added in the waves' order and the parts' in the parts'."""
    KB, one = qa.shape[1] // 128, bfq.bfq_tile.from_dict({**_twin(bfq, t, wl).as_dict(), "split_k": 1})

    def w(blocks, cols):
        if not wl:
            return qw[:, cols].contiguous()
        return qw.view(qw.shape[0] // 16, KB, 2048)[:, blocks].contiguous().view(qw.shape[0], -1)
    total = None
    for z in range(t.split_k):
        part = None
        for v in range(t.waves_m):
            blocks = torch.tensor(range(z * KB // t.split_k + v, (z + 1) * KB // t.split_k, t.waves_m),
                                  dtype=torch.long, device=DEV)
            if len(blocks):
                cols = (blocks[:, None] * 128 + torch.arange(128, device=DEV)).flatten()
                x = bfq.block_gemm(qa[:, cols].contiguous(), sa[:, blocks].contiguous(),
                                   w(blocks, cols), sw[:, blocks].contiguous(),
                                   out_dtype=torch.float32, tile=one, w_layout=wl, scale_fmt=sfmt)
                part = x if part is None else part + x
        total = part if total is None else total + part
    return total.double()


def _gu(bfq, qa, sa, qw, sw, t, wl, sfmt):
    """(g, u) of gated tile t: the fp32 output of its twin on the 2F rows."""
    if t.variant == 1 and t.sched == 2:
        return _gu_interleaved(bfq, qa, sa, qw, sw, t, wl, sfmt)
    gu = bfq.block_gemm(qa, sa, qw, sw, out_dtype=torch.float32, tile=_twin(bfq, t, wl),
                        w_layout=wl, scale_fmt=sfmt)
    return gu.double()


def _h_ref(gu, act):
    F = gu.shape[1] // 2
    g, u = gu[:, :F], gu[:, F:]
    a, _, z = _act(g, act)
    h = a * u
    return h, (16 + 4 * z.abs()) * U * h.abs() + 1e-30 * (1 + (g * u).abs())


def _run_gated(bfq, qa, sa, qw, sw, odt, act, t, wl, sfmt, pre, a_layout=0, out_layout=0):
    M, K = qa.shape
    F = qw.shape[0] // 2
    codes = odt == torch.uint8
    pad = 64                                        # guard elements behind every output
    buf = torch.full((M * F + pad,), 77 if codes else 3.0, dtype=odt, device=DEV)
    pbuf = torch.full((M * 2 * F + pad,), 3.0, dtype=torch.bfloat16, device=DEV)
    scales = None
    if codes:
        G = F // 128
        if out_layout == bfq.BFQ_SCALES_PACKED_UE8M0:
            scales = torch.full(((G + 3) // 4, (M + 3) // 4 * 4 + 4), -1, dtype=torch.int32, device=DEV)
        else:
            shape = (M, G + 3) if out_layout == bfq.BFQ_SCALES_ROW_MAJOR else (G, M + 3)
            scales = torch.full(shape, 5.0, dtype=torch.float32, device=DEV)
    n = bfq.bfq_gated_gemm_workspace_bytes(M, F, K, bfq.BFQ_E4M3FN if codes else bfq.BFQ_BF16, wl, sfmt, t)
    ws = torch.full((n + 64,), 0xFF, dtype=torch.uint8, device=DEV)
    bfq.bfq_gated_gemm(qa, sa, qw, sw, buf[:M * F].view(M, F), act=act, a_layout=a_layout,
                       out_scales=scales, out_layout=out_layout,
                       preact=pbuf[:M * 2 * F].view(M, 2 * F) if pre else None, tile=t,
                       workspace=ws[:n] if n else None, w_layout=wl, scale_fmt=sfmt)
    torch.cuda.synchronize()
    assert bool((buf[M * F:] == (77 if codes else 3.0)).all()) and bool((ws[n:] == 0xFF).all())
    assert bool((pbuf[M * 2 * F if pre else 0:] == 3.0).all())
    return buf[:M * F].view(M, F), scales, pbuf[:M * 2 * F].view(M, 2 * F)


def _gated_tiles(bfq, wl, sfmt):
    return [bfq.bfq_gated_get_tile_candidate(i, wl, sfmt)
            for i in range(bfq.bfq_gated_num_tile_candidates(wl, sfmt))]


@pytest.mark.parametrize("act", [0, 1])
@pytest.mark.parametrize("sfmt", [0, 1])
@pytest.mark.parametrize("wl", [0, 1])
def test_gated_every_tile(bfq, wl, sfmt, act):
    """Each compiled tile, plain and with its K range split, at token counts around its height."""
    F, K = 384, 1152
    for n, t0 in enumerate(_gated_tiles(bfq, wl, sfmt)):
        for M, split in ((1, 1), (t0.bm, 1), (t0.bm + 1, 3), (2 * t0.bm - 3, 2)):
            d = t0.as_dict()
            t = bfq.bfq_tile.from_dict({**d, "split_k": split})
            print("gated", wl, sfmt, act, M, t.as_dict(), flush=True)
            qa, sa, qw, sw, _ = _pair(bfq, M, F, K, 100 + n, sfmt, wl)
            gu = _gu(bfq, qa, sa, qw, sw, t, wl, sfmt)
            h, tol = _h_ref(gu, act)
            for odt in (torch.float32, torch.bfloat16, torch.float16):
                out, _, pre = _run_gated(bfq, qa, sa, qw, sw, odt, act, t, wl, sfmt, True)
                _within(out, h, tol + H[odt] * h.abs() + TINY[odt], f"{odt} {t.as_dict()}")
                assert torch.equal(pre, gu.bfloat16()), t.as_dict()
            q, s, pre = _run_gated(bfq, qa, sa, qw, sw, torch.uint8, act, t, wl, sfmt, True)
            _check_codes(q, s[:, :F // 128], h, tol, sfmt == 1, f"{t.as_dict()}")
            assert bool((s[:, F // 128:] == 5.0).all())
            assert torch.equal(pre, gu.bfloat16()), t.as_dict()


@pytest.mark.parametrize("M,F,K", [(1, 128, 128), (2, 256, 7168), (5, 640, 384), (16, 2304, 1536),
                                   (47, 1536, 1536), (130, 2048, 640), (257, 1280, 2048),
                                   (1030, 768, 256)])
@pytest.mark.parametrize("a_lay,o_lay,sfmt", [(0, 0, 0), (1, 1, 0), (0, 1, 1), (2, 2, 1)])
def test_gated_selected_tile_and_layouts(bfq, M, F, K, a_lay, o_lay, sfmt):
    """The tile that the rule picks, every scale layout in and out, both weight layouts."""
    for wl in (0, 1):
        qa, sa, qw, sw, _ = _pair(bfq, M, F, K, M + F, sfmt, wl)
        t = bfq.bfq_gated_select_tile(M, F, K, w_layout=wl, scale_fmt=sfmt)
        print("gated select", M, F, K, wl, t.as_dict(), flush=True)
        gu = _gu(bfq, qa, sa, qw, sw, t, wl, sfmt)
        h, tol = _h_ref(gu, 0)
        sa_in = sa
        if a_lay == 1:
            sa_in = sa.t().contiguous()
        elif a_lay == 2:
            sa_in = bfq.quant_tokens(synth.activations(M, K, seed=M + F).to(DEV), scale_fmt=sfmt, layout=2)[1]
        out, _, _ = _run_gated(bfq, qa, sa_in, qw, sw, torch.bfloat16, 0, None, wl, sfmt, False, a_lay)
        _within(out, h, tol + H[torch.bfloat16] * h.abs(), f"{t.as_dict()}")
        # the rule may pick another tile when codes are wanted
        t = bfq.bfq_gated_select_tile(M, F, K, bfq.BFQ_E4M3FN, wl, sfmt)
        gu = _gu(bfq, qa, sa, qw, sw, t, wl, sfmt)
        h, tol = _h_ref(gu, 0)
        q, s, pre = _run_gated(bfq, qa, sa_in, qw, sw, torch.uint8, 0, None, wl, sfmt, True, a_lay, o_lay)
        _check_codes(q, _unpack_scales(bfq, s, o_lay, M, F // 128), h, tol, sfmt == 1, f"{t.as_dict()}")
        assert torch.equal(pre, gu.bfloat16())


def test_gated_against_64_bits(bfq):
    """Independent of the block GEMM: sums of dequantized operands in 64 bits, at the accuracy bar
    of the block GEMM (relative Frobenius 1e-3 on each factor; |act'| <= 1.13, so at most 1.13e-3
    and 1e-3 on the product's two terms), one output rounding on top."""
    for M, F, K, wl, sfmt in ((3, 512, 1024, 1, 0), (200, 512, 2048, 0, 0), (700, 1024, 1024, 1, 1)):
        qa, sa, qw, sw, row = _pair(bfq, M, F, K, 7, sfmt, wl)
        a = qa.view(torch.float8_e4m3fn).double() * sa.double().repeat_interleave(128, 1)
        w = (row.view(torch.float8_e4m3fn).double()
             * sw.double().repeat_interleave(128, 0).repeat_interleave(128, 1))
        gu = torch.mm(a, w.t())
        for act in (0, 1):
            g, u = gu[:, :F], gu[:, F:]
            v, slope, _ = _act(g, act)
            out = bfq.gated_gemm(qa, sa, qw, sw, act=act, out_dtype=torch.float32, w_layout=wl,
                                 scale_fmt=sfmt).double()
            # terms of the error: act'(g) u dg and act(g) du, with ||dg|| <= 1e-3 ||g|| spread evenly
            bar = 1e-3 * ((slope * u).norm() * g.norm() + v.norm() * u.norm()) / math.sqrt(g.numel())
            assert float((out - v * u).norm()) <= float(bar)


def test_gated_special_values(bfq):
    """Zero tokens, NaN codes, saturated and vanishing gates."""
    F, K = 256, 256
    for wl in (0, 1):
        qa, sa, qw, sw, _ = _pair(bfq, 40, F, K, 3, 0, wl)
        qa[0] = 0                                     # a token of zeros: outputs 0, scale eps / 448
        sa[1] *= 1e4                                  # gates far out on both sides
        qa[2, 5] = 0x7F                               # NaN code: the whole token's outputs are NaN
        t = bfq.bfq_gated_select_tile(40, F, K, w_layout=wl)
        gu = _gu(bfq, qa, sa, qw, sw, t, wl, 0)
        for act in (0, 1):
            h, tol = _h_ref(gu, act)
            out = bfq.gated_gemm(qa, sa, qw, sw, act=act, out_dtype=torch.float32, w_layout=wl)
            _within(out, h, tol + U * h.abs(), f"wl {wl} act {act}")
            assert bool((out[0] == 0).all()) and bool(out[2].isnan().all())
            tc = bfq.bfq_gated_select_tile(40, F, K, bfq.BFQ_E4M3FN, wl)
            h, tol = _h_ref(_gu(bfq, qa, sa, qw, sw, tc, wl, 0), act)
            q, s = bfq.gated_gemm(qa, sa, qw, sw, act=act, codes=True, w_layout=wl)
            assert not bool(q[0].view(torch.float8_e4m3fn).float().any())
            assert torch.equal(s[0], torch.full_like(s[0], np.float32(1e-10) / np.float32(448)))
            assert bool((q[2] == 0x7F).all()) and bool(s[2].isnan().all())
            keep = torch.arange(40, device=DEV) != 2
            _check_codes(q[keep], s[keep], h[keep], tol[keep], False, f"wl {wl} act {act}")


@pytest.mark.parametrize("wl", [0, 1])
@pytest.mark.parametrize("sfmt", [0, 1])
def test_gated_batch_invariant(bfq, wl, sfmt):
    """With the batch-invariant switch set, a token's outputs do not depend on the batch."""
    F, K = 512, 1536
    kw = dict(w_layout=wl, scale_fmt=sfmt)
    was = bfq.bfq_get_batch_invariant()
    bfq.bfq_set_batch_invariant(True)
    try:
        qa, sa, qw, sw, _ = _pair(bfq, 600, F, K, 5, sfmt, wl)
        full = bfq.gated_gemm(qa, sa, qw, sw, out_dtype=torch.float32, **kw)
        qf, sf = bfq.gated_gemm(qa, sa, qw, sw, codes=True, **kw)
        for M in (1, 16, 30, 64, 100, 129, 513):
            part = bfq.gated_gemm(qa[:M], sa[:M].contiguous(), qw, sw, out_dtype=torch.float32, **kw)
            assert torch.equal(part, full[:M]), M
            q, s = bfq.gated_gemm(qa[:M], sa[:M].contiguous(), qw, sw, codes=True, **kw)
            assert torch.equal(q, qf[:M]) and torch.equal(s, sf[:M]), M
    finally:
        bfq.bfq_set_batch_invariant(was)


# ---------------------------------------------------------------------- gated backward

def _pre(M, F, seed):
    pre = (_randn(seed, M, 2 * F) * 2).bfloat16()
    if M > 2:
        pre[1, :F] *= 60                              # gates on the flat ends
        pre[2] = 0
    return pre, (_randn(seed + 1, M, F) * 0.3).bfloat16()


@pytest.mark.parametrize("act", [0, 1])
@pytest.mark.parametrize("M,F", [(1, 8), (3, 136), (7, 2048), (65, 2056), (129, 18432), (1, 128)])
def test_gated_backward_bf16(bfq, M, F, act):
    pre, dh = _pre(M, F, M + F)
    dpre, h = bfq.gated_backward(pre, dh, act=act, want_h=True)
    g, u, d = pre[:, :F].double(), pre[:, F:].double(), dh.double()
    a, slope, z = _act(g, act)
    b = H[torch.bfloat16]
    rel = (24 + 4 * z.abs()) * U
    tiny = 1e-30 * (1 + g.abs()) * (1 + u.abs())
    _within(h, a * u, (rel + b) * (a * u).abs() + tiny, "h")
    _within(dpre[:, F:], d * a, (rel + b) * (d * a).abs() + tiny, "du")
    # the slope is a sum of p and g p (1 - p) (c1 + 3 c3 g^2): its error counts both terms, and 1 - p
    # carries u of 1 where p rounds
    p = torch.sigmoid(z)
    k = 1 if act == 0 else 2 * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * g * g)
    terms = p + (a * k).abs() * ((1 - p) + 4 * U) + 4 * U * 0
    tol = rel * terms + 4 * U * (a * k).abs()
    _within(dpre[:, :F], d * u * slope, (d * u).abs() * tol + b * (d * u * slope).abs() + tiny, "dg")
    only = torch.full((M, F), 3.0, dtype=torch.bfloat16, device=DEV)
    bfq.bfq_gated_backward(pre, dh, act=act, h=only)
    assert torch.equal(only, h)
    bfq.bfq_gated_backward(pre, dh, act=act, dpre=pre, h=dh)            # both in place
    assert torch.equal(pre, dpre) and torch.equal(dh, h)


@pytest.mark.parametrize("lay,sfmt,int8", [(0, 0, False), (1, 0, True), (1, 1, False), (2, 1, False),
                                           (2, 1, True)])
@pytest.mark.parametrize("M,F", [(1, 128), (3, 384), (66, 2176), (5, 4608)])
def test_gated_backward_codes(bfq, M, F, lay, sfmt, int8):
    """Codes of the gradient: both halves' groups, words that straddle them (F / 128 odd)."""
    pre, dh = _pre(M, F, M + F)
    g, u, d = pre[:, :F].double(), pre[:, F:].double(), dh.double()
    a, slope, z = _act(g, 0)
    ref = torch.cat([d * u * slope, d * a], 1)
    p = torch.sigmoid(z)
    rel = (24 + 4 * z.abs()) * U
    tol = torch.cat([(d * u).abs() * (rel * (p + a.abs()) + 4 * U * a.abs()), rel * (d * a).abs()], 1) + 1e-28
    q, s = bfq.gated_backward(pre, dh, codes=True, layout=lay, scale_fmt=sfmt,
                              q_dtype=bfq.BFQ_INT8 if int8 else bfq.BFQ_E4M3FN)
    s = _unpack_scales(bfq, s, lay, M, 2 * F // 128)
    _check_codes(q, s, ref, tol, sfmt == 1, "dpre", int8=int8)


@pytest.mark.parametrize("act", [0, 1])
def test_gated_backward_against_differences(bfq, act):
    """The gradient along a direction against central differences of the product in 64 bits."""
    M, F = 9, 256
    pre, dh = _pre(M, F, 11)
    dpre = bfq.gated_backward(pre, dh, act=act).double()
    v = _randn(12, M, 2 * F).double()

    def loss(x):
        return (_act(x[:, :F], act)[0] * x[:, F:] * dh.double()).sum()
    e = 1e-5
    want = (loss(pre.double() + e * v) - loss(pre.double() - e * v)) / (2 * e)
    # bf16 outputs: half a step each; the differences' own error is of order e^2
    tol = (H[torch.bfloat16] * (dpre * v).abs()).sum() + 1e-6 * (dpre * v).abs().sum() + 1e-7
    assert abs(float((dpre * v).sum() - want)) <= float(tol)


@pytest.mark.parametrize("N,K", [(128, 128), (256, 640), (4096, 1536), (1536, 7168)])
def test_transpose_weights(bfq, N, K):
    for dt in (torch.uint8, torch.int8):
        w = torch.randint(0, 127, (N, K), dtype=dt, device=DEV, generator=_gen(N))
        s = _randn(K, N // 128, K // 128)
        wt, st = bfq.transpose_weights(w, s)
        assert torch.equal(wt, w.t()) and torch.equal(st, s.t())


# ------------------------------------------------------------------------------- norms

def _norm_case(M, K, post, kind, rt, seed):
    c = {"y": (_randn(seed, M, K) * 0.7).bfloat16(), "w_pre": (1 + 0.3 * _randn(seed + 1, K)).bfloat16(),
         "w_post": (1 + 0.3 * _randn(seed + 2, K)).bfloat16() if post else None,
         "residual": (_randn(seed + 3, M, K) * 3).to(rt)}
    shape = {0: None, 1: (K,), 2: (M,), 3: (M, K)}[kind]
    c["gate"] = (0.5 + 0.5 * _randn(seed + 4, *shape)).bfloat16() if shape else None
    c["gate_kind"] = kind
    c["res_scale"] = 0.6
    return c


def _norm_ref(c, eps=1e-6):
    """r', n and their tolerances in 64 bits."""
    r0 = c["residual"].double()
    alpha = float(np.float32(c["res_scale"]))
    g = torch.ones((), device=DEV, dtype=torch.float64) if c["gate"] is None else c["gate"].double()
    if c["gate_kind"] == 2:
        g = g[:, None]
    rms = lambda x: 1 / torch.sqrt(x.square().mean(1, keepdim=True) + eps)  # noqa: E731
    r, rtol = r0, torch.zeros_like(r0)
    if c["y"] is not None:
        y = c["y"].double()
        z = y * rms(y) * c["w_post"].double() if c["w_post"] is not None else y
        r = r0 + alpha * g * z
        rtol = U * r.abs() + 60 * U * (alpha * g * z).abs()
    n, ntol = None, None
    if c["w_pre"] is not None:
        w = c["w_pre"].double()
        n = r * rms(r) * w
        ntol = 60 * U * n.abs() + 2 * rtol * rms(r) * w.abs()
    return r, rtol, n, ntol


KS = [8, 72, 128, 200, 1544, 2048, 4096, 7168, 8200, 16384]


@pytest.mark.parametrize("rt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("K", KS)
def test_norm_bf16_out(bfq, K, rt):
    for M in (1, 5, 130):
        for post in (False, True):
            for kind in range(4):
                c = _norm_case(M, K, post, kind, rt, K + M)
                r, rtol, n, ntol = _norm_ref(c)
                res, nrm = bfq.norm_residual(**c)
                _within(res, r, rtol + H[rt] * r.abs(), f"res {M} {post} {kind}")
                _within(nrm, n, ntol + H[torch.bfloat16] * n.abs(), f"normed {M} {post} {kind}")
                c2 = dict(c, w_pre=None)
                (alone,) = bfq.norm_residual(**c2)
                assert torch.equal(alone, res)
                same = c["residual"].clone()          # in place
                bfq.bfq_norm_residual(same, **{k: v for k, v in c2.items() if k != "residual"}, res_out=same)
                assert torch.equal(same, res)
        c = _norm_case(M, K, False, 0, rt, K + M)
        c["y"] = None
        _, _, n, ntol = _norm_ref(c)
        (nrm,) = bfq.norm_residual(**c)
        _within(nrm, n, ntol + H[torch.bfloat16] * n.abs(), f"plain norm {M}")


@pytest.mark.parametrize("lay,sfmt,int8,per_token", [
    (0, 0, False, False), (1, 0, True, False), (1, 1, False, False), (2, 1, False, False),
    (2, 1, True, False), (0, 0, False, True), (1, 0, True, True), (0, 1, False, True)])
@pytest.mark.parametrize("K", [128, 256, 640, 1536, 2176, 7168, 16384])
def test_norm_codes(bfq, K, lay, sfmt, int8, per_token):
    for M, post, kind, rt in ((1, True, 1, torch.bfloat16), (7, False, 0, torch.float32),
                              (66, True, 2, torch.float32)):
        c = _norm_case(M, K, post, kind, rt, K + M)
        r, rtol, n, ntol = _norm_ref(c)
        G = 1 if per_token else K // 128
        res, q, s = bfq.norm_residual(**c, codes=True, layout=lay, scale_fmt=sfmt, per_token=per_token,
                                      q_dtype=bfq.BFQ_INT8 if int8 else bfq.BFQ_E4M3FN)
        _within(res, r, rtol + H[rt] * r.abs(), "res")
        s = _unpack_scales(bfq, s, lay, M, G)
        _check_codes(q, s, n, ntol, sfmt == 1, f"{M}", int8=int8, group=K if per_token else 128)
        both_n, both_q = torch.empty_like(c["y"]), torch.empty_like(q)
        s2 = torch.empty((M, G), dtype=torch.float32, device=DEV)
        bfq.bfq_norm_residual(**c, res_out=res, normed=both_n, q=both_q, scales=s2,
                              group_size=K if per_token else 128, scale_fmt=sfmt)
        assert torch.equal(both_q, q) and torch.equal(s2, s)
        _within(both_n, n, ntol + H[torch.bfloat16] * n.abs(), "normed with codes")


def test_norm_special_rows(bfq):
    """Rows of zeros, a NaN, an infinity; neighbours keep their values."""
    M, K = 6, 512
    c = _norm_case(M, K, True, 0, torch.float32, 1)
    clean = bfq.norm_residual(**c, codes=True)
    c["y"][1] = 0
    c["residual"][1] = 0
    c["residual"][2, 7] = float("nan")
    c["residual"][4, 9] = float("inf")
    res, q, s = bfq.norm_residual(**c, codes=True)
    for a, b in zip((res, q, s), clean):
        assert torch.equal(a[[0, 3, 5]], b[[0, 3, 5]])
    assert not bool(res[1].any()) and not bool((q[1] & 0x7F).any())
    assert bool(s[2].isnan().all()) and bool((q[2] == 0x7F).all())      # rms is NaN
    assert bool(s[4, 0].isnan()) and bool((q[4, :128] == 0x7F).all())   # inf * 0
    assert bool(torch.isinf(res[4, 9])) and not bool(q[4, 128:].view(torch.float8_e4m3fn).float().any())


def _bwd_ref(c, r, dn, dro, eps=1e-6):
    """Gradients and tolerances in 64 bits; r is the stored sum."""
    alpha = float(np.float32(c["res_scale"]))
    K = r.shape[1]
    r = r.double()
    g = torch.ones((), device=DEV, dtype=torch.float64) if c["gate"] is None else c["gate"].double()
    if c["gate_kind"] == 2:
        g = g[:, None]
    zero = torch.zeros_like(r)
    dr, tol = (dro.double(), U * dro.double().abs()) if dro is not None else (zero, zero.clone())
    out, tols = {}, {}
    A = 150 * U
    if c["w_pre"] is not None:
        w, d = c["w_pre"].double(), dn.double()
        ir = 1 / torch.sqrt(r.square().mean(1, keepdim=True) + eps)
        x = r * ir
        dr = dr + ir * (w * d - x * (w * d * x).mean(1, keepdim=True))
        tol = tol + A * (dr.abs() + ir * ((w * d).abs() + x.abs() * (w * d * x).abs().mean(1, keepdim=True)))
        out["d_w_pre"] = (d * x).sum(0)
        tols["d_w_pre"] = A * (d * x).abs().sum(0)
    out["d_res"], tols["d_res"] = dr, tol
    if c["y"] is None:
        return out, tols
    y = c["y"].double()
    dz, dztol = alpha * g * dr, (alpha * g).abs() * (tol + 4 * U * dr.abs())
    if c["w_post"] is not None:
        w = c["w_post"].double()
        iy = 1 / torch.sqrt(y.square().mean(1, keepdim=True) + eps)
        x = y * iy
        z = x * w
        t = dz * w
        out["d_y"] = iy * (t - x * (t * x).mean(1, keepdim=True))
        tabs, ttol = t.abs(), dztol * w.abs()
        tols["d_y"] = (A * iy * (tabs + x.abs() * (tabs * x.abs()).mean(1, keepdim=True))
                       + iy * (ttol + x.abs() * (ttol * x.abs()).mean(1, keepdim=True)))
        out["d_w_post"] = (dz * x).sum(0)
        tols["d_w_post"] = ((A * dz.abs() + dztol) * x.abs()).sum(0)
    else:
        z = y
        out["d_y"], tols["d_y"] = dz.expand_as(y), dztol.expand_as(y)
    dg, dgtol = alpha * dr * z, abs(alpha) * (tol + A * dr.abs()) * z.abs()
    if c["gate_kind"] in (1, 2):
        ax = 0 if c["gate_kind"] == 1 else 1
        out["d_gate"] = dg.sum(ax)
        tols["d_gate"] = (dgtol + A * dg.abs()).sum(ax)
    elif c["gate_kind"] == 3:
        out["d_gate"], tols["d_gate"] = dg, dgtol
    return out, tols


@pytest.mark.parametrize("rt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("K", KS)
def test_norm_backward(bfq, K, rt):
    for M in (1, 7, 300):
        for post in (False, True):
            for kind in range(4):
                c = _norm_case(M, K, post, kind, rt, K + M)
                r = c.pop("residual")
                dn = (_randn(K + 9, M, K) * 0.1).bfloat16()
                dro = (_randn(K + 10, M, K) * 0.1).to(rt) if (M + kind) % 3 else None
                ref, tols = _bwd_ref(c, r, dn, dro)
                got = bfq.norm_residual_backward(r, **c, d_normed=dn, d_res_out=dro)
                assert set(got) == set(ref)
                for k in ref:
                    _within(got[k], ref[k], tols[k] + H[got[k].dtype] * ref[k].abs() + 1e-30,
                            f"{k} M {M} post {post} gate {kind}")
                again = bfq.norm_residual_backward(r, **c, d_normed=dn, d_res_out=dro)
                assert all(torch.equal(got[k], again[k]) for k in got)


def test_norm_backward_parts(bfq):
    """Operands left out: no pre-norm, no y; gradients not asked for; in place; M = 0."""
    M, K = 33, 1544
    c = _norm_case(M, K, True, 1, torch.float32, 4)
    r = c.pop("residual")
    dro = _randn(5, M, K)
    c1 = dict(c, w_pre=None)
    ref, tols = _bwd_ref(c1, r, None, dro)
    got = bfq.norm_residual_backward(r, **c1, d_res_out=dro)
    for k in ref:
        _within(got[k], ref[k], tols[k] + H[got[k].dtype] * ref[k].abs(), k)
    assert torch.equal(got["d_res"], dro)
    c2 = dict(c, y=None, w_post=None, gate=None, gate_kind=0)
    dn = _randn(6, M, K).bfloat16()
    ref, tols = _bwd_ref(c2, r, dn, dro)
    got = bfq.norm_residual_backward(r, **c2, d_normed=dn, d_res_out=dro)
    assert set(got) == {"d_res", "d_w_pre"}
    for k in ref:
        _within(got[k], ref[k], tols[k] + H[got[k].dtype] * ref[k].abs(), k)
    full = bfq.norm_residual_backward(r, **c, d_normed=dn, d_res_out=dro)
    same, dy = dro.clone(), torch.empty_like(c["y"])
    bfq.bfq_norm_residual_backward(r, same, **c, d_normed=dn, d_res_out=same, d_y=dy)   # in place, no sums
    assert torch.equal(same, full["d_res"]) and torch.equal(dy, full["d_y"])
    e = lambda t: t[:0]  # noqa: E731
    empty = bfq.norm_residual_backward(e(r), **dict(c, y=e(c["y"])), d_normed=e(dn), d_res_out=e(dro))
    assert all(not bool(empty[k].any()) for k in ("d_w_pre", "d_w_post", "d_gate"))


@pytest.mark.parametrize("K", [8192, 8200, 12288])
def test_norm_backward_in_place_long_rows(bfq, K):
    """In place on both sides of the widest row that a workgroup holds in one chunk a thread, with
    more rows than workgroups (each then walks several)."""
    M = 700
    c = _norm_case(M, K, True, 1, torch.float32, K)
    r = c.pop("residual")
    dn, dro = _randn(K + 1, M, K).bfloat16(), _randn(K + 2, M, K)
    full = bfq.norm_residual_backward(r, **c, d_normed=dn, d_res_out=dro)
    ref, tols = _bwd_ref(c, r, dn, dro)
    for k in ref:
        _within(full[k], ref[k], tols[k] + H[full[k].dtype] * ref[k].abs() + 1e-30, k)
    same, dy = dro.clone(), torch.empty_like(c["y"])
    bfq.bfq_norm_residual_backward(r, same, **c, d_normed=dn, d_res_out=same, d_y=dy)
    assert torch.equal(same, full["d_res"]) and torch.equal(dy, full["d_y"])


@pytest.mark.parametrize("kind", range(4))
def test_norm_backward_against_differences(bfq, kind):
    """Every gradient along a random direction against central differences in 64 bits."""
    M, K = 6, 264
    c = _norm_case(M, K, True, kind, torch.float32, 20 + kind)
    A, B = (_randn(30, M, K) * 0.1).bfloat16(), _randn(31, M, K) * 0.1
    r, _, _, _ = _norm_ref(c)
    stored = r.float()
    got = bfq.norm_residual_backward(stored, **{k: v for k, v in c.items() if k != "residual"},
                                     d_normed=A, d_res_out=B)

    def loss(d):
        r, _, n, _ = _norm_ref(d)
        return (n * A.double()).sum() + (r * B.double()).sum()
    for name, grad in (("residual", "d_res"), ("y", "d_y"), ("w_pre", "d_w_pre"),
                       ("w_post", "d_w_post"), ("gate", "d_gate")):
        if c[name] is None:
            continue
        v = torch.randn(c[name].shape, generator=_gen(40), device=DEV, dtype=torch.float64)
        e = 1e-5
        want = (loss({**c, name: c[name].double() + e * v}) - loss({**c, name: c[name].double() - e * v})) / (2 * e)
        gv = got[grad].double() * v
        tol = (H[got[grad].dtype] + 1e-5) * gv.abs().sum() + 1e-7
        assert abs(float(gv.sum() - want)) <= float(tol), name


# ------------------------------------------------------------------------- used together

def test_feed_forward_block_and_its_gradient(bfq):
    """A whole block as it is used: norm to codes, gated product to codes, down projection, the
    residual step of the next block; then its gradient back to the residual stream, through
    quantized gradients and transposed weights. Each stage against 64 bits on its own inputs: the
    GEMMs at their accuracy bar (relative Frobenius 1e-3) plus their output's rounding."""
    M, K, F = 150, 1536, 2048
    wl, sf = bfq.BFQ_W_PACKED16, bfq.BFQ_SCALE_FP32
    r0 = synth.activations(M, K, seed=1).to(DEV)
    w1, w2 = ((1 + 0.1 * _randn(s, K)).bfloat16() for s in (2, 3))
    gate = (1 + 0.1 * _randn(4, K)).bfloat16()
    wgu, wd = _randn(5, 2 * F, K) * 0.02, _randn(6, K, F) * 0.02
    qgu, sgu = bfq.quant_weight_blocks(wgu)
    qd, sd = bfq.quant_weight_blocks(wd)
    deq = lambda q, s, r: (q.view(torch.float8_e4m3fn).double()  # noqa: E731
                           * (s.double().repeat_interleave(r, 0) if r > 1 else s.double())
                           .repeat_interleave(128, 1))
    near = lambda got, ref, rel: float((got.double() - ref).norm()) <= rel * float(ref.norm())  # noqa: E731
    qx, sx = bfq.norm_residual(r0, w_pre=w1, codes=True)
    qh, sh, pre = bfq.gated_gemm(qx, sx, bfq.pack_weights(qgu), sgu, codes=True, keep_preact=True, w_layout=wl)
    y = bfq.block_gemm(qh, sh, bfq.pack_weights(qd), sd, w_layout=wl)
    gu = deq(qx, sx, 1) @ deq(qgu, sgu, 128).t()
    b = 2.0 ** -8
    assert near(pre, gu, 1e-3 + b)
    assert near(y, deq(qh, sh, 1) @ deq(qd, sd, 128).t(), 1e-3 + b)
    r1, n1 = bfq.norm_residual(r0, y=y, gate=gate, gate_kind=bfq.BFQ_GATE_CHANNEL, w_pre=w2)
    # backward, from gradients of r1 and n1
    dn, dr1 = (_randn(7, M, K) * 0.1).bfloat16(), (_randn(8, M, K) * 0.1).bfloat16()
    g1 = bfq.norm_residual_backward(r1, y=y, gate=gate, gate_kind=bfq.BFQ_GATE_CHANNEL, w_pre=w2,
                                    d_normed=dn, d_res_out=dr1)
    qdt, sdt = bfq.transpose_weights(qd, sd)                    # [F, K]
    qgt, sgt = bfq.transpose_weights(qgu, sgu)                  # [K, 2F]
    qy, sy = bfq.quant_tokens(g1["d_y"])
    dh = bfq.block_gemm(qy, sy, bfq.pack_weights(qdt), sdt, w_layout=wl)
    assert near(dh, deq(qy, sy, 1) @ deq(qd, sd, 128), 1e-3 + b)
    qg, sg = bfq.gated_backward(pre, dh, codes=True)
    dx = bfq.block_gemm(qg, sg, bfq.pack_weights(qgt), sgt, w_layout=wl)
    assert near(dx, deq(qg, sg, 1) @ deq(qgu, sgu, 128), 1e-3 + b)
    g0 = bfq.norm_residual_backward(r0, w_pre=w1, d_normed=dx, d_res_out=g1["d_res"])
    # the whole gradient against autograd through the dequantized block in 64 bits: codes of
    # activations and of gradients are each off by up to 2^-4 of a value, 2^-5 on the mean square
    # root of a step's uniform error (2^-4 / sqrt(3) at worst), in four quantizations on the way
    x = r0.double().requires_grad_()
    rms = lambda t: t / torch.sqrt(t.square().mean(1, keepdim=True) + 1e-6)  # noqa: E731
    p = (rms(x) * w1.double()) @ deq(qgu, sgu, 128).t()
    yy = (p[:, :F] * torch.sigmoid(p[:, :F]) * p[:, F:]) @ deq(qd, sd, 128).t()
    rr = x + gate.double() * yy
    ((rms(rr) * w2.double() * dn.double()).sum() + (rr * dr1.double()).sum()).backward()
    assert near(g0["d_res"], x.grad, 4 * 2.0 ** -4 / math.sqrt(3))


def test_streams_and_graphs(bfq):
    """Calls on a side stream; a captured sequence replayed with eager work between."""
    M, K, F = 70, 1536, 1280
    c = _norm_case(M, K, True, 1, torch.bfloat16, 50)
    qgu, sgu = bfq.quant_weight_blocks(_randn(51, 2 * F, K) * 0.02)
    res, q, s = (torch.empty_like(c["residual"]), torch.empty((M, K), dtype=torch.uint8, device=DEV),
                 torch.empty((M, K // 128), device=DEV))
    tile = bfq.bfq_gated_select_tile(M, F, K)
    tile.split_k = 3
    n = bfq.bfq_gated_gemm_workspace_bytes(M, F, K, bfq.BFQ_E4M3FN, tile=tile)
    ws = torch.empty(n, dtype=torch.uint8, device=DEV)
    h, hs = torch.empty((M, F), dtype=torch.uint8, device=DEV), torch.empty((M, F // 128), device=DEV)
    pre = torch.empty((M, 2 * F), dtype=torch.bfloat16, device=DEV)
    dh = (_randn(52, M, F) * 0.1).bfloat16()
    dpre = torch.empty_like(pre)
    dn = (_randn(53, M, K) * 0.1).bfloat16()
    g = {"d_res": torch.empty_like(res), "d_y": torch.empty_like(res), "d_w_pre": torch.empty(K, device=DEV),
         "d_w_post": torch.empty(K, device=DEV), "d_gate": torch.empty(K, device=DEV)}
    wsb = torch.empty(bfq.bfq_norm_residual_backward_workspace_bytes(M, K), dtype=torch.uint8, device=DEV)
    nb = {k: v for k, v in c.items() if k != "residual"}

    def step():
        bfq.bfq_norm_residual(**c, res_out=res, q=q, scales=s)
        bfq.bfq_gated_gemm(q, s, qgu, sgu, h, out_scales=hs, preact=pre, tile=tile, workspace=ws)
        bfq.bfq_gated_backward(pre, dh, dpre=dpre)
        bfq.bfq_norm_residual_backward(res, **nb, d_normed=dn, workspace=wsb, **g)
    outs = [res, q, s, h, hs, pre, dpre] + list(g.values())
    step()
    torch.cuda.synchronize()
    want = [o.clone() for o in outs]

    def check():
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want))
        for o in outs:
            o.zero_()
    check()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    check()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(4):
        graph.replay()
        torch.cuda.synchronize()
        torch.ones(1 << 20, device=DEV).sum()
        check()


def test_two_streams_at_once(bfq):
    """Calls in flight on two streams, each with its own workspace and outputs."""
    M, K, F = 40, 2048, 1024
    qw, sw = bfq.quant_weight_blocks(_randn(60, 2 * F, K) * 0.02)
    tile = bfq.bfq_gated_select_tile(M, F, K)
    tile.split_k = 4
    n = bfq.bfq_gated_gemm_workspace_bytes(M, F, K, tile=tile)
    jobs = []
    for i in range(2):
        qa, sa = bfq.quant_tokens(synth.activations(M, K, seed=61 + i).to(DEV))
        c = _norm_case(300, 1544, True, 1, torch.bfloat16, 70 + i)
        jobs.append((qa, sa, torch.empty(n, dtype=torch.uint8, device=DEV),
                     torch.empty((M, F), dtype=torch.bfloat16, device=DEV), c, torch.cuda.Stream()))
    want = [bfq.gated_gemm(qa, sa, qw, sw, tile=tile) for qa, sa, *_ in jobs]
    rn = [bfq.norm_residual(**c) for *_, c, _ in jobs]
    torch.cuda.synchronize()
    for _ in range(5):
        got = []
        for qa, sa, ws, out, c, st in jobs:
            with torch.cuda.stream(st):
                bfq.bfq_gated_gemm(qa, sa, qw, sw, out, tile=tile, workspace=ws)
                got.append(bfq.norm_residual(**c))
        torch.cuda.synchronize()
        for w, r, g, (*_, out, _, _) in zip(want, rn, got, jobs):
            assert torch.equal(out, w) and all(torch.equal(a, b) for a, b in zip(g, r))


def test_empty_batches(bfq):
    qgu, sgu = bfq.quant_weight_blocks(_randn(1, 256, 256))
    q, s = torch.empty((0, 256), dtype=torch.uint8, device=DEV), torch.empty((0, 2), device=DEV)
    assert bfq.gated_gemm(q, s, qgu, sgu).shape == (0, 128)
    assert bfq.gated_gemm(q, s, qgu, sgu, codes=True)[0].shape == (0, 128)
    assert bfq.gated_backward(q.bfloat16(), torch.empty((0, 128), device=DEV).bfloat16()).shape == (0, 256)
    assert bfq.norm_residual(torch.empty((0, 256), device=DEV),
                             w_pre=torch.ones(256, device=DEV).bfloat16())[0].shape == (0, 256)


def test_offsets_past_32_bits(bfq):
    """Rows whose element offsets pass 2^31: the last rows against a call on those rows alone."""
    F = 16384
    M = (1 << 31) // (2 * F) + 3                      # preact has 2^31 + 6F elements
    pre = torch.empty((M, 2 * F), dtype=torch.bfloat16, device=DEV)
    pre.normal_(generator=_gen(1))
    dh = torch.empty((M, F), dtype=torch.bfloat16, device=DEV).normal_(generator=_gen(2))
    dpre = bfq.gated_backward(pre, dh)
    tail = slice(M - 4, M)
    assert torch.equal(dpre[tail], bfq.gated_backward(pre[tail].contiguous(), dh[tail].contiguous()))
    q, s = bfq.gated_backward(pre, dh, codes=True)
    q4, s4 = bfq.gated_backward(pre[tail].contiguous(), dh[tail].contiguous(), codes=True)
    assert torch.equal(q[tail], q4) and torch.equal(s[tail], s4)
    del dpre, q, s
    x = pre.view(2 * M, F)                            # 2^31 elements of a residual stream
    w = torch.ones(F, device=DEV).bfloat16()
    tail = slice(2 * M - 4, 2 * M)
    res, nrm = bfq.norm_residual(x, y=x, w_post=w, w_pre=w)
    res4, nrm4 = bfq.norm_residual(x[tail].contiguous(), y=x[tail].contiguous(), w_post=w, w_pre=w)
    assert torch.equal(res[tail], res4) and torch.equal(nrm[tail], nrm4)
    got = bfq.norm_residual_backward(res, y=x, w_post=w, w_pre=w, d_normed=nrm)
    got4 = bfq.norm_residual_backward(res4, y=x[tail].contiguous(), w_post=w, w_pre=w, d_normed=nrm4)
    assert torch.equal(got["d_res"][tail], got4["d_res"]) and torch.equal(got["d_y"][tail], got4["d_y"])
    del res, nrm, got
    # gated product: out past 2^31 elements
    K, F2 = 128, 16384
    M2 = (1 << 31) // F2 + 5
    qa, sa = bfq.quant_tokens(pre.view(-1)[:M2 * K].view(M2, K))
    qw, sw = bfq.quant_weight_blocks(_randn(3, 2 * F2, K))
    out = bfq.gated_gemm(qa, sa, qw, sw)
    tail = slice(M2 - 130, M2)
    t = bfq.bfq_gated_select_tile(M2, F2, K)
    part = bfq.gated_gemm(qa[tail].contiguous(), sa[tail].contiguous(), qw, sw, tile=t)
    assert torch.equal(out[tail], part)


def test_readme_example():
    """The feed-forward example of the README runs as it stands, after its first one."""
    import os
    import re
    text = open(os.path.join(os.path.dirname(__file__), "..", "README.md")).read()
    code = re.findall(r"```python\n(.*?)```", text, re.S)
    env = {}
    for block in code:
        exec(block.replace('device="cuda"', 'device="cuda:0"'), env)
    torch.cuda.synchronize()
    assert env["out"].shape == (64, 7168) and env["dx"].shape == (64, 7168)
    assert all(bool(env[n].float().isfinite().all()) for n in ("y", "res", "out", "dx"))


@pytest.mark.parametrize("rt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("K", [1536, 7168, 12288])
def test_large_outputs_equal_small_ones(bfq, K, rt):
    """Calls that write more than the L2s hold store past them; their rows are those of a small
    call, bit for bit (300 rows: fewer may split a long row over more threads)."""
    M = (40 << 20) // (2 * K)
    some = torch.linspace(0, M - 1, 300, device=DEV).long()
    c = _norm_case(M, K, True, 3, rt, K)
    small = {k: v[some].contiguous() if k in ("residual", "y", "gate") else v for k, v in c.items()}
    for kw in (dict(codes=False), dict(codes=True), dict(codes=True, q_dtype=bfq.BFQ_INT8, per_token=True)):
        for a, b in zip(bfq.norm_residual(**c, **kw), bfq.norm_residual(**small, **kw)):
            assert torch.equal(a[some], b)
    r, rs = c.pop("residual"), small.pop("residual")
    dn, dro = (_randn(K + 1, M, K) * 0.1).bfloat16(), (_randn(K + 2, M, K) * 0.1).to(rt)
    a = bfq.norm_residual_backward(r, **c, d_normed=dn, d_res_out=dro)
    b = bfq.norm_residual_backward(rs, **small, d_normed=dn[some].contiguous(), d_res_out=dro[some].contiguous())
    for k in ("d_res", "d_y", "d_gate"):
        assert torch.equal(a[k][some], b[k]), k


def test_large_gated_outputs_equal_small_ones(bfq):
    F, K = 2048, 256
    M = (40 << 20) // F                               # more than 32 MB even as codes
    some = torch.tensor([0, 1, M // 2, M - 1], device=DEV)
    for wl, sfmt in ((0, 0), (1, 0), (1, 1)):
        qa, sa, qw, sw, _ = _pair(bfq, M, F, K, 11, sfmt, wl)
        t = bfq.bfq_gated_select_tile(M, F, K, bfq.BFQ_E4M3FN, wl, sfmt)
        kw = dict(keep_preact=True, tile=t, w_layout=wl, scale_fmt=sfmt)
        qs, ss = qa[some].contiguous(), sa[some].contiguous()
        for codes in (False, True):
            for a, b in zip(bfq.gated_gemm(qa, sa, qw, sw, codes=codes, **kw),
                            bfq.gated_gemm(qs, ss, qw, sw, codes=codes, **kw)):
                assert torch.equal(a[some], b)
    pre, dh = _randn(12, M, 2 * F).bfloat16(), _randn(13, M, F).bfloat16()
    for codes in (False, True):
        for a, b in zip(bfq.gated_backward(pre, dh, codes=codes, want_h=True),
                        bfq.gated_backward(pre[some].contiguous(), dh[some].contiguous(), codes=codes, want_h=True)):
            assert torch.equal(a[some], b)


@pytest.mark.parametrize("wl", [0, 1])
def test_gated_longest_k(bfq, wl):
    """K = 2^23, the longest: offsets inside a tile's operands stay below 2^32."""
    F, K = 128, 1 << 23
    g = _gen(5)
    qw = torch.randint(0, 120, (2 * F, K), dtype=torch.uint8, device=DEV, generator=g)
    sw = torch.rand(2, K // 128, device=DEV, generator=g) * 1e-4
    qw = bfq.pack_weights(qw) if wl else qw
    for M in (3, 40, 130):
        qa = torch.randint(0, 250, (M, K), dtype=torch.uint8, device=DEV, generator=g)
        qa[(qa & 0x7F) == 0x7F] = 0
        sa = torch.rand(M, K // 128, device=DEV, generator=g) * 1e-3
        t = bfq.bfq_gated_select_tile(M, F, K, w_layout=wl)
        print("longest K", wl, M, t.as_dict(), flush=True)
        gu = _gu(bfq, qa, sa, qw, sw, t, wl, 0)
        h, tol = _h_ref(gu, 0)
        out, _, pre = _run_gated(bfq, qa, sa, qw, sw, torch.float32, 0, t, wl, 0, True)
        _within(out, h, tol + U * h.abs() + TINY[torch.float32], f"{t.as_dict()}")
        assert torch.equal(pre, gu.bfloat16())


@pytest.mark.parametrize("wl,sfmt", [(0, 0), (1, 0), (1, 1)])
def test_gated_split_last_round(bfq, wl, sfmt):
    """Variant 2 (tiles in plain row order): the first 256 tiles have the sums of whole tiles, the
    others those of a split K range; a batch with too few tiles for a round, and one with none left
    over, are plain launches."""
    K = 1152
    seen = set()
    for t0 in _gated_tiles(bfq, wl, sfmt):
        if t0.variant != 0 or (t0.bm, t0.bn) in seen:
            continue
        seen.add((t0.bm, t0.bn))
        F = 128 * 34
        M = t0.bm * (-(-300 // (F // t0.bn))) - 3           # a little over a round of tiles
        tiles = -(-M // t0.bm) * (F // t0.bn)
        parts = min(256 // (tiles - 256), K // 256)
        assert 256 < tiles < 384 and parts > 1
        t = bfq.bfq_tile.from_dict({**t0.as_dict(), "variant": 2, "raster": 1, "group_m": 1})
        print("last round", wl, sfmt, M, t.as_dict(), tiles, parts, flush=True)
        n = bfq.bfq_gated_gemm_workspace_bytes(M, F, K, bfq.BFQ_BF16, wl, sfmt, t)
        assert n == (tiles - 256) * parts * t.bm * 2 * t.bn * 4
        qa, sa, qw, sw, _ = _pair(bfq, M, F, K, 300 + t.bm, sfmt, wl)
        whole, split = [_gu(bfq, qa, sa, qw, sw, bfq.bfq_tile.from_dict({**t0.as_dict(), "split_k": s}), wl, sfmt)
                        for s in (1, parts)]
        late = (torch.arange(tiles, device=DEV) >= 256).view(-1, F // t.bn)             # [tile row, tile column]
        pick = late.repeat_interleave(t.bm, 0)[:M].repeat_interleave(t.bn, 1).repeat(1, 2)
        gu = torch.where(pick, split, whole)
        h, tol = _h_ref(gu, 0)
        for odt in (torch.float32, torch.bfloat16) + ((torch.uint8,) if t.bn == 128 else ()):
            out, s, pre = _run_gated(bfq, qa, sa, qw, sw, odt, 0, t, wl, sfmt, True)
            assert torch.equal(pre, gu.bfloat16()), t.as_dict()
            if odt == torch.uint8:
                _check_codes(out, s[:, :F // 128], h, tol, sfmt == 1, f"{t.as_dict()}")
            else:
                _within(out, h, tol + H[odt] * h.abs() + TINY[odt], f"{odt} {t.as_dict()}")
        for m in (5, t.bm * 8 if t.bn == 128 else t.bm * 4):     # no whole round, one whole round
            f = F if m == 5 else 32 * 128
            qa2, sa2, qw2, sw2, _ = _pair(bfq, m, f, 384, 7, sfmt, wl)
            assert bfq.bfq_gated_gemm_workspace_bytes(m, f, 384, bfq.BFQ_BF16, wl, sfmt, t) == 0
            a = bfq.gated_gemm(qa2, sa2, qw2, sw2, tile=t, w_layout=wl, scale_fmt=sfmt)
            assert torch.equal(a, bfq.gated_gemm(qa2, sa2, qw2, sw2, tile=t0, w_layout=wl, scale_fmt=sfmt))
    assert len(seen) == 6

"""GPU tests of the gated product with an 8-bit checkpoint and of its gradient from the checkpoint.

The checkpoint's codes and scales are the token quantizer's, bit for bit. Computed values count
roundings, u = 2^-24: the activation 16 u and (GELU) 4 u |z| in the exponential, a product each for
the other factors; a value of the checkpoint is one product of code and scale. The sigmoid is the
reciprocal of 1 + exp(-z), which the hardware flushes to zero below the smallest normal number, so
products with it are off by up to 2^-126 of the other factors as well.
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U = 2.0 ** -24
BF = 2.0 ** -8
FLUSH = 2.0 ** -126


def _randn(seed, *shape):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return torch.randn(shape, generator=g, device=DEV)


def _act(g, act):
    """act(g), its slope and the sigmoid's argument, in 64 bits."""
    if act == 0:
        p = torch.sigmoid(g)
        return g * p, p * (1 + g * (1 - p)), g
    c = 2 * math.sqrt(2 / math.pi)
    z = c * (g + 0.044715 * g ** 3)
    p = torch.sigmoid(z)
    return g * p, p + g * p * (1 - p) * c * (1 + 3 * 0.044715 * g * g), z


def _close(got, ref, tol, what):
    bad = (got.double() - ref).abs() > tol
    assert not bool(bad.any()), f"{what}: {int(bad.sum())} of {bad.numel()}, worst {float(((got.double() - ref).abs() / tol).max())}"


def _check_codes(q, s, x, xtol, ue8m0, int8, what):
    """Codes with scales [M, G] of x, known to xtol."""
    M, N = x.shape
    qmax = 127.0 if int8 else 448.0
    g, t = x.view(M, N // 128, 128), xtol.view(M, N // 128, 128)
    amax, far = g.abs().amax(dim=2), t.amax(dim=2)
    lo, hi = (torch.clamp(v, min=1e-10) / qmax for v in (amax - far, amax + far))
    s = s.double()
    if ue8m0:
        assert bool((torch.frexp(s)[0] == 0.5).all()), what
        lo, hi = (torch.exp2(torch.ceil(torch.log2(v * (1 + e)))) for v, e in ((lo, -U), (hi, U)))
        assert bool(((s >= lo) & (s <= hi)).all()), what
    else:
        assert bool(((s >= lo * (1 - 2 * U)) & (s <= hi * (1 + 2 * U))).all()), what
    v = g / s.unsqueeze(2)
    got = (q.view(torch.int8) if int8 else q.view(torch.float8_e4m3fn)).double().view_as(v)
    half = torch.full_like(v, 0.5) if int8 else torch.clamp(v.abs() * 2.0 ** -4, min=2.0 ** -10)
    _close(got, v, half * (1 + 4 * U) + t / s.unsqueeze(2) + 4 * U * v.abs(), what)


def _scales(bfq, layout, M, G):
    if layout == "packed":
        t = torch.full(((G + 3) // 4, (M + 3) // 4 * 4), -1, dtype=torch.int32, device=DEV)

        def value(rows):
            b = t.view(torch.uint8).view(t.shape[0], t.shape[1], 4)
            assert not bool(b[:, M:].any())
            b = b[:, rows].permute(1, 0, 2).reshape(rows.numel(), -1)
            assert not bool(b[:, G:].any())
            return torch.exp2(b[:, :G].double() - 127)
        return t, dict(layout=bfq.BFQ_SCALES_PACKED_UE8M0, scale_fmt=bfq.BFQ_SCALE_UE8M0), value
    if layout == "row":
        t = torch.full((M, G), -77.0, device=DEV)
        return t, dict(layout=bfq.BFQ_SCALES_ROW_MAJOR), lambda rows: t[rows]
    t = torch.full((G, M + 3), -77.0, device=DEV)
    return t, dict(layout=bfq.BFQ_SCALES_COL_MAJOR, scale_fmt=bfq.BFQ_SCALE_UE8M0), lambda rows: t.t()[rows]


SHAPES = [(1, 128), (1, 2048), (7, 640), (130, 1536), (33, 2304), (3, 18432)]


@pytest.mark.parametrize("M,F", SHAPES)
@pytest.mark.parametrize("act", [0, 1])
@pytest.mark.parametrize("layout,int8", [("row", False), ("col", True), ("packed", False), ("packed", True)])
def test_checkpoint(bfq, M, F, act, layout, int8):
    pre = (_randn(F, M, 2 * F) * 2 * torch.exp(_randn(1, M, 1))).bfloat16()
    live = M - M // 3
    n = torch.tensor([live], dtype=torch.int32, device=DEV)
    rows = torch.arange(live, device=DEV)
    s, form, value = _scales(bfq, layout, M, F // 128)
    ct = torch.uint8 if int8 else torch.int8               # of the checkpoint: the other code type
    q = torch.full((M, F), 0x55, dtype=torch.int8 if int8 else torch.uint8, device=DEV)
    h = torch.full((M, F), 77.0, dtype=torch.bfloat16, device=DEV)
    ck, cs = torch.full((M, 2 * F), 0x55, dtype=ct, device=DEV), torch.full((M, 2 * F // 128), -77.0, device=DEV)
    bfq.bfq_gated_checkpoint(pre, act=act, h=h, q=q, scales=s, ckpt=ck, ckpt_scales=cs, live_rows=n, **form)
    tq, ts = bfq.quant_tokens(pre, q_dtype=bfq.BFQ_E4M3FN if int8 else bfq.BFQ_INT8)
    assert torch.equal(ck[:live], tq[:live]) and torch.equal(cs[:live], ts[:live])
    assert bool((ck[live:] == 0x55).all()) and bool((cs[live:] == -77).all())
    g, u = pre[:live].double().split(F, dim=1)
    a, _, z = _act(g, act)
    ref = a * u
    tol = ref.abs() * U * (18 + 4 * act * z.abs()) + (g * u).abs() * FLUSH + 1e-40
    _close(h[:live], ref, tol + ref.abs() * BF + 2.0 ** -133, "h")
    assert bool((h[live:] == 77).all()) and bool((q[live:] == 0x55).all())
    _check_codes(q[:live], value(rows), ref, tol, layout != "row", int8, "codes")
    if layout == "row":
        assert bool((s[live:] == -77).all())
    # without a checkpoint, and the checkpoint alone
    h2, ck2, cs2 = torch.empty_like(h[:live]), torch.empty_like(ck[:live]), torch.empty_like(cs[:live])
    bfq.bfq_gated_checkpoint(pre[:live], act=act, h=h2)
    bfq.bfq_gated_checkpoint(pre[:live], act=act, ckpt=ck2, ckpt_scales=cs2)
    assert torch.equal(h2, h[:live]) and torch.equal(ck2, ck[:live]) and torch.equal(cs2, cs[:live])


@pytest.mark.parametrize("M,F", SHAPES)
@pytest.mark.parametrize("act", [0, 1])
@pytest.mark.parametrize("layout,int8", [("row", False), ("col", True), ("packed", False), ("packed", True)])
def test_checkpoint_backward(bfq, M, F, act, layout, int8):
    pre = (_randn(F, M, 2 * F) * 2 * torch.exp(_randn(1, M, 1))).bfloat16()
    dh = (_randn(2, M, F) * 1e-2).bfloat16()
    ck, cs = bfq.quant_tokens(pre, q_dtype=bfq.BFQ_E4M3FN if int8 else bfq.BFQ_INT8)
    live = M - M // 3
    n = torch.tensor([live], dtype=torch.int32, device=DEV)
    cs[live:] = math.nan
    s, form, value = _scales(bfq, layout, M, 2 * F // 128)
    q = torch.full((M, 2 * F), 0x55, dtype=torch.int8 if int8 else torch.uint8, device=DEV)
    dpre, h = torch.full((M, 2 * F), 77.0, dtype=torch.bfloat16, device=DEV), dh.clone()
    bfq.bfq_gated_checkpoint_backward(ck, cs, h, act=act, dpre=dpre, q=q, scales=s, h=h, live_rows=n, **form)   # h is dh
    v = (ck.view(torch.float8_e4m3fn) if int8 else ck)[:live].double() * cs[:live].double().repeat_interleave(128, dim=1)
    g, u = v.split(F, dim=1)
    d = dh[:live].double()
    a, slope, z = _act(g, act)
    # a value is a rounded product of code and scale: u of it is u |z| in the exponential
    rel = U * (24 + (2 + 8 * act) * z.abs())
    # the slope's two terms may cancel: each with its own roundings, 1 - p with 4 u of p
    p = torch.sigmoid(z)
    c = 1.0 if act == 0 else 2 * math.sqrt(2 / math.pi)
    inner = 1.0 if act == 0 else 1 + 3 * 0.044715 * g * g
    smag = p + (g * p * (1 - p) * c * inner).abs() + (g * p * p * c * inner).abs() * 4 / 24
    ref = torch.cat([d * u * slope, d * a], dim=1)
    tol = torch.cat([(d * u).abs() * (smag * rel + (1 + g.abs() * c * inner) * FLUSH), (d * a).abs() * rel + (d * g).abs() * FLUSH], dim=1) + 1e-40
    _close(dpre[:live], ref, tol + ref.abs() * BF + 2.0 ** -133, "dpre")
    _close(h[:live], a * u, (a * u).abs() * (rel + BF) + (g * u).abs() * FLUSH + 2.0 ** -133, "h")
    assert bool((dpre[live:] == 77).all()) and bool((q[live:] == 0x55).all()) and torch.equal(h[live:], dh[live:])
    _check_codes(q[:live], value(torch.arange(live, device=DEV)), ref, tol, layout != "row", int8, "codes")


@pytest.mark.parametrize("act", [0, 1])
def test_backward_from_exact_checkpoint_equals_the_plain_one(bfq, act):
    """Pre-activations that their codes hold exactly: the gradient is bfq_gated_backward's."""
    M, F = 19, 512
    code = torch.randint(0, 127, (M, 2 * F), device=DEV, dtype=torch.uint8) | (torch.randint(0, 2, (M, 2 * F), device=DEV, dtype=torch.uint8) << 7)
    code[:, ::128] = 0x7E                                  # 448: every group's scale is 2^-5
    pre = (code.view(torch.float8_e4m3fn).float() * 2.0 ** -5).bfloat16()
    h0, ck, cs = bfq.gated_checkpoint(pre, act=act)
    assert torch.equal(ck & 0x7F, code & 0x7F) and bool((cs == 2.0 ** -5).all())
    dh = _randn(3, M, F).bfloat16()
    dpre, h = bfq.gated_backward(pre, dh, act=act, want_h=True)
    dpre2, h2 = bfq.gated_checkpoint_backward(ck, cs, dh, act=act, want_h=True)
    # the two kernels may place their products differently: a rounding of fp32 before that of bf16
    _close(dpre2, dpre.double(), dpre.double().abs() * 2.0 ** -7 + 1e-30, "dpre")
    _close(h2, h.double(), h.double().abs() * 2.0 ** -7 + 1e-30, "h")
    assert float((dpre2 != dpre).float().mean()) < 1e-3 and float((h2 != h).float().mean()) < 1e-3


@pytest.mark.parametrize("act", [0, 1])
def test_large_calls_equal_small_ones(bfq, act):
    """Calls that write more than the L2s hold store past them: their rows are those of a small call, bit for bit."""
    M, F = 9000, 2048
    pre = (_randn(1, M, 2 * F) * 2).bfloat16()
    dh = (_randn(2, M, F) * 1e-2).bfloat16()
    some = torch.linspace(0, M - 1, 40, device=DEV).long()
    for codes in (False, True):
        for ct in (bfq.BFQ_E4M3FN, bfq.BFQ_INT8):
            a = bfq.gated_checkpoint(pre, act=act, codes=codes, ckpt_dtype=ct)
            b = bfq.gated_checkpoint(pre[some], act=act, codes=codes, ckpt_dtype=ct)
            assert len(a) == len(b) and all(torch.equal(x[some], y) for x, y in zip(a, b))
            ga = bfq.gated_checkpoint_backward(a[-2], a[-1], dh, act=act, codes=codes, want_h=True)
            gb = bfq.gated_checkpoint_backward(b[-2], b[-1], dh[some], act=act, codes=codes, want_h=True)
            assert len(ga) == len(gb) and all(torch.equal(x[some], y) for x, y in zip(ga, gb))


def test_checkpoint_extremes(bfq):
    """Zeros, infinities, NaN, saturated gates; fewer live rows than none and more than all."""
    pre = torch.zeros((4, 512), dtype=torch.bfloat16, device=DEV)
    pre[0, 0], pre[1, 128], pre[2, 300] = math.nan, math.inf, -math.inf
    pre[3] = torch.tensor([1e30, -1e30], device=DEV).repeat(256).bfloat16()
    h, ck, cs = bfq.gated_checkpoint(pre)
    tq, ts = bfq.quant_tokens(pre)
    assert torch.equal(ck, tq) and torch.equal(cs.view(torch.int32), ts.view(torch.int32))
    g, u = pre.float().split(256, dim=1)
    ref = torch.nn.functional.silu(g) * u
    assert torch.equal(torch.isnan(h), torch.isnan(ref)) and torch.equal(torch.isinf(h), torch.isinf(ref.bfloat16()))
    dpre = bfq.gated_checkpoint_backward(ck, cs, torch.ones((4, 256), dtype=torch.bfloat16, device=DEV))
    assert bool(torch.isnan(dpre[0, :128]).all()) and not bool(torch.isnan(dpre[3]).any())
    for n, rows in ((-3, 0), (0, 0), (99, 4)):
        out = torch.full((4, 256), 77.0, dtype=torch.bfloat16, device=DEV)
        bfq.bfq_gated_checkpoint(pre, h=out, live_rows=torch.tensor([n], dtype=torch.int32, device=DEV))
        assert bool((out[rows:] == 77).all()) and (rows == 0 or torch.equal(out.view(torch.int16), h.view(torch.int16)))


def test_gradient_against_differences(bfq):
    """Central differences of act(g) u in 64 bits at the checkpoint's values."""
    M, F, e = 6, 128, 2.0 ** -8
    pre = _randn(1, M, 2 * F).bfloat16()
    for act in (0, 1):
        ck, cs = bfq.quant_tokens(pre, q_dtype=bfq.BFQ_INT8)
        dh = _randn(2, M, F).bfloat16()
        d = bfq.gated_checkpoint_backward(ck, cs, dh, act=act).double()
        v = ck.double() * cs.double().repeat_interleave(128, dim=1)
        g, u = v.split(F, dim=1)
        dg = (_act(g + e, act)[0] - _act(g - e, act)[0]) / (2 * e) * u * dh.double()
        # the activations' third derivatives stay below 3: e^2 / 2 of the factors; bf16 out
        tol = (u * dh.double()).abs() * e * e / 2 + dg.abs() * BF + 1e-6
        _close(d[:, :F], dg, tol, "dg")
        du = _act(g, act)[0] * dh.double()
        _close(d[:, F:], du, du.abs() * (BF + 64 * U) + 1e-30, "du")


def test_empty(bfq):
    pre = torch.empty((0, 512), dtype=torch.bfloat16, device=DEV)
    h, ck, cs = bfq.gated_checkpoint(pre)
    assert h.shape == (0, 256) and bfq.gated_checkpoint_backward(ck, cs, h).shape == (0, 512)

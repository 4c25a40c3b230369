"""GPU tests of the dispatch and the combine of expert rows and of the combine's gradient.

Codes of values that fp32 holds exactly (bf16 rows, products of one rounding) are compared bit for bit
with the quantizer's definition. Sums count roundings, u = 2^-24: a combine adds topk products to its
base in order; a weight's gradient adds eight products in a lane, one more sum a round of 512 threads,
6 over the wave and 8 over the waves.
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U = 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
TINY = {torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -149}
LAYOUTS = ("row", "col", "padded", "packed")


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _randn(seed, *shape):
    return torch.randn(shape, generator=_gen(seed), device=DEV)


def _bits(t):
    return t.contiguous().view({1: torch.uint8, 2: torch.int16, 4: torch.int32}[t.element_size()])


def _quant(z, ue8m0, int8):
    """The quantizer's definition on fp32 z [M, K]: codes (as bytes) and scales [M, K/128]."""
    M, K = z.shape
    qmax = 127.0 if int8 else 448.0
    g = z.view(M, K // 128, 128)
    amax = g.abs().amax(dim=2)
    # torch divides by a constant as a product with its reciprocal: a tensor makes it a quotient
    s = torch.clamp(amax, min=1e-10) / torch.full_like(amax, qmax)
    if ue8m0:
        m, e = torch.frexp(s)
        s = torch.ldexp(torch.ones_like(s), torch.where(m == 0.5, e - 1, e))
    v = g / s.unsqueeze(2)
    if int8:
        q = torch.clamp(torch.round(v), -127, 127).to(torch.int8)
    else:
        q = v.to(torch.float8_e4m3fn)
    return q.view(M, K).view(torch.uint8), s


def _places(T, topk, R, drop, seed):
    """Distinct rows for the pairs, some of which have none."""
    perm = torch.randperm(R, generator=_gen(seed), device=DEV)[: T * topk].int().view(T, topk)
    if drop:
        out = torch.rand((T, topk), generator=_gen(seed + 1), device=DEV) < 0.4
        bad = torch.tensor([-1, R, -2 ** 31, 2 ** 31 - 1], device=DEV, dtype=torch.int32)
        perm = torch.where(out, bad[torch.arange(T * topk, device=DEV) % 4].view(T, topk), perm)
        perm[0] = -1                                       # a token without any
    return perm


def _scale_buffer(bfq, layout, R, G):
    """(tensor of a marker, keyword arguments, function to [R, G] fp32)."""
    if layout == "packed":
        t = torch.full(((G + 3) // 4, (R + 3) // 4 * 4 + 4), 0x0BADBEEF, dtype=torch.int32, device=DEV)
        ld = t.shape[1]

        def value(rows):
            b = t.view(torch.uint8).view(t.shape[0], ld, 4)[:, rows].permute(1, 0, 2).reshape(rows.numel(), -1)
            assert not bool(b[:, G:].any()), "bytes past the last group"
            return torch.exp2(b[:, :G].double() - 127).float()
        return t, dict(layout=bfq.BFQ_SCALES_PACKED_UE8M0, scale_fmt=bfq.BFQ_SCALE_UE8M0, scale_ld=ld), value
    if layout == "row":
        t = torch.full((R, G), -77.0, device=DEV)
        return t, dict(layout=bfq.BFQ_SCALES_ROW_MAJOR), lambda rows: t[rows]
    t = torch.full((G, R + (5 if layout == "padded" else 0)), -77.0, device=DEV)
    return t, dict(layout=bfq.BFQ_SCALES_COL_MAJOR), lambda rows: t[:, :R].t()[rows]


def _untouched(t, rows, R, layout):
    """Scales of rows that no pair has are as they were (packed: zero words past the last row)."""
    keep = torch.ones(R, dtype=torch.bool, device=DEV)
    keep[rows] = False
    if layout == "packed":
        assert bool((t[:, :R][:, keep] == 0x0BADBEEF).all())
        r4 = (R + 3) // 4 * 4
        assert not bool(t[:, R:r4].any()) and bool((t[:, r4:] == 0x0BADBEEF).all())
    elif layout == "row":
        assert bool((t[keep] == -77.0).all())
    else:
        assert bool((t[:, :R][:, keep] == -77.0).all()) and bool((t[:, R:] == -77.0).all())


# --------------------------------------------------------------------------- dispatch

@pytest.mark.parametrize("T,topk,K", [(1, 1, 8), (1, 8, 7168), (5, 3, 1544), (130, 6, 264), (33, 64, 2056), (700, 2, 4096)])
@pytest.mark.parametrize("drop", [False, True])
def test_dispatch_rows(bfq, T, topk, K, drop):
    R = T * topk + 3
    x = _randn(K, T, K).bfloat16()
    at = _places(T, topk, R, drop, T)
    rows = torch.full((R, K), 77.0, dtype=torch.bfloat16, device=DEV)
    bfq.bfq_moe_dispatch(x, at, rows=rows)
    want = torch.full_like(rows, 77.0)
    live = (at >= 0) & (at < R)
    want[at[live].long()] = x[torch.nonzero(live)[:, 0]]
    assert torch.equal(_bits(rows), _bits(want))


@pytest.mark.parametrize("T,topk,K", [(1, 1, 128), (1, 8, 7168), (7, 5, 640), (130, 3, 2048), (9, 64, 512), (50, 33, 1152), (6, 2, 16384)])
@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("int8", [False, True])
def test_dispatch_codes(bfq, T, topk, K, layout, int8):
    """From bf16 rows, and copies of codes: what the quantizer writes for the same rows."""
    R, G, ue = T * topk + 2, K // 128, layout in ("packed", "padded")
    x = (_randn(K + T, T, K) * torch.exp(_randn(3, T, 1))).bfloat16()
    at = _places(T, topk, R, T > 1, T + 1)
    fmt = bfq.BFQ_SCALE_UE8M0 if ue else bfq.BFQ_SCALE_FP32
    qd = bfq.BFQ_INT8 if int8 else bfq.BFQ_E4M3FN
    pl = bfq.BFQ_SCALES_PACKED_UE8M0 if layout == "packed" else bfq.BFQ_SCALES_COL_MAJOR
    xq, xs = bfq.quant_tokens(x, q_dtype=qd, scale_fmt=fmt, layout=pl)
    live = (at >= 0) & (at < R)
    rows, tok = at[live].long(), torch.nonzero(live)[:, 0]
    tq, ts = bfq.quant_tokens(x, q_dtype=qd, scale_fmt=fmt)
    for copy in (False, True):
        s, form, value = _scale_buffer(bfq, layout, R, G)
        form.setdefault("scale_fmt", fmt)
        q = torch.full((R, K), 0x55, dtype=xq.dtype, device=DEV)
        both = torch.full((R, K), 77.0, dtype=torch.bfloat16, device=DEV)
        if copy:
            bfq.bfq_moe_dispatch(xq, at, q=q, scales=s, x_scales=xs, x_layout=pl, **form)
        else:
            bfq.bfq_moe_dispatch(x, at, q=q, scales=s, rows=both, **form)
            want = torch.full_like(both, 77.0)
            want[rows] = x[tok]
            assert torch.equal(_bits(both), _bits(want))
        want = torch.full_like(q, 0x55)
        want[rows] = tq[tok]
        assert torch.equal(q, want)
        assert torch.equal(value(rows), ts[tok])
        _untouched(s, rows, R, layout)


def test_dispatch_special_groups(bfq):
    """Groups with a NaN or an infinity: the quantizer's codes and scales, NaN scales copied bit for bit."""
    x = _randn(1, 4, 512).bfloat16()
    x[0, 5], x[1, 130], x[2, 300], x[3] = math.nan, math.inf, -math.inf, 0.0
    at = torch.tensor([[3], [1], [0], [2]], dtype=torch.int32, device=DEV)
    tq, ts = bfq.quant_tokens(x)
    for kw in (dict(x=x, codes=True), dict(x=tq, x_scales=ts)):
        q, s = bfq.moe_dispatch(pair_rows=at, **kw)
        assert torch.equal(q[at[:, 0].long()], tq) and torch.equal(_bits(s[at[:, 0].long()]), _bits(ts))


def test_dispatch_past_32_bit_offsets(bfq):
    """Rows whose byte and element offsets pass 2^32."""
    K, R, T = 8192, 600_000, 4                             # 9.8 GB of bf16, 4.9 GB of codes
    x = _randn(1, T, K).bfloat16()
    at = torch.tensor([[R - 1, 0], [R // 2, 7], [262_144, 524_288], [R - 2, 262_143]], dtype=torch.int32, device=DEV)
    rows = torch.empty((R, K), dtype=torch.bfloat16, device=DEV)
    bfq.bfq_moe_dispatch(x, at, rows=rows)
    tq, ts = bfq.quant_tokens(x)
    q = torch.empty((R, K), dtype=torch.uint8, device=DEV)
    s = torch.empty((R, K // 128), device=DEV)
    bfq.bfq_moe_dispatch(x, at, q=q, scales=s)
    for j in range(2):
        r = at[:, j].long()
        assert torch.equal(_bits(rows[r]), _bits(x)) and torch.equal(q[r], tq) and torch.equal(s[r], ts)
    w = torch.rand((T, 2), generator=_gen(2), device=DEV)
    out = bfq.moe_combine(rows, 2, weights=w, pair_rows=at)
    ref = (x.double() * w.double().sum(dim=1, keepdim=True))
    assert bool(((out.double() - ref).abs() <= ref.abs() * (2.0 ** -8 + 4 * U)).all())
    g = bfq.moe_combine_backward(x, 2, weights=w, rows=q, rows_scales=s, pair_rows=at)
    assert torch.equal(_bits(g["d_rows"][at[:, 0].long()]), _bits((x.float() * w[:, :1]).bfloat16()))


# ---------------------------------------------------------------------------- combine

def _combine_inputs(T, topk, K, order, rt, drop, seed):
    R = T * topk if order == "pair" else T * topk + 3
    rows = _randn(seed, R, K) * torch.exp(0.5 * _randn(seed + 1, R, 1))
    E = 16
    if order == "expert":
        at = _places(T, topk, R, drop, seed)
        live = (at >= 0) & (at < R)
        kw = dict(pair_rows=at)
    else:
        ids = torch.randint(-8 if drop else 0, 24 if drop else E, (T, topk), generator=_gen(seed + 2), device=DEV, dtype=torch.int32)
        at = torch.arange(T * topk, device=DEV, dtype=torch.int32).view(T, topk)
        live = (ids >= 0) & (ids < E)
        kw = dict(topk_ids=ids, E=E) if drop else {}
    used = torch.zeros(R, dtype=torch.bool, device=DEV)
    used[at[live].long()] = True
    rows[~used] = math.nan                                 # rows that nothing wrote
    w = torch.rand((T, topk), generator=_gen(seed + 3), device=DEV) - 0.2
    w[~live] = math.nan
    return rows.to(rt), w, torch.where(live, at, 0).long(), live, used, kw


SHAPES = [(1, 1, 8), (1, 8, 7168), (3, 2, 1544), (130, 6, 264), (17, 64, 520), (65, 9, 2048), (2, 33, 4104)]


@pytest.mark.parametrize("T,topk,K", SHAPES)
@pytest.mark.parametrize("order,drop", [("pair", False), ("pair", True), ("expert", True)])
@pytest.mark.parametrize("rt,ot", [(torch.bfloat16, torch.bfloat16), (torch.bfloat16, torch.float32), (torch.float32, torch.float16),
                                   (torch.float16, torch.bfloat16), (torch.float32, torch.float32)])
def test_combine(bfq, T, topk, K, order, drop, rt, ot):
    rows, w, at, live, used, kw = _combine_inputs(T, topk, K, order, rt, drop, K + T)
    for weights in (None, w):
        for based in (False, True):
            base = _randn(9, T, K).to(ot) if based else None
            out = torch.full((T + 2, K), 77.0, dtype=ot, device=DEV)
            if based:
                out[1:-1] = base                           # in place
            bfq.bfq_moe_combine(rows, out[1:-1], topk, weights=weights, base=out[1:-1] if based else None, **kw)
            x = torch.where(live.unsqueeze(2), rows[at].double(), 0.0)
            terms = x if weights is None else x * torch.where(live, w, 0.0).double().unsqueeze(2)
            ref, mag = terms.sum(dim=1), terms.abs().sum(dim=1)
            if based:
                ref, mag = ref + base.double(), mag + base.double().abs()
            tol = mag * U * (topk + 1) + ref.abs() * HALF[ot] * (1 + 2 ** -8) + TINY[ot]
            assert bool(((out[1:-1].double() - ref).abs() <= tol).all())
            assert bool((out[0] == 77).all()) and bool((out[-1] == 77).all())
            if not bool(live.any(dim=1).all()):
                gone = ~live.any(dim=1)
                assert torch.equal(out[1:-1][gone], base[gone] if based else torch.zeros_like(out[1:-1][gone]))


@pytest.mark.parametrize("T,topk,K", [(1, 1, 128), (1, 8, 7168), (7, 3, 640), (40, 12, 2048)])
@pytest.mark.parametrize("order", ["pair", "expert"])
@pytest.mark.parametrize("rt", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("int8", [False, True])
def test_combine_checkpoint(bfq, T, topk, K, order, rt, int8):
    rows, w, at, live, used, kw = _combine_inputs(T, topk, K, order, rt, True, K + 5)
    R = rows.shape[0]
    out = torch.empty((T, K), dtype=torch.bfloat16, device=DEV)
    q = torch.full((R, K), 0x55, dtype=torch.int8 if int8 else torch.uint8, device=DEV)
    s = torch.full((R, K // 128), -77.0, device=DEV)
    bfq.bfq_moe_combine(rows, out, topk, weights=w, ckpt=q, ckpt_scales=s, **kw)
    rq, rs = _quant(rows.float(), False, int8)
    assert torch.equal(q[used].view(torch.uint8), rq[used]) and torch.equal(s[used], rs[used])
    assert bool((q[~used] == 0x55).all()) and bool((s[~used] == -77.0).all())
    if rt == torch.bfloat16:
        tq, ts = bfq.quant_tokens(rows, q_dtype=bfq.BFQ_INT8 if int8 else bfq.BFQ_E4M3FN)
        assert torch.equal(q[used], tq[used]) and torch.equal(s[used], ts[used])
    plain = torch.empty_like(out)
    bfq.bfq_moe_combine(rows, plain, topk, weights=w, **kw)
    assert torch.equal(_bits(out), _bits(plain))


def test_combine_nan_and_inf_of_live_rows_reach_the_output(bfq):
    rows = _randn(1, 6, 256).bfloat16()
    rows[1, 3], rows[4, 9] = math.nan, math.inf
    w = torch.ones((3, 2), device=DEV)
    out, q, s = bfq.moe_combine(rows, 2, weights=w, ckpt_dtype=bfq.BFQ_E4M3FN)
    assert bool(torch.isnan(out[0, 3])) and int(torch.isnan(out).sum()) == 1 and bool(torch.isinf(out[2, 9]))
    tq, ts = bfq.quant_tokens(rows)
    assert torch.equal(q, tq) and torch.equal(_bits(s), _bits(ts))
    w[0, 1] = math.inf                                     # a weight of a live row too
    assert not bool(torch.isfinite(bfq.moe_combine(rows, 2, weights=w)[0]).any())


# ------------------------------------------------------------------- combine's gradient

@pytest.mark.parametrize("T,topk,K", SHAPES + [(3, 10, 12288)])
@pytest.mark.parametrize("order,drop", [("pair", False), ("pair", True), ("expert", True)])
@pytest.mark.parametrize("kind", ["none", "bf16", "fp16", "fp32"])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_combine_backward(bfq, T, topk, K, order, drop, kind, dt):
    rt = {"fp16": torch.float16, "fp32": torch.float32}.get(kind, torch.bfloat16)
    rows, w, at, live, used, kw = _combine_inputs(T, topk, K, order, rt, drop, K + 7)
    d = (_randn(8, T, K) * 0.1).to(dt)
    R = rows.shape[0]
    dr = torch.full((R + 2, K), 77.0, dtype=torch.bfloat16, device=DEV)
    dw = torch.full((T, topk), 77.0, device=DEV)
    if kind == "none":
        bfq.bfq_moe_combine_backward(d, topk, weights=w, d_rows=dr[1:-1], **kw)
    else:
        bfq.bfq_moe_combine_backward(d, topk, weights=w, rows=rows, d_rows=dr[1:-1], d_weights=dw, **kw)
        terms = torch.where(live.unsqueeze(2), rows[at].double(), 0.0) * d.double().unsqueeze(1)
        tol = terms.abs().sum(dim=2) * U * (24 + (K + 4095) // 4096) + 1e-40
        assert bool(((dw.double() - terms.sum(dim=2)).abs() <= tol).all())
        assert not bool(dw[~live].any())
    want = torch.full((R, K), 77.0, dtype=torch.bfloat16, device=DEV)
    want[at[live]] = (w.unsqueeze(2) * d.float().unsqueeze(1))[live].bfloat16()      # one product, one rounding
    assert torch.equal(_bits(dr[1:-1]), _bits(want))
    assert bool((dr[0] == 77).all()) and bool((dr[-1] == 77).all())


@pytest.mark.parametrize("T,topk,K", [(1, 1, 128), (2, 8, 7168), (7, 3, 640), (40, 12, 2048), (9, 64, 4224)])
@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_combine_backward_codes(bfq, T, topk, K, layout, int8, dt):
    """Codes of the products, rows as codes."""
    rows, w, at, live, used, kw = _combine_inputs(T, topk, K, "expert", torch.float32, T > 1, K + 11)
    R, G, ue = rows.shape[0], K // 128, layout in ("packed", "padded")
    rq, rs = _quant(torch.nan_to_num(rows), False, int8)
    rs[~used] = math.nan
    d = (_randn(8, T, K) * 0.1).to(dt)
    s, form, value = _scale_buffer(bfq, layout, R, G)
    form.setdefault("scale_fmt", bfq.BFQ_SCALE_UE8M0 if ue else bfq.BFQ_SCALE_FP32)
    q = torch.full((R, K), 0x55, dtype=torch.int8 if int8 else torch.uint8, device=DEV)
    dw = torch.empty((T, topk), device=DEV)
    codes = rq.view(torch.int8) if int8 else rq
    bfq.bfq_moe_combine_backward(d, topk, weights=w, rows=codes, rows_scales=rs, q=q, scales=s, d_weights=dw, **kw, **form)
    z = (w.unsqueeze(2) * d.float().unsqueeze(1))[live]
    zq, zs = _quant(z, ue, int8)
    assert torch.equal(q[at[live]].view(torch.uint8), zq)
    assert torch.equal(value(at[live]), zs)
    assert bool((q[~used] == 0x55).all())
    _untouched(s, at[live], R, layout)
    v = (codes.double() if int8 else rq.view(torch.float8_e4m3fn).double()) * torch.where(used.unsqueeze(1), rs, 0.0).double().repeat_interleave(128, dim=1)
    terms = torch.where(live.unsqueeze(2), v[at], 0.0) * d.double().unsqueeze(1)
    tol = terms.abs().sum(dim=2) * U * (26 + (K + 4095) // 4096) + 1e-40
    assert bool(((dw.double() - terms.sum(dim=2)).abs() <= tol).all())


def test_combine_backward_special_values(bfq):
    """Gradients and weights that are infinite, NaN or zero: the codes of the products themselves."""
    d = _randn(1, 5, 256)
    d[0, 3], d[1, 200], d[2] = math.nan, math.inf, 0.0
    w = torch.tensor([[1.0], [0.0], [math.inf], [math.nan], [3e38]], device=DEV)
    d[4, 0] = 1e3                                          # overflows in the product
    g = bfq.moe_combine_backward(d, 1, weights=w, codes=True)
    z = w * d
    amax = z.view(5, 2, 128).abs().amax(dim=2)
    nan = torch.isnan(z.view(5, 2, 128)).any(dim=2)
    assert torch.equal(torch.isnan(g["scales"]), nan)
    assert torch.equal(torch.isinf(g["scales"]), torch.isinf(amax) & ~nan)
    ok = ~nan & ~torch.isinf(amax)
    zq, zs = _quant(z, False, False)
    same = ok.repeat_interleave(128, dim=1)
    assert torch.equal(g["q"][same], zq[same]) and torch.equal(g["scales"][ok], zs[ok])
    assert bool((g["q"][nan.repeat_interleave(128, dim=1)] == 0x7F).all())


def test_combine_gradient_against_differences(bfq):
    """The combine is linear in its rows and its weights: differences of fp32 calls are its gradient."""
    T, topk, K = 5, 3, 136
    rows, w, at, live, used, kw = _combine_inputs(T, topk, K, "expert", torch.float32, True, 21)
    d = _randn(3, T, K)
    g = bfq.moe_combine_backward(d, topk, weights=w, rows=rows, **kw)
    run = lambda r, ww: (bfq.moe_combine(r, topk, weights=ww, out_dtype=torch.float32, **kw).double() * d.double()).sum()  # noqa: E731
    y0 = run(rows, w)
    for t, j in ((0, 0), (1, 2), (2, 1), (4, 0)):
        w2 = w.clone()
        w2[t, j] += 1.0
        if bool(live[t, j]):
            # fp32 outputs: (topk + 1) u of the magnitudes, summed over K, twice
            tol = 2 * 2 * (topk + 1) * U * K * 8 * float(rows[at[t]].nan_to_num().abs().max()) * float(d.abs().max())
            assert abs(float(run(rows, w2) - y0) - float(g["d_weights"][t, j])) <= tol
            r2 = rows.clone()
            r2[at[t, j], 7] += 1.0
            want = float(g["d_rows"][at[t, j], 7])
            assert abs(float(run(r2, w) - y0) - want) <= tol + 2.0 ** -8 * abs(want)
        else:
            assert float(run(rows, w2.nan_to_num()) - y0) == 0.0 and float(g["d_weights"][t, j]) == 0.0


def test_dispatch_and_combine_are_transposes(bfq):
    """<dispatch(x), g> = <x, combine(g) without weights>, in numbers whose sums are exact."""
    T, topk, K = 37, 5, 520
    ids = torch.randint(-4, 12, (T, topk), generator=_gen(1), device=DEV, dtype=torch.int32)
    off, _, at = bfq.moe_sort(ids, 8)
    n = int(off[8])
    x = torch.randint(-8, 9, (T, K), generator=_gen(2), device=DEV).bfloat16()
    g = torch.randint(-8, 9, (T * topk, K), generator=_gen(3), device=DEV).bfloat16()
    g[n:] = math.nan
    rows = torch.zeros((T * topk, K), dtype=torch.bfloat16, device=DEV)
    bfq.bfq_moe_dispatch(x, at, rows=rows)
    dx = bfq.moe_combine(g, topk, pair_rows=at, out_dtype=torch.float32)
    assert float((rows[:n].double() * g[:n].double()).sum()) == float((x.double() * dx.double()).sum())


@pytest.mark.parametrize("T,topk,K", [(1100, 8, 4096), (5000, 2, 4096), (1030, 64, 640)])
def test_large_calls_equal_small_ones(bfq, T, topk, K):
    """Calls that write more than the L2s hold store past them and take more pairs at a time: the rows of a few
    tokens are those of a call of their own, bit for bit."""
    R, G = T * topk, K // 128
    assert R * K > 32 << 20
    ids = torch.randint(-8, 24, (T, topk), generator=_gen(1), device=DEV, dtype=torch.int32)
    _, _, at = bfq.moe_sort(ids, 16)
    some = torch.tensor([0, 1, T // 2, T - 2, T - 1], device=DEV)
    live = at[some] >= 0
    rows_of = at[some][live].long()
    # the same pairs in a call of five tokens: their rows in a small tensor
    few = torch.where(live, torch.arange(5 * topk, device=DEV, dtype=torch.int32).view(5, topk), -1).int()
    few_rows = few[live].long()
    x = _randn(2, T, K).bfloat16()
    w = torch.rand((T, topk), generator=_gen(3), device=DEV)

    def small(big):
        t = torch.zeros((5 * topk, *big.shape[1:]), dtype=big.dtype, device=DEV)
        t[few_rows] = big[rows_of]
        return t

    def same(a, b, what):
        assert torch.equal(_bits(a), _bits(b)), what

    rows, rq, rs = torch.zeros((R, K), dtype=torch.bfloat16, device=DEV), torch.zeros((R, K), dtype=torch.uint8, device=DEV), torch.zeros((R, G), device=DEV)
    bfq.bfq_moe_dispatch(x, at, rows=rows)
    same(rows[rows_of], bfq.moe_dispatch(x[some], few)[few_rows], "dispatch")
    bfq.bfq_moe_dispatch(x, at, rows=rows, q=rq, scales=rs)
    q2, s2 = bfq.moe_dispatch(x[some], few, codes=True)
    same(rq[rows_of], q2[few_rows], "codes")
    same(rs[rows_of], s2[few_rows], "scales")
    same(rows[rows_of], bfq.moe_dispatch(x[some], few)[few_rows], "rows beside codes")
    xq, xs = bfq.quant_tokens(x)
    cq = torch.zeros_like(rq)
    bfq.bfq_moe_dispatch(xq, at, q=cq, scales=torch.zeros_like(rs), x_scales=xs)
    same(cq, rq, "copied codes")
    wide = rows.float() if R * K < 40 << 20 else None
    for r in (rows,) if wide is None else (rows, wide):
        for ct in (None, bfq.BFQ_E4M3FN, bfq.BFQ_INT8):
            a = bfq.moe_combine(r, topk, weights=w, pair_rows=at, base=x, ckpt_dtype=ct)
            b = bfq.moe_combine(small(r), topk, weights=w[some], pair_rows=few, base=x[some], ckpt_dtype=ct)
            a, b = ((a,), (b,)) if ct is None else (a, b)
            same(a[0][some], b[0], "combine")
            for u, v in zip(a[1:], b[1:]):
                same(u[rows_of], v[few_rows], "checkpoint")
    for kw, kws in ((dict(rows=rows), dict(rows=small(rows))), (dict(rows=rq, rows_scales=rs), dict(rows=small(rq), rows_scales=small(rs)))):
        for codes in (False, True):
            a = bfq.moe_combine_backward(x, topk, weights=w, pair_rows=at, codes=codes, **kw)
            b = bfq.moe_combine_backward(x[some], topk, weights=w[some], pair_rows=few, codes=codes, **kws)
            same(a["d_weights"][some], b["d_weights"], "d_weights")
            for k in set(a) - {"d_weights"}:
                same(a[k][rows_of], b[k][few_rows], k)


@pytest.mark.parametrize("T", [9, 1300])
@pytest.mark.parametrize("kind", ["bf16", "codes", "none"])
def test_gradient_as_rows_and_codes_at_once(bfq, T, kind):
    topk, K = 5, 640
    rows, w, at, live, used, kw = _combine_inputs(T, topk, K, "expert", torch.bfloat16, True, 31)
    d = _randn(8, T, K).bfloat16()
    R = rows.shape[0]
    more = {}
    if kind != "none":
        more = dict(rows=rows, d_weights=torch.empty((T, topk), device=DEV))
    if kind == "codes":
        q, s = bfq.quant_tokens(torch.nan_to_num(rows))
        more.update(rows=q, rows_scales=s)
    dr, q, s = torch.zeros((R, K), dtype=torch.bfloat16, device=DEV), torch.zeros((R, K), dtype=torch.uint8, device=DEV), torch.zeros((R, K // 128), device=DEV)
    bfq.bfq_moe_combine_backward(d, topk, weights=w, d_rows=dr, q=q, scales=s, **kw, **more)
    z = (w.unsqueeze(2) * d.float().unsqueeze(1))[live]
    zq, zs = _quant(z, False, False)
    assert torch.equal(_bits(dr[at[live]]), _bits(z.bfloat16())) and torch.equal(q[at[live]], zq) and torch.equal(s[at[live]], zs)
    assert not bool(dr[~used].any()) and not bool(q[~used].any()) and not bool(s[~used].any())


@pytest.mark.parametrize("kind", ["none", "bf16", "codes"])
@pytest.mark.parametrize("topk", [3, 6, 9])
def test_gradients_do_not_depend_on_the_tokens_beside(bfq, kind, topk):
    """Calls of few and of many pairs take two, four or eight of a token's at a time, some batches short: a
    token's gradients are the same bits in each."""
    T, K, G = 4100, 256, 2
    w = torch.rand((T, topk), generator=_gen(1), device=DEV) - 0.3
    d = _randn(2, T, K)
    at = _places(T, topk, T * topk, True, 3)
    rows = _randn(4, T * topk, K).bfloat16()
    kw = {} if kind == "none" else dict(rows=rows) if kind == "bf16" else dict(zip(("rows", "rows_scales"), bfq.quant_tokens(rows)))

    def run(n, codes):
        dw = torch.full((n, topk), 7.0, device=DEV) if kw else None
        q, s = torch.full((T * topk, K), 9, dtype=torch.uint8, device=DEV), torch.full((T * topk, G), 9.0, device=DEV)
        dr = torch.full((T * topk, K), 9.0, dtype=torch.bfloat16, device=DEV)
        form = dict(q=q, scales=s) if codes else dict(d_rows=dr)
        bfq.bfq_moe_combine_backward(d[:n], topk, weights=w[:n].contiguous(), pair_rows=at[:n].contiguous(), d_weights=dw, **form, **kw)
        return dw, (q, s) if codes else (dr,)

    for codes in (False, True):
        dw, full = run(T, codes)
        for n in (1, 100, 1300, 2900):
            dn, part = run(n, codes)
            live = at[:n][(at[:n] >= 0) & (at[:n] < T * topk)].long()
            assert dw is None or torch.equal(_bits(dn), _bits(dw[:n]))
            for a, b in zip(part, full):
                assert torch.equal(_bits(a[live]), _bits(b[live]))
                a[live] = 9
                assert bool((a.float() == 9).all())


def test_scale_floor(bfq):
    """q_eps floors every scale that is written."""
    x = (_randn(1, 6, 256) * 0.01).bfloat16()
    at = torch.arange(6, device=DEV, dtype=torch.int32).view(6, 1)
    tq, ts = torch.empty((6, 256), dtype=torch.uint8, device=DEV), torch.empty((6, 2), device=DEV)
    bfq.bfq_quant_tokens(x, tq, ts, eps=0.5)
    assert bool((ts == 0.5 / torch.full_like(ts, 448.0)).all())
    out = torch.empty_like(x)
    for call in (lambda q, s: bfq.bfq_moe_dispatch(x, at, q=q, scales=s, q_eps=0.5),
                 lambda q, s: bfq.bfq_moe_combine(x, out, 1, ckpt=q, ckpt_scales=s, q_eps=0.5),
                 lambda q, s: bfq.bfq_moe_combine_backward(x, 1, q=q, scales=s, q_eps=0.5),
                 lambda q, s: bfq.bfq_gated_checkpoint(x, ckpt=q, ckpt_scales=s, q_eps=0.5)):
        q, s = torch.zeros_like(tq), torch.zeros_like(ts)
        call(q, s)
        assert torch.equal(q, tq) and torch.equal(s, ts)


def test_pairs_that_share_a_row(bfq):
    """Reading, a row may be several pairs'; a token may name one twice."""
    T, topk, K, R = 40, 4, 264, 5
    rows = _randn(1, R, K).bfloat16()
    at = torch.randint(0, R, (T, topk), generator=_gen(2), device=DEV, dtype=torch.int32)
    at[3] = 2
    w = torch.rand((T, topk), generator=_gen(3), device=DEV)
    out = bfq.moe_combine(rows, topk, weights=w, pair_rows=at)
    terms = rows[at.long()].double() * w.double().unsqueeze(2)
    tol = terms.abs().sum(dim=1) * U * (topk + 1) + terms.sum(dim=1).abs() * HALF[torch.bfloat16]
    assert bool(((out.double() - terms.sum(dim=1)).abs() <= tol).all())
    d = _randn(4, T, K).bfloat16()
    dw = torch.empty((T, topk), device=DEV)
    bfq.bfq_moe_combine_backward(d, topk, rows=rows, pair_rows=at, d_weights=dw)         # the weights' alone
    terms = rows[at.long()].double() * d.double().unsqueeze(1)
    assert bool(((dw.double() - terms.sum(dim=2)).abs() <= terms.abs().sum(dim=2) * U * 25).all())


def test_no_rows(bfq):
    """R = 0: the base or zeros come back, the weights have no gradient, nothing else happens."""
    T, topk, K = 5, 3, 256
    x, at = _randn(1, T, K).bfloat16(), torch.randint(-2, 3, (T, topk), generator=_gen(2), device=DEV, dtype=torch.int32)
    none, w = torch.empty((0, K), dtype=torch.bfloat16, device=DEV), torch.full((T, topk), math.nan, device=DEV)
    assert bfq.moe_dispatch(x, at, R=0).shape == (0, K) and bfq.moe_dispatch(x, at, R=0, codes=True)[0].shape == (0, K)
    assert torch.equal(bfq.moe_combine(none, topk, weights=w, pair_rows=at, base=x), x)
    out, q, s = bfq.moe_combine(none, topk, weights=w, pair_rows=at, ckpt_dtype=bfq.BFQ_E4M3FN)
    assert not bool(out.any()) and q.numel() == 0
    for codes in (False, True):
        assert not bool(bfq.moe_combine_backward(x, topk, weights=w, rows=none, pair_rows=at, codes=codes)["d_weights"].any())
    scales = torch.empty((0, K // 128), device=DEV)
    assert not bool(bfq.moe_combine_backward(x, topk, rows=none.view(torch.uint8)[:, :K].contiguous(), rows_scales=scales,
                                             pair_rows=at)["d_weights"].any())


def test_empty_batches(bfq):
    for T in (0,):
        x, at = torch.empty((T, 256), dtype=torch.bfloat16, device=DEV), torch.empty((T, 2), dtype=torch.int32, device=DEV)
        assert bfq.moe_dispatch(x, at).shape == (0, 256)
        assert bfq.moe_dispatch(x, at, codes=True)[1].shape == (0, 2)
        assert bfq.moe_combine(x, 2, pair_rows=at).shape == (0, 256)
        assert bfq.moe_combine_backward(x, 2, rows=x, pair_rows=at)["d_weights"].shape == (0, 2)

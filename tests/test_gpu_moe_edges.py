"""GPU tests of the mixture-of-experts operators where rows are narrow or end inside a wave, batches empty,
experts many: calls that the documentation allows and that are seldom made."""
import math

import pytest
import torch

import test_gpu_moe_route as route

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U = 2.0 ** -24


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _randn(seed, *shape):
    return torch.randn(shape, generator=_gen(seed), device=DEV)


def _codes(z):
    """e4m3 codes (bytes) and scales of fp32 z [M, K], the quantizer's definition."""
    M, K = z.shape
    g = z.view(M, K // 128, 128)
    amax = g.abs().amax(dim=2)
    s = torch.clamp(amax, min=1e-10) / torch.full_like(amax, 448.0)       # a quotient: by a number torch multiplies
    return (g / s.unsqueeze(2)).to(torch.float8_e4m3fn).view(M, K).view(torch.uint8), s


@pytest.mark.parametrize("T,topk,K", [(5, 64, 8), (3, 2, 8), (9, 64, 72), (60, 61, 128), (400, 64, 128), (7, 64, 2056),
                                      (5, 33, 4224), (70, 64, 640)])
@pytest.mark.parametrize("kind", ["none", "bf16", "codes"])
def test_weights_of_lanes_past_the_row(bfq, T, topk, K, kind):
    """A pair's weight lies in a lane that may have no column of the row: rows shorter than a wave, last rounds
    of a few lanes, in batches of two, four and eight pairs. Each product is one rounding."""
    if kind == "codes" and K % 128:
        K = (K // 128 + 1) * 128
    R = T * topk
    at = torch.randperm(R, generator=_gen(1), device=DEV).int().view(T, topk)
    d = _randn(2, T, K)
    # no two weights of a token alike, and each far from its neighbours
    w = torch.randperm(R, generator=_gen(3), device=DEV).view(T, topk).float() * 1.0009765625 - 0.37 * R
    kw = {}
    if kind != "none":
        rows = _randn(4, R, K).bfloat16()
        kw = dict(rows=rows)
        if kind == "codes":
            q, s = bfq.quant_tokens(rows)
            kw = dict(rows=q, rows_scales=s)
    z = w.unsqueeze(2) * d.unsqueeze(1)
    g = bfq.moe_combine_backward(d, topk, weights=w, pair_rows=at, **kw)
    assert torch.equal(g["d_rows"][at.long()].view(torch.int16), z.bfloat16().view(torch.int16))
    if K % 128 == 0:
        g = bfq.moe_combine_backward(d, topk, weights=w, pair_rows=at, codes=True, **kw)
        zq, zs = _codes(z.view(R, K))
        p = at.reshape(-1).long()
        assert torch.equal(g["q"][p], zq) and torch.equal(g["scales"][p], zs)


@pytest.mark.parametrize("R", [1, 6, 8])
def test_empty_batch_writes_the_words_past_the_last_row(bfq, R):
    """Packed scales of a batch without tokens: the rows' words stay, those up to the next multiple of four are zero."""
    K, R4 = 640, (R + 3) // 4 * 4
    at = torch.empty((0, 2), dtype=torch.int32, device=DEV)
    q = torch.full((R, K), 9, dtype=torch.uint8, device=DEV)
    form = dict(layout=bfq.BFQ_SCALES_PACKED_UE8M0, scale_fmt=bfq.BFQ_SCALE_UE8M0)
    x, w = torch.empty((0, K), dtype=torch.bfloat16, device=DEV), torch.empty((0, 2), device=DEV)
    xs = torch.empty((2, 4), dtype=torch.int32, device=DEV)
    for call in (lambda s: bfq.bfq_moe_dispatch(x, at, q=q, scales=s, **form),
                 lambda s: bfq.bfq_moe_dispatch(x.view(torch.uint8)[:, :K].contiguous(), at, q=q, scales=s, x_scales=xs, x_layout=form["layout"],
                                                x_scale_ld=4, **form),
                 lambda s: bfq.bfq_moe_combine_backward(x, 2, pair_rows=at, q=q, scales=s, **form),
                 lambda s: bfq.bfq_moe_combine_backward(x, 2, weights=w, pair_rows=at, rows=torch.zeros((R, K), dtype=torch.bfloat16, device=DEV),
                                                        d_weights=w, q=q, scales=s, **form)):
        s = torch.full((2, R4 + 4), 0x0BADBEEF, dtype=torch.int32, device=DEV)
        call(s)
        assert bool((s[:, :R] == 0x0BADBEEF).all()) and not bool(s[:, R:R4].any()) and bool((s[:, R4:] == 0x0BADBEEF).all())
        assert bool((q == 9).all())


# ------------------------------------------------------------------ routers of many experts

@pytest.mark.parametrize("E,topk", [(300, 8), (384, 64), (385, 2), (448, 8), (512, 6), (512, 64), (513, 8)])
@pytest.mark.parametrize("score", [0, 1])
@pytest.mark.parametrize("form", ["plain", "bias", "groups", "ties"])
def test_route_of_many_experts(bfq, E, topk, score, form):
    """Every choice after the first from lists of six, eight and sixteen experts a lane, logits that repeat,
    masked experts."""
    T, groups, kept = 21, 1, 1
    x = _randn(E, T, E) * 2
    if form == "ties":                                       # eight values for all the experts
        x = torch.randint(-4, 4, (T, E), generator=_gen(1), device=DEV).float()
    if form == "groups":
        groups = next(g for g in (8, 7, 5, 3) if E % g == 0)
        kept = -(-topk * groups // E) + 1
    x[:, 3::11] = -math.inf
    x[5, topk // 2 + 1:] = -math.inf                          # fewer than topk are left (of two: both)
    b = 0.2 * _randn(4, E) if form == "bias" else None
    renorm = topk > 2
    ids, w = bfq.moe_route(x, topk, bias=b, score=score, n_groups=groups, topk_groups=kept, renorm=renorm, weight_scale=2.5)
    rid, rw = route._reference(x, topk, b, score, groups, kept, renorm, 2.5)
    assert torch.equal(ids.long(), rid)
    assert bool((ids[5] == -1).any()) == (topk > 2) and bool((ids[0] >= 0).any())
    assert bool(((w.double() - rw).abs() <= rw.abs() * U * (2 * route._spread(x) + 32)).all())


@pytest.mark.parametrize("E,topk", [(65, 6), (100, 8), (128, 64), (257, 8), (300, 6), (384, 64), (385, 2), (448, 8), (512, 64)])
@pytest.mark.parametrize("score,renorm", [(0, False), (0, True), (1, False), (1, True)])
@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
def test_route_backward_of_many_experts(bfq, E, topk, score, renorm, dt):
    """Against the formula in 64 bits, by autograd; an expert named twice, pairs that went elsewhere."""
    T = 19
    x = (_randn(E, T, E) * 2).to(dt)
    x[:, 5::13] = -math.inf
    ids, _ = bfq.moe_route(x, topk, score=score, renorm=renorm)
    ids[::3, -1] = -1
    ids[4, 1] = ids[4, 0]
    ids[3, 0] = E
    gw = _randn(5, T, topk)
    gw[ids < 0] = math.nan
    d = bfq.moe_route_backward(x, ids, gw, score=score, renorm=renorm, weight_scale=1.5)
    live = (ids >= 0) & (ids < E)
    at, g = ids.long().clamp(0, E - 1), torch.where(live, gw, 0.0).double()
    x64 = x.double().requires_grad_()
    s = torch.sigmoid(x64) if score else torch.softmax(x64, dim=1)
    w = s.gather(1, at) * live
    if renorm:
        w = w / (w.sum(dim=1, keepdim=True) + 1e-20)
    (1.5 * w * g).sum().backward()
    p, ref = s.detach(), x64.grad
    sj = p.gather(1, at) * live
    # the terms that are summed: A_j of ds_j, and their mean under the softmax
    A = 1.5 * g.abs()
    if renorm:
        D = sj.sum(dim=1, keepdim=True) + 1e-20
        A = A * sj.sum(dim=1, keepdim=True) / D ** 2 + 1.5 * (g.abs() * sj).sum(dim=1, keepdim=True) / D ** 2 + A * 1e-20 / D ** 2
    A = torch.where(live, A, 0.0)
    dense = torch.zeros_like(p).scatter_add_(1, at, A)
    terms = dense * p * (1 - p) if score else p * (dense + (A * sj).sum(dim=1, keepdim=True))
    # a score: the difference to the largest (u of it in the exponential), 16 additions in a lane, 6 over the wave,
    # a division, some 32 u in all, three times over in ds; then topk additions; one rounding to the output
    tol = terms * U * ((0 if score else 4) * route._spread(x) + 96 + 2 * topk) + torch.finfo(dt).eps / 2 * ref.abs() + 2.0 ** -133
    assert bool(((d.double() - ref).abs() <= tol).all()), float(((d.double() - ref).abs() / tol).max())
    assert bool((ref.abs() > tol).any(dim=1)[1])              # zeros would not pass for the tokens left as they were


# -------------------------------------------------------------- sums of the weights' gradient

@pytest.mark.parametrize("T,topk,K", [(2, 3, 264), (2, 3, 2048), (3, 9, 2056), (3, 10, 12288), (2, 5, 16384), (500, 9, 4224)])
@pytest.mark.parametrize("kind", ["bf16", "fp16", "fp32", "codes"])
@pytest.mark.parametrize("codes", [False, True])
def test_roundings_of_the_weights_gradient(bfq, T, topk, K, kind, codes):
    """Counted on the kernel's sum: a thread takes W = 8 columns a round (16 from codes to codes), W products, one
    addition to what earlier rounds gave, for rows of codes one product with the scale; at most 256 threads, so
    ceil(K / (256 W)) rounds; 6 additions over a wave and one less than the waves over them."""
    if K % 128 and (codes or kind == "codes"):
        K = K // 128 * 128 + 128
    R = T * topk
    at = torch.randperm(R, generator=_gen(1), device=DEV).int().view(T, topk)
    d, w = _randn(2, T, K), torch.rand((T, topk), generator=_gen(3), device=DEV)
    rows = _randn(4, R, K).to({"fp16": torch.float16, "fp32": torch.float32}.get(kind, torch.bfloat16))
    kw, value = dict(rows=rows), rows.double()
    if kind == "codes":
        q, s = bfq.quant_tokens(rows)
        kw = dict(rows=q, rows_scales=s)
        value = q.view(torch.float8_e4m3fn).double() * s.double().repeat_interleave(128, dim=1)
    dw = bfq.moe_combine_backward(d, topk, weights=w, pair_rows=at, codes=codes, **kw)["d_weights"]
    W = 16 if kind == "codes" and codes else 8
    count = W + (kind == "codes") + (-(-K // (256 * W)) - 1) + 6 + 3
    terms = value[at.long()] * d.double().unsqueeze(1)
    ref, tol = terms.sum(dim=2), terms.abs().sum(dim=2) * U * count * (1 + 64 * U)
    assert bool(((dw.double() - ref).abs() <= tol).all()), float(((dw.double() - ref).abs() / tol).max())
    assert float((ref.abs() > tol).float().mean()) > 0.9

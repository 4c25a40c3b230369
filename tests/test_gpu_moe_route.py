"""GPU tests of the router and its gradient, and of the sort of pairs by expert.

Ids are compared exactly with a stable descending sort of the keys in 64 bits. Weights and gradients
count roundings (u = 2^-24): a score relative to itself is off by the difference x - max (u |x - max|
in the exponential), the exponential, its sum (16 additions in a lane, 6 over the wave) and a division,
32 u with room for the products after it; `spread` is the largest |x - max| of a row.
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U = 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -9, torch.float16: 2.0 ** -12, torch.float32: 2.0 ** -25}   # of a unit of 2 |x|
EPS = 1e-20


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _randn(seed, *shape):
    return torch.randn(shape, generator=_gen(seed), device=DEV)


def _scores(x, score):
    x = x.double().clamp(max=torch.finfo(torch.float32).max)
    if score:
        return torch.sigmoid(x)
    top = x.amax(dim=1, keepdim=True)
    e = torch.exp(x - torch.where(torch.isinf(top), 0.0, top))
    return e / e.sum(dim=1, keepdim=True)


def _reference(logits, topk, bias, score, groups, topk_groups, renorm, scale):
    x = logits.double()
    T, E = x.shape
    s = _scores(logits, score)
    masked = x == -math.inf
    key = x.clamp(max=torch.finfo(torch.float32).max)
    if bias is not None or groups > 1:
        key = torch.where(masked, -math.inf, s + (0.0 if bias is None else bias.double()))
    if groups > 1:
        per = key.view(T, groups, E // groups)
        best = torch.sort(per, dim=2, descending=True).values[:, :, :2]
        total = torch.where(best == -math.inf, 0.0, best).sum(dim=2)
        total = torch.where(best[:, :, 0] == -math.inf, -math.inf, total)
        first = torch.sort(total, dim=1, descending=True, stable=True).indices[:, :topk_groups]
        keep = torch.zeros((T, groups), dtype=torch.bool, device=DEV).scatter_(1, first, True)
        key = torch.where(keep.unsqueeze(2), per, -math.inf).reshape(T, E)
    order = torch.sort(key, dim=1, descending=True, stable=True)
    ids = order.indices[:, :topk]
    got = order.values[:, :topk] != -math.inf
    w = torch.where(got, s.gather(1, ids), 0.0)
    if renorm:
        w = w / (w.sum(dim=1, keepdim=True) + EPS)
    return torch.where(got, ids, -1), w * scale


def _spread(logits):
    x = logits.double()
    x = torch.where(torch.isinf(x), x.amax(dim=1, keepdim=True), x)
    return (x.amax(dim=1, keepdim=True) - x).amax(dim=1, keepdim=True).nan_to_num(nan=0.0)   # none is left: 0


CASES = [
    # T, E, topk, dtype, bias, score, groups, topk_groups, renorm
    (1, 1, 1, torch.float32, False, 0, 1, 1, False),
    (1, 1, 1, torch.bfloat16, True, 1, 1, 1, True),
    (5, 7, 3, torch.float16, False, 0, 1, 1, True),
    (37, 64, 8, torch.bfloat16, False, 1, 1, 1, False),
    (130, 65, 6, torch.float32, False, 0, 1, 1, True),
    (9, 160, 6, torch.float32, True, 0, 8, 3, False),
    (64, 256, 8, torch.float32, True, 1, 8, 4, True),
    (33, 256, 8, torch.bfloat16, False, 1, 8, 4, True),
    (17, 257, 64, torch.float32, True, 1, 1, 1, True),
    (12, 512, 1, torch.bfloat16, False, 0, 64, 1, False),
    (6, 1023, 16, torch.float32, False, 0, 1, 1, False),
    (6, 1023, 16, torch.float32, True, 1, 31, 2, False),
    (4, 60, 60, torch.float16, True, 0, 60, 60, True),
    (1000, 24, 4, torch.bfloat16, True, 1, 3, 2, True),
]


@pytest.mark.parametrize("T,E,topk,dt,bias,score,groups,kept,renorm", CASES)
@pytest.mark.parametrize("mask", [False, True])
def test_route(bfq, T, E, topk, dt, bias, score, groups, kept, renorm, mask):
    x = (_randn(E + T, T, E) * 2).to(dt)                    # 16-bit logits meet many ties
    if mask:
        x[torch.rand((T, E), generator=_gen(3), device=DEV) < 0.4] = -math.inf
        x[0] = -math.inf
    b = 0.2 * _randn(4, E) if bias else None
    ids, w = bfq.moe_route(x, topk, bias=b, score=score, n_groups=groups, topk_groups=kept, renorm=renorm,
                           weight_scale=2.5)
    rid, rw = _reference(x, topk, b, score, groups, kept, renorm, 2.5)
    assert torch.equal(ids.long(), rid)
    if mask:
        assert bool((ids[0] == -1).all()) and not bool(w[0].any())
    tol = rw.abs() * U * (2 * _spread(x) + 32)
    assert bool(((w.double() - rw).abs() <= tol).all())


def test_route_extreme_logits(bfq):
    inf, nan, low = math.inf, math.nan, torch.finfo(torch.float32).min
    x = torch.tensor([[1.0, inf, 2.0, -inf, 0.0, -0.0],      # +inf takes all of a softmax
                      [low, low, -inf, -inf, -inf, low],     # the type's lowest value is no mask
                      [nan, 1.0, 2.0, 3.0, -inf, 0.0],       # a NaN comes first and spreads
                      [0.0, -0.0, 0.0, -0.0, 0.0, -0.0],     # zeros of both signs are equal
                      [-inf] * 6, [inf] * 6], device=DEV)
    ids, w = bfq.moe_route(x, 4)
    assert ids.tolist() == [[1, 2, 0, 4], [0, 1, 5, -1], [0, 3, 2, 1], [0, 1, 2, 3], [-1] * 4, [0, 1, 2, 3]]
    assert w[0].tolist() == [1.0, 0.0, 0.0, 0.0] and w[4].tolist() == [0.0] * 4
    assert torch.allclose(w[1, :3], torch.full((3,), 1 / 3, device=DEV)) and w[1, 3] == 0
    assert bool(torch.isnan(w[2]).all())
    assert torch.allclose(w[5], torch.full((4,), 1 / 6, device=DEV))
    # sigmoid: a NaN is its expert's alone; biased keys; sums that are all zero divide by the floor
    ids, w = bfq.moe_route(x, 4, score=bfq.BFQ_SCORE_SIGMOID, bias=torch.zeros(6, device=DEV))
    assert ids[2].tolist() == [0, 3, 2, 1] and bool(torch.isnan(w[2, 0])) and not bool(torch.isnan(w[2, 1:]).any())
    assert ids[0].tolist() == [1, 2, 0, 4] and ids[3].tolist() == [0, 1, 2, 3]
    _, w = bfq.moe_route(torch.full((1, 6), -1e4, device=DEV), 4, score=bfq.BFQ_SCORE_SIGMOID, renorm=True)
    assert w.tolist() == [[0.0] * 4]
    # a bias of -inf takes an expert out of the choice
    b = torch.tensor([0.0, -inf, 0.0, 0.0, 0.0, 0.0], device=DEV)
    ids, _ = bfq.moe_route(torch.arange(6.0, device=DEV).view(1, 6), 6, bias=b)
    assert ids.tolist() == [[5, 4, 3, 2, 0, -1]]


def test_route_masked_groups(bfq):
    """A masked expert counts as nothing in its group's sum; a group of masked ones never stays, and
    experts of the groups that went are not taken even where those that stay have too few."""
    inf = math.inf
    x = torch.full((3, 8), -inf, device=DEV)
    x[0] = torch.tensor([3.0, -inf, 1.0, 0.9, -inf, -inf, 0.0, 0.1])
    x[1, 2] = 5.0
    x[2] = torch.tensor([-inf, -inf, -inf, -inf, 0.0, 0.0, -inf, 0.0])
    ids, _ = bfq.moe_route(x, 4, score=bfq.BFQ_SCORE_SIGMOID, n_groups=4, topk_groups=2)
    rid, _ = _reference(x, 4, None, 1, 4, 2, False, 1.0)
    assert torch.equal(ids.long(), rid)
    assert ids.tolist() == [[2, 3, 7, 6], [2, -1, -1, -1], [4, 5, 7, -1]]


@pytest.mark.parametrize("T,E,topk,dt,score,renorm", [
    (1, 1, 1, torch.float32, 0, True), (3, 5, 5, torch.bfloat16, 1, True), (40, 64, 8, torch.float32, 0, False),
    (65, 256, 8, torch.float32, 1, True), (65, 256, 8, torch.float16, 0, True), (33, 130, 3, torch.float32, 1, False),
    (7, 1023, 64, torch.float32, 0, False), (7, 1023, 64, torch.float32, 1, True), (2000, 16, 2, torch.bfloat16, 0, True)])
def test_route_backward(bfq, T, E, topk, dt, score, renorm):
    x = (_randn(E, T, E) * 2).to(dt)
    if E > 2:
        x[torch.rand((T, E), generator=_gen(2), device=DEV) < 0.2] = -math.inf
    ids, _ = bfq.moe_route(x, topk, score=score, renorm=renorm)
    ids[::3, -1] = -1                                      # a pair that went elsewhere, its gradient anything
    if T > 4 and topk > 1:
        ids[4, 1] = ids[4, 0]                              # an expert twice
        ids[3, 0] = E
    gw = _randn(5, T, topk)
    gw[ids < 0] = math.nan
    d = bfq.moe_route_backward(x, ids, gw, score=score, renorm=renorm, weight_scale=1.5)
    # the formula in 64 bits, by autograd
    live = (ids >= 0) & (ids < E)
    at, g = ids.long().clamp(0, E - 1), torch.where(live, gw, 0.0).double()
    x64 = x.double().requires_grad_()
    s = torch.sigmoid(x64) if score else torch.softmax(x64, dim=1)
    w = s.gather(1, at) * live
    if renorm:
        w = w / (w.sum(dim=1, keepdim=True) + EPS)
    (1.5 * w * g).sum().backward()
    ref = torch.nan_to_num(x64.grad, nan=0.0)              # a row without a live logit
    p = torch.nan_to_num(s.detach(), nan=0.0)
    # magnitudes of the terms that are summed: A_j of ds_j, and their mean under the softmax
    sj = p.gather(1, at) * live
    if renorm:
        D = sj.sum(dim=1, keepdim=True) + EPS
        A = 1.5 * (g.abs() * sj.sum(dim=1, keepdim=True) + (g.abs() * sj).sum(dim=1, keepdim=True) + EPS * g.abs()) / D ** 2
    else:
        A = 1.5 * g.abs()
    A = torch.where(live, A, 0.0)
    dense = torch.zeros_like(p).scatter_add_(1, at, A)
    terms = dense * p * (1 - p) if score else p * (dense + (A * sj).sum(dim=1, keepdim=True))
    # roundings: the scores' (spread and sum) enter ds three times over, then topk additions
    tol = terms * U * (4 * (0 if score else 1) * _spread(x) + 96 + 2 * topk) + 2 * HALF[dt] * ref.abs()
    tol = tol + (2.0 ** -25 if dt == torch.float16 else 2.0 ** -134 if dt == torch.bfloat16 else 2.0 ** -140)
    assert not bool(torch.isnan(d).any())
    assert bool(((d.double() - ref).abs() <= tol).all()), float(((d.double() - ref).abs() / tol).max())


def test_route_gradient_against_differences(bfq):
    """Central differences of the weights that the router itself gives."""
    T, E, topk, h = 8, 32, 4, 2.0 ** -6
    for score, renorm in ((0, False), (0, True), (1, False), (1, True)):
        x = _randn(1, T, E)
        g = _randn(2, T, topk)
        ids, w0 = bfq.moe_route(x, topk, score=score, renorm=renorm)
        d = bfq.moe_route_backward(x, ids, g, score=score, renorm=renorm)

        def weights(x):                                    # of the same ids
            s = _scores(x, score).gather(1, ids.long())
            return s / (s.sum(dim=1, keepdim=True) + EPS) if renorm else s
        assert bool(((weights(x) - w0).abs() <= 64 * U * w0).all())
        for e in range(0, E, 5):
            up, dn = x.double(), x.double()
            up[:, e] += h
            dn[:, e] -= h
            slope = ((weights(up) - weights(dn)) * g).sum(dim=1) / (2 * h)
            # third derivatives of softmax and sigmoid ratios are at most 6: h^2 each, by sum |g|
            tol = h * h * g.abs().sum(dim=1) + 1e-6
            assert bool(((d[:, e] - slope).abs() <= tol).all())


def test_route_empty_and_guards(bfq):
    i32 = torch.int32
    bfq.moe_route(torch.empty((0, 8), device=DEV), 2)
    bfq.moe_route_backward(torch.empty((0, 8), device=DEV), torch.empty((0, 2), dtype=i32, device=DEV), torch.empty((0, 2), device=DEV))
    x = _randn(1, 7, 10)
    ids, w, d = torch.full((9, 3), 77, dtype=i32, device=DEV), torch.full((9, 3), 77.0, device=DEV), torch.full((9, 10), 77.0, device=DEV)
    bfq.bfq_moe_route(x, ids[1:8], w[1:8])
    bfq.bfq_moe_route_backward(x, ids[1:8], w[1:8], d[1:8])
    for t in (ids, w, d):
        assert bool((t[0] == 77).all()) and bool((t[8] == 77).all()) and not bool((t[1:8] == 77).any())


# ------------------------------------------------------------------------------- sort

def _sorted(ids, E):
    flat = ids.reshape(-1).long()
    b = torch.where((flat >= 0) & (flat < E), flat, E)
    order = torch.argsort(b, stable=True)
    at = torch.empty_like(order)
    at[order] = torch.arange(order.numel(), device=DEV)
    off = torch.zeros(E + 2, dtype=torch.long, device=DEV)
    off[1:] = torch.cumsum(torch.bincount(b, minlength=E + 1), 0)
    return off[: E + 1].int(), order.int(), torch.where(b < E, at, -1).int().view_as(ids)


@pytest.mark.parametrize("T,topk,E", [(1, 1, 1), (1, 8, 256), (3, 5, 1023), (128, 8, 256), (1024, 1, 7), (1025, 1, 7), (205, 5, 1),
                                      (4096, 8, 256), (777, 8, 1023), (1024, 8, 256), (1025, 8, 256), (4097, 8, 256), (300000, 1, 64), (40000, 33, 1000)])
@pytest.mark.parametrize("kind", ["all", "some", "one"])
def test_sort(bfq, T, topk, E, kind):
    lo, hi = {"all": (0, E), "some": (-E, 2 * E), "one": (E - 1, E)}[kind]
    ids = torch.randint(lo, hi, (T, topk), generator=_gen(T + E), device=DEV, dtype=torch.int32)
    if kind == "some":
        ids[0, 0], ids[-1, -1] = -2 ** 31, 2 ** 31 - 1
    off, srt, places = bfq.moe_sort(ids, E)
    roff, rsrt, rplaces = _sorted(ids, E)
    assert torch.equal(off, roff) and torch.equal(srt, rsrt) and torch.equal(places, rplaces)
    aoff, asrt = bfq.moe_align(ids, E)
    assert torch.equal(off, aoff) and torch.equal(srt, asrt)


def test_sort_empty_and_guards(bfq):
    off, srt, places = bfq.moe_sort(torch.empty((0, 4), dtype=torch.int32, device=DEV), 1023)
    assert not bool(off.any()) and srt.numel() == 0 and places.shape == (0, 4)
    for T in (400, 12000):                                  # in one launch, in two
        ids = torch.randint(0, 5, (T, 3), generator=_gen(1), device=DEV, dtype=torch.int32)
        off, srt, places = (torch.full((n,), 77777, dtype=torch.int32, device=DEV) for n in (5 + 1 + 2, 3 * T + 2, 3 * T + 2))
        n = bfq.bfq_moe_sort_workspace_bytes(T, 3, 5)
        assert (n > 0) == (T == 12000)
        ws = torch.full((n + 8,), 99, dtype=torch.uint8, device=DEV)
        bfq.bfq_moe_sort(ids, 5, off[1:7], srt[1:-1], places[1:-1].view(T, 3), workspace=ws[4:4 + n])
        for t in (off, srt, places):
            assert t[0] == 77777 and t[-1] == 77777 and not bool((t[1:-1] == 77777).any())
        assert bool((ws[:4] == 99).all()) and bool((ws[-4:] == 99).all())

"""GPU tests of the mixture-of-experts operators where rows are narrow or end inside a wave, batches empty,
experts many: calls that the documentation allows and that are seldom made."""
import pytest
import torch

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

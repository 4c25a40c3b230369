"""GPU tests of the gated product's values: infinities and overflow, one rounding to each output type,
equal bits from equal calls."""
import pytest
import torch

from test_gpu_ffn import _act, _gated_tiles, _gu, _pair

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _same(a, b):
    return torch.equal(a.isnan(), b.isnan()) and torch.equal(a[~a.isnan()], b[~b.isnan()])


@pytest.mark.parametrize("act", [0, 1])
@pytest.mark.parametrize("wl", [0, 1])
def test_infinite_and_overflowing_sums(bfq, wl, act):
    """Tokens whose sums pass the range of fp32 on either side: act(+inf) is +inf, act(-inf) the NaN that
    -inf * 0 is, and a product past the range an infinity; groups of codes that hold one have an infinite
    scale and zeros beside it, groups with a NaN a NaN scale. The other tokens keep their values."""
    F, K = 256, 256
    for t in _gated_tiles(bfq, wl, 0):
        M = t.bm + 3
        qa, sa, qw, sw, _ = _pair(bfq, M, F, K, 9, 0, wl)
        kw = dict(act=act, tile=t, w_layout=wl)
        clean = bfq.gated_gemm(qa, sa, qw, sw, out_dtype=torch.float32, **kw)
        q0, s0 = bfq.gated_gemm(qa, sa, qw, sw, codes=True, **kw)
        sa[1] *= 2.0 ** 126                          # sums past 2^128, both factors infinite
        sa[2] *= 2.0 ** 70                           # finite sums, products past 2^128
        sa[3] = float("inf")
        gu = _gu(bfq, qa, sa, qw, sw, t, wl, 0)
        g, u = gu[:, :F], gu[:, F:]
        h = (_act(g, act)[0] * u).float()
        out = bfq.gated_gemm(qa, sa, qw, sw, out_dtype=torch.float32, **kw)
        far = ~torch.isfinite(h)
        # a product that is finite in 64 bits but within the tolerance of the end of fp32's range may be
        # either; there is none here: sums are a few times 2^-3 * 2^70, their products past 2^134 or gates
        # that have vanished
        assert bool(far[1:4].any()) and not bool(far[[0] + list(range(4, M))].any())
        assert _same(out[far], h[far]) and bool(torch.isfinite(out[~far]).all())
        keep = [m for m in range(M) if m not in (1, 2, 3)]
        assert torch.equal(out[keep], clean[keep])
        q, s = bfq.gated_gemm(qa, sa, qw, sw, codes=True, **kw)
        assert torch.equal(q[keep], q0[keep]) and torch.equal(s[keep], s0[keep])
        for m in (1, 2, 3):
            for b in range(F // 128):
                part, codes = out[m, b * 128:b * 128 + 128], q[m, b * 128:b * 128 + 128]
                if bool(part.isnan().any()):
                    assert bool(s[m, b].isnan()) and bool((codes == 0x7F).all())
                elif bool(part.isinf().any()):
                    assert bool(s[m, b].isinf())
                    assert bool((codes[part.isinf()] == 0x7F).all()) and not bool((codes[~part.isinf()] & 0x7F).any())


@pytest.mark.parametrize("sfmt", [0, 1])
@pytest.mark.parametrize("wl", [0, 1])
def test_outputs_are_the_fp32_ones_rounded(bfq, wl, sfmt):
    """bf16 and fp16 outputs are the fp32 outputs of the same tile, rounded once to nearest even, over the
    whole range of fp16: overflow, subnormals, zeros. Calls repeated give the same bits."""
    F, K = 384, 640
    for t0 in _gated_tiles(bfq, wl, sfmt):
        M = 2 * t0.bm - 3
        qa, sa, qw, sw, _ = _pair(bfq, M, F, K, 13, sfmt, wl)
        sa *= torch.exp2((7 * torch.arange(M, device=DEV)).remainder(48) - 32.0)[:, None]
        for split in (1, 2):
            t = bfq.bfq_tile.from_dict({**t0.as_dict(), "split_k": split})
            kw = dict(tile=t, w_layout=wl, scale_fmt=sfmt)
            full, pre = bfq.gated_gemm(qa, sa, qw, sw, out_dtype=torch.float32, keep_preact=True, **kw)
            assert bool((full.abs() > 65504).any()) and bool((full.abs() < 2.0 ** -20).any())
            for dt in (torch.bfloat16, torch.float16):
                assert _same(bfq.gated_gemm(qa, sa, qw, sw, out_dtype=dt, **kw), full.to(dt)), t.as_dict()
            codes = bfq.gated_gemm(qa, sa, qw, sw, codes=True, **kw)
            for _ in range(3):
                again = bfq.gated_gemm(qa, sa, qw, sw, out_dtype=torch.float32, keep_preact=True, **kw)
                assert torch.equal(again[0], full) and torch.equal(again[1], pre), t.as_dict()
                assert all(torch.equal(a, b) for a, b in zip(bfq.gated_gemm(qa, sa, qw, sw, codes=True, **kw), codes))

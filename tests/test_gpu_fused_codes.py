"""GPU tests: the kernels that quantize what they compute store encode(x / scale) with the IEEE
quotient, as the token quantizer does, where the fp32 values x they quantize are known exactly."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _randn(seed, *shape):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return torch.randn(shape, generator=g, device=DEV)


def _differ(codes, want, int8):
    """Places where codes stand for another number: the norm step's sum with an absent y is r + 0, which
    makes -0 a +0, so the sign of a zero is not compared."""
    codes = codes.cpu()
    if int8:
        return codes != want
    return codes.view(torch.float8_e4m3fn).float() != want.view(torch.float8_e4m3fn).float()


def _expected(x, int8, ue8m0, group, eps=1e-10):
    """Codes and scales of fp32 x by IEEE fp32 operations on the host."""
    g = x.cpu().numpy().reshape(x.shape[0], -1, group)
    s = np.maximum(np.abs(g).max(2), np.float32(eps)) / np.float32(127 if int8 else 448)
    if ue8m0:
        m, e = np.frexp(s)
        s = np.ldexp(np.float32(1), np.where(m == 0.5, e - 1, e)).astype(np.float32)
    v = g / s[:, :, None]
    assert v.dtype == np.float32
    if int8:
        return torch.from_numpy(np.rint(v).astype(np.int8)).view(x.shape), torch.from_numpy(s)
    return torch.from_numpy(v).to(torch.float8_e4m3fn).view(torch.uint8).view(x.shape), torch.from_numpy(s)


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("sfmt", [0, 1])
@pytest.mark.parametrize("M,K,per_token", [(4096, 1536, False), (1500, 7168, False), (600, 16384, False),
                                           (2000, 2176, True)])
def test_norm_codes_are_the_ieee_quotients(bfq, M, K, per_token, sfmt, int8):
    """Rows so small that the mean square is lost beside norm_eps = 1: 1 / rms is 1 and the normed row
    is the residual itself, any fp32 values. Zeros of both signs among them."""
    r = _randn(K, M, K) * torch.exp(2 * _randn(M, M, 1).clamp(-3, 3)) * 1e-7
    r[:, 5] = 0.0
    r[:, 7] = -0.0
    assert float((r.double() ** 2).mean(1).max()) < 2.0 ** -26
    q, s = bfq.norm_residual(r, w_pre=torch.ones(K, device=DEV).bfloat16(), norm_eps=1.0, codes=True,
                             per_token=per_token, scale_fmt=sfmt, q_dtype=bfq.BFQ_INT8 if int8 else bfq.BFQ_E4M3FN)
    want_q, want_s = _expected(r, int8, sfmt == 1, K if per_token else 128)
    assert torch.equal(s.cpu(), want_s)
    wrong = _differ(q, want_q, int8)
    assert not bool(wrong.any()), f"{int(wrong.sum())} of {wrong.numel()} codes"


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("exp", [-90, -64, -59, 0, 80, 110])
def test_norm_codes_at_the_ends_of_the_range(bfq, exp, int8):
    """Group maxima from far below the default floor to far above 1, through a norm that scales nothing
    (rows past 2^-30 have their own norm_eps, which takes the mean square's place)."""
    M, K = 64, 512
    base = torch.exp2(_randn(1, M, K).clamp(-3, 3)) * torch.sign(_randn(2, M, K))
    w = torch.full((K,), 2.0 ** exp, device=DEV).bfloat16()       # exact: n = r * w
    r = base * 2.0 ** -30
    q, s = bfq.norm_residual(r, w_pre=w, norm_eps=1.0, codes=True, q_dtype=bfq.BFQ_INT8 if int8 else bfq.BFQ_E4M3FN)
    q2, s2 = torch.empty_like(q), torch.empty_like(s)
    bfq.bfq_norm_residual(r, w_pre=w, norm_eps=1.0, q=q2, scales=s2, q_eps=1e-36)
    for codes, scales, eps in ((q, s, 1e-10), (q2, s2, 1e-36)):
        want_q, want_s = _expected(r * 2.0 ** exp, int8, False, 128, eps)
        assert torch.equal(scales.cpu(), want_s) and torch.equal(codes.cpu(), want_q)


@pytest.mark.parametrize("int8", [False, True])
def test_gradient_codes_are_the_ieee_quotients(bfq, int8):
    """Gates so large that the sigmoid is 1: dg = dh * u exactly (products of two bf16), du = dh * g.
    Zeros of both signs among them."""
    M, F = 3000, 2048
    g = torch.full((M, F), 64.0, device=DEV)
    u, dh = _randn(1, M, F).bfloat16(), _randn(2, M, F).bfloat16()
    u[:, 3], dh[:, 9] = 0.0, -0.0
    q, s = bfq.gated_backward(torch.cat([g.bfloat16(), u], 1), dh, codes=True,
                              q_dtype=bfq.BFQ_INT8 if int8 else bfq.BFQ_E4M3FN)
    x = torch.cat([dh.float() * u.float(), dh.float() * 64], 1)
    want_q, want_s = _expected(x, int8, False, 128)
    assert torch.equal(s.cpu(), want_s)
    wrong = q.cpu() != want_q                        # here the sign of a zero is known too
    assert not bool(wrong.any()), f"{int(wrong.sum())} of {wrong.numel()} codes"


@pytest.mark.parametrize("wl", [0, 1])
@pytest.mark.parametrize("sfmt", [0, 1])
def test_gated_codes_are_the_ieee_quotients(bfq, wl, sfmt):
    """One nonzero column of tokens and weights and gates past 64, whose sigmoid is 1: every step to the
    product is one known fp32 rounding, on each compiled tile, plain and split."""
    F, K = 384, 512
    g = torch.Generator().manual_seed(3 + sfmt)
    finite = torch.tensor([c for c in range(256) if c & 0x7F != 0x7F], dtype=torch.uint8)
    val = lambda c: c.view(torch.float8_e4m3fn).float()  # noqa: E731
    for n, t0 in enumerate(bfq.bfq_gated_get_tile_candidate(i, wl, sfmt)
                           for i in range(bfq.bfq_gated_num_tile_candidates(wl, sfmt))):
        M = 2 * t0.bm - 3
        a, w = torch.zeros(M, K, dtype=torch.uint8), torch.zeros(2 * F, K, dtype=torch.uint8)
        a[:, 200] = torch.randint(0x38, 0x7F, (M,), generator=g).to(torch.uint8)           # 1 .. 448
        w[:F, 200] = 0x38                                                                    # 1
        w[F:, 200] = finite[torch.randint(0, len(finite), (F,), generator=g)]
        sa, sw = 1 + torch.rand(M, K // 128, generator=g), 1 + torch.rand(2 * F // 128, K // 128, generator=g)
        if sfmt:
            sa, sw = (2.0 ** torch.randint(0, 8, s.shape, generator=g) for s in (sa, sw))
        sw[:F // 128] *= 64
        c = sa[:, 1:2] * sw[:, 1].repeat_interleave(128)
        gu = (val(a[:, 200])[:, None] * val(w[:, 200])) * c         # products of codes are exact
        h = gu[:, :F] * gu[:, F:]
        want_q, want_s = _expected(h, False, sfmt == 1, 128)
        qa, qw, sa, sw = a.to(DEV), w.to(DEV), sa.to(DEV), sw.to(DEV)
        qw = bfq.pack_weights(qw) if wl else qw
        for split in (1, 2):
            t = bfq.bfq_tile.from_dict({**t0.as_dict(), "split_k": split})
            q, s = bfq.gated_gemm(qa, sa, qw, sw, codes=True, tile=t, w_layout=wl, scale_fmt=sfmt)
            assert torch.equal(s.cpu(), want_s), t.as_dict()
            wrong = _differ(q, want_q, False)
            assert not bool(wrong.any()), f"{int(wrong.sum())} of {wrong.numel()} codes, {t.as_dict()}"

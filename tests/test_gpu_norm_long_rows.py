"""GPU tests of the norm step on rows past 8192 channels in batches of more than 256 tokens, which take
a kernel of their own (four chunks a thread), against the formulas in 64 bits."""
import pytest
import torch

from test_gpu_ffn import H, _check_codes, _norm_case, _norm_ref, _unpack_scales, _within

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("K", [8200, 10248, 16384])
def test_long_rows_bf16_out(bfq, K, rt):
    for M, post, kind in ((257, True, 0), (300, True, 1), (300, False, 2), (301, True, 3)):
        c = _norm_case(M, K, post, kind, rt, K + kind)
        r, rtol, n, ntol = _norm_ref(c)
        res, nrm = bfq.norm_residual(**c)
        _within(res, r, rtol + H[rt] * r.abs(), f"res {M} {post} {kind}")
        _within(nrm, n, ntol + H[torch.bfloat16] * n.abs(), f"normed {M} {post} {kind}")


@pytest.mark.parametrize("lay,sfmt,int8,per_token", [
    (0, 0, False, False), (1, 0, True, False), (1, 1, False, False), (2, 1, False, False),
    (2, 1, True, False), (0, 0, False, True), (1, 0, True, True), (0, 1, False, True)])
@pytest.mark.parametrize("K", [8320, 12288, 16384])
def test_long_rows_codes(bfq, K, lay, sfmt, int8, per_token):
    for M, post, kind, rt in ((257, True, 1, torch.bfloat16), (258, False, 0, torch.float32)):
        c = _norm_case(M, K, post, kind, rt, K + M)
        r, rtol, n, ntol = _norm_ref(c)
        G = 1 if per_token else K // 128
        res, q, s = bfq.norm_residual(**c, codes=True, layout=lay, scale_fmt=sfmt, per_token=per_token,
                                      q_dtype=bfq.BFQ_INT8 if int8 else bfq.BFQ_E4M3FN)
        _within(res, r, rtol + H[rt] * r.abs(), "res")
        _check_codes(q, _unpack_scales(bfq, s, lay, M, G), n, ntol, sfmt == 1, f"{M}", int8=int8,
                     group=K if per_token else 128)

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


def test_more_rows_than_one_launch_holds(bfq):
    """K = 8192 takes 512 threads a row, and a grid dimension fewer than 2^32 threads: past 2^23 - 1 rows
    a call takes two launches. Rows on both sides of the seam and at the ends, packed words with their
    padding rows, against a call on those rows alone."""
    M, K = (1 << 23) + 6, 8192
    if torch.cuda.mem_get_info()[0] < (3 * M * K) + (4 << 30):
        pytest.skip("needs 210 GB of free device memory")
    pick = torch.tensor([0, 1, 4095, (1 << 23) - 6] + list(range((1 << 23) - 5, M)), device="cuda:0")
    few = torch.randn(len(pick), K, device="cuda:0").bfloat16()
    w = torch.ones(K, device="cuda:0").bfloat16()
    x = torch.empty((M, K), dtype=torch.bfloat16, device="cuda:0")        # the other rows hold anything
    x[pick] = few
    q = torch.empty((M, K), dtype=torch.uint8, device="cuda:0")
    words = torch.full((K // 512, M + 6), -1, dtype=torch.int32, device="cuda:0")
    bfq.bfq_norm_residual(x, w_pre=w, q=q, scales=words, layout=bfq.BFQ_SCALES_PACKED_UE8M0,
                          scale_fmt=bfq.BFQ_SCALE_UE8M0)
    q2, words2 = bfq.norm_residual(few, w_pre=w, codes=True, layout=bfq.BFQ_SCALES_PACKED_UE8M0,
                                   scale_fmt=bfq.BFQ_SCALE_UE8M0)
    assert torch.equal(q[pick], q2) and torch.equal(words[:, pick], words2[:, :len(pick)])
    assert not bool(words[:, M:M + 2].any()) and bool((words[:, M + 2:] == -1).all())
    del x, q, words
    torch.cuda.empty_cache()

"""GPU tests of the batch-invariant switch on the norm step and its gradients: with it set, a token's
rows do not depend on how many tokens there are."""
import pytest
import torch

from test_gpu_ffn import _norm_case, _randn

pytestmark = pytest.mark.gpu


@pytest.fixture
def invariant(bfq):
    was = bfq.bfq_get_batch_invariant()
    bfq.bfq_set_batch_invariant(True)
    yield
    bfq.bfq_set_batch_invariant(was)


@pytest.mark.parametrize("rt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("K", [2048, 2176, 8192, 8320, 12288, 16384])
def test_norm_rows_do_not_depend_on_the_batch(bfq, invariant, K, rt):
    full = _norm_case(300, K, True, 3, rt, K)
    forms = (dict(), dict(codes=True), dict(codes=True, per_token=True, q_dtype=bfq.BFQ_INT8),
             dict(codes=True, scale_fmt=1))
    want = [bfq.norm_residual(**full, **kw) for kw in forms]
    for M in (1, 7, 256, 257):
        part = {k: v[:M] if k in ("residual", "y", "gate") else v for k, v in full.items()}
        for kw, ref in zip(forms, want):
            for a, b in zip(bfq.norm_residual(**part, **kw), ref):
                assert torch.equal(a, b[:M]), (M, kw)


@pytest.mark.parametrize("K", [1544, 8192, 8200, 16384])
def test_norm_gradient_rows_do_not_depend_on_the_batch(bfq, invariant, K):
    full = _norm_case(700, K, True, 3, torch.float32, K)
    r = full.pop("residual")
    dn, dro = _randn(K + 1, 700, K).bfloat16(), _randn(K + 2, 700, K)
    want = bfq.norm_residual_backward(r, **full, d_normed=dn, d_res_out=dro)
    for M in (1, 255, 257):
        part = {k: v[:M] if k in ("y", "gate") else v for k, v in full.items()}
        got = bfq.norm_residual_backward(r[:M], **part, d_normed=dn[:M], d_res_out=dro[:M])
        for k in ("d_res", "d_y", "d_gate"):
            assert torch.equal(got[k], want[k][:M]), (M, k)

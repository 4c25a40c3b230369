"""CPU tests of empty batches in the mixture-of-experts layer's entry points: no launch is needed to serve them."""
import torch

import test_moe_layer_checks as checks


def test_empty_batch_beside_rows(bfq):
    """A batch without tokens, its rows in a buffer of any size. The places of no pairs are an empty tensor, whose
    address is NULL: without pairs both orders of rows are the same."""
    for places in (None, checks.P):
        assert checks.combine(bfq, T=0, places=places, R=8) == bfq.BFQ_OK
        assert checks.combine(bfq, T=0, places=places, R=3, w=None, base=None, ckpt=None, cs=None) == bfq.BFQ_OK
        assert checks.combine_bwd(bfq, T=0, places=places, R=8) == bfq.BFQ_OK
        assert checks.dispatch(bfq, T=0, places=places, x=None, R=8) == bfq.BFQ_OK
    assert torch.empty((0, 2), dtype=torch.int32).data_ptr() == 0
    # with tokens, rows in pair order are one a pair
    assert checks.combine(bfq, places=None, R=9) == checks.combine_bwd(bfq, places=None, R=9) == bfq.BFQ_ERR_SHAPE

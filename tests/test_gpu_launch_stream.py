"""GPU tests of the allocating conveniences' `stream` argument: workspaces and outputs of a call belong
to the stream that it launches on."""
import pytest
import torch

from block_scaled_w8a8_amd import synth

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _randn(seed, *shape):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return torch.randn(shape, generator=g, device=DEV)


def _jobs(bfq, count):
    """Calls that need a workspace, each a function of the stream."""
    M, K, F = 40, 2048, 1024
    qw, sw = bfq.quant_weight_blocks(_randn(1, 2 * F, K) * 0.02)
    gated = bfq.bfq_gated_select_tile(M, F, K)
    gated.split_k = 4
    dense = bfq.bfq_tile.from_dict({**bfq.bfq_get_tile_candidate(0).as_dict(), "split_k": 4})

    def job(i):
        x = synth.activations(M, K, seed=10 + i).to(DEV)
        qa, sa = bfq.quant_tokens(x)
        r, y, dn = _randn(20 + i, 300, 1544), _randn(30 + i, 300, 1544).bfloat16(), _randn(40 + i, 300, 1544).bfloat16()
        w = (1 + 0.1 * _randn(50 + i, 1544)).bfloat16()

        def call(stream):
            g = bfq.norm_residual_backward(r, y=y, w_post=w, w_pre=w, d_normed=dn, stream=stream)
            return (bfq.gated_gemm(qa, sa, qw, sw, tile=gated, stream=stream),
                    *bfq.gated_gemm(qa, sa, qw, sw, tile=gated, codes=True, keep_preact=True, stream=stream),
                    bfq.block_gemm(qa, sa, qw, sw, tile=dense, stream=stream),
                    *bfq.quant_tokens(x, stream=stream), *(g[k] for k in sorted(g)))
        return call
    return [job(i) for i in range(count)]


@pytest.mark.parametrize("raw", [False, True])
def test_calls_on_given_streams(bfq, raw):
    """Calls in flight on three streams, given as such or as raw handles, equal those made one by one."""
    jobs = _jobs(bfq, 3)
    want = [job(None) for job in jobs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in jobs]
    for _ in range(6):
        got = [job(s.cuda_stream if raw else s) for job, s in zip(jobs, streams)]
        torch.cuda.synchronize()
        for w, g in zip(want, got):
            assert len(w) == len(g) and all(torch.equal(a, b) for a, b in zip(w, g))


def test_workspace_is_not_given_out_on_the_callers_stream(bfq, monkeypatch):
    """The block that held a side stream's workspace does not go to the caller's next allocation."""
    used = []
    for name in ("bfq_gated_gemm", "bfq_norm_residual_backward", "bfq_block_gemm"):
        def launch(*a, inner=getattr(bfq, name), **kw):
            used.append((kw["workspace"].data_ptr(), kw["workspace"].numel()))
            return inner(*a, **kw)
        monkeypatch.setattr(bfq, name, launch)
    (job,) = _jobs(bfq, 1)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    job(side)
    mine = [torch.empty(n, dtype=torch.uint8, device=DEV) for _, n in used for _ in range(4)]
    torch.cuda.synchronize()
    assert len(used) == 4 and not {p for p, _ in used} & {t.data_ptr() for t in mine}


def test_captured_calls_on_a_forked_stream(bfq):
    """A capture that forks to a side stream, launches there and joins, replayed with eager work."""
    jobs = _jobs(bfq, 2)
    want = [job(None) for job in jobs]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cur = torch.cuda.current_stream()
        side.wait_stream(cur)
        forked = jobs[0](side)
        own = jobs[1](None)
        cur.wait_stream(side)
    for _ in range(4):
        for t in forked + own:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        jobs[0](None)
        torch.ones(1 << 20, device=DEV).sum()
        torch.cuda.synchronize()
        for w, g in zip(want, (forked, own)):
            assert all(torch.equal(a, b) for a, b in zip(w, g))

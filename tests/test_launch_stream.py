"""CPU tests of the allocating conveniences' `stream` argument: everything that such a call allocates
is allocated under the stream that it launches on. The caching allocator gives a freed block out again
at once to allocations under the stream that it came from, so a workspace from the caller's stream
would be shared with whatever the caller allocates next while the launch still uses it. Streams, the
allocator's calls and the launches are stand-ins here; which tensors the calls make is the real code."""
import contextlib

import pytest
import torch

LAUNCHES = ("bfq_quant_tokens", "bfq_quant_weight_blocks", "bfq_moe_align", "bfq_moe_block_gemm",
            "bfq_pack_weights", "bfq_block_gemm", "bfq_gated_gemm", "bfq_gated_backward",
            "bfq_transpose_weights", "bfq_norm_residual", "bfq_norm_residual_backward")


class _Stream:
    def __init__(self, handle):
        self.cuda_stream = handle


@pytest.fixture
def streams(bfq, monkeypatch):
    """Records (kind, stream handle) of every allocation, launch and hand-over."""
    caller, log, external = _Stream(11), [], {0: _Stream(0)}
    now = [caller]

    @contextlib.contextmanager
    def under(s):
        now.append(s)
        yield
        now.pop()

    def seen(kind, fn):
        def call(*a, **kw):
            log.append((kind, now[-1].cuda_stream))
            return fn(*a, **kw)
        return call
    bfq._torch_module()
    monkeypatch.setattr(torch.cuda, "is_initialized", lambda: True)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: now[-1])
    monkeypatch.setattr(torch.cuda, "default_stream", lambda *a: external[0])
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda h, *a: external.setdefault(h, _Stream(h)))
    monkeypatch.setattr(torch.cuda, "stream", under)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: now[-1].cuda_stream, raising=False)
    monkeypatch.setattr(torch, "empty", seen("alloc", torch.empty))
    monkeypatch.setattr(torch, "empty_like", seen("alloc", torch.empty_like))
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: log.append(("keep", s.cuda_stream)), raising=False)
    for name in LAUNCHES:
        def launch(*a, stream=None, **kw):
            log.append(("launch", bfq._stream(stream)))
        monkeypatch.setattr(bfq, name, launch)
    return log


def _calls(bfq):
    z, u8 = torch.zeros, torch.uint8
    M, F, K, E = 8, 256, 512, 4
    bf = torch.bfloat16
    a, sa = z((M, K), dtype=u8), z((M, K // 128))
    w, sw = z((2 * F, K), dtype=u8), z((2 * F // 128, K // 128))
    y, v = z((M, K), dtype=bf), z(K, dtype=bf)
    pre, dh = z((M, 2 * F), dtype=bf), z((M, F), dtype=bf)
    split = bfq.bfq_gated_select_tile(M, F, K)
    split.split_k = 2
    dense = bfq.bfq_tile.from_dict({**bfq.bfq_get_tile_candidate(0).as_dict(), "split_k": 2})
    moe = bfq.bfq_tile.from_dict({**bfq.bfq_moe_get_tile_candidate(0).as_dict(), "split_k": 2})
    ids = z((M, 2), dtype=torch.int32)
    off, srt = z(E + 1, dtype=torch.int32), z(M * 2, dtype=torch.int32)
    return {
        "quant_tokens": (1, 2, lambda s: bfq.quant_tokens(y, stream=s)),
        "quant_tokens positional": (1, 2, lambda s: bfq.quant_tokens(y, bfq.BFQ_E4M3FN, 0, 1e-10, s)),
        "quant_weight_blocks": (1, 2, lambda s: bfq.quant_weight_blocks(z(256, 256), stream=s)),
        "moe_align": (1, 2, lambda s: bfq.moe_align(ids, E, stream=s)),
        "moe_block_gemm": (6, 1, lambda s: bfq.moe_block_gemm(a, sa, srt, off, 2, z((E, F, K), dtype=u8), z((E, 2, 4)),
                                                           tile=moe, stream=s)),
        "pack_weights": (1, 1, lambda s: bfq.pack_weights(w, stream=s)),
        "block_gemm": (4, 1, lambda s: bfq.block_gemm(a, sa, w, sw, tile=dense, stream=s)),
        "gated_gemm": (4, 3, lambda s: bfq.gated_gemm(a, sa, w, sw, codes=True, keep_preact=True, tile=split, stream=s)),
        "gated_gemm out": (4, 1, lambda s: bfq.gated_gemm(a, sa, w, sw, tile=split, stream=s)),
        "gated_backward": (2, 3, lambda s: bfq.gated_backward(pre, dh, codes=True, want_h=True, stream=s)),
        "transpose_weights": (2, 2, lambda s: bfq.transpose_weights(w, sw, stream=s)),
        "norm_residual": (3, 3, lambda s: bfq.norm_residual(y, y, w_pre=v, codes=True, stream=s)),
        "norm_residual_backward": (6, 5, lambda s: bfq.norm_residual_backward(
            y, y=y, w_post=v, w_pre=v, gate=v, gate_kind=bfq.BFQ_GATE_CHANNEL, d_normed=y, stream=s)),
    }


NAMES = ("quant_tokens", "quant_tokens positional", "quant_weight_blocks", "moe_align", "moe_block_gemm",
         "pack_weights", "block_gemm", "gated_gemm", "gated_gemm out", "gated_backward",
         "transpose_weights", "norm_residual", "norm_residual_backward")
SPLIT = ("moe_block_gemm", "block_gemm", "gated_gemm", "gated_gemm out", "norm_residual_backward", "moe_align")


@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("given", ["stream", "handle", "default handle"])
def test_allocations_are_under_the_launch_stream(bfq, streams, name, given):
    operands, outputs, call = _calls(bfq)[name]
    streams.clear()
    handle = 0 if given == "default handle" else 22
    call(_Stream(handle) if given == "stream" else handle)
    made = [s for kind, s in streams if kind == "alloc"]
    assert len(made) == outputs + (name in SPLIT) and set(made) == {handle}
    assert [s for kind, s in streams if kind == "launch"] == [handle]
    # operands and outputs are the caller's to drop
    kept = [s for kind, s in streams if kind == "keep"]
    assert kept.count(handle) == operands > 0 and kept.count(11) == outputs and len(kept) == operands + outputs


@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("given", [None, 11])
def test_the_current_stream_needs_no_hand_over(bfq, streams, name, given):
    _, _, call = _calls(bfq)[name]
    streams.clear()
    call(given)
    assert {s for _, s in streams} == {11} and not any(kind == "keep" for kind, _ in streams)


def test_a_default_tile_is_reported_at_the_callers_line(bfq, streams, monkeypatch):
    monkeypatch.setattr(bfq, "_warned", set())
    z, u8 = torch.zeros, torch.uint8
    for stream in (None, 22):
        bfq._warned.clear()
        with pytest.warns(RuntimeWarning, match="default tile") as seen:
            bfq.block_gemm(z((8, 640), dtype=u8), z(8, 5), z((256, 640), dtype=u8), z(2, 5), stream=stream)
        assert seen[0].filename == __file__


def test_host_tensors_are_still_refused(bfq):
    """Without a GPU there is no stream to switch to, and the device check answers."""
    if torch.cuda.is_available():
        pytest.skip("the runtime is initialised")
    with pytest.raises(bfq.BfqArgumentError, match="device"):
        bfq.norm_residual(torch.zeros(2, 128), w_pre=torch.ones(128, dtype=torch.bfloat16), stream=5)

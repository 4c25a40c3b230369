"""CPU tests of the host side of the mixture-of-experts layer: every refusal of the C entry points
(before any launch, so host addresses stand in for device pointers), empty batches, the binding's
argument checks and the allocating conveniences' streams."""
import ctypes

import pytest
import torch

BUF = ctypes.create_string_buffer(1 << 16)
P = (ctypes.addressof(BUF) + 255) // 256 * 256       # an aligned address that nothing is read from
NAN, INF = float("nan"), float("inf")


def _caller(fn, defaults):
    def call(bfq, extra=None, **kw):
        kw = {**(extra or {}), **kw}
        assert set(kw) <= set(defaults), kw
        return getattr(bfq.lib, fn)(*{**defaults, **kw}.values(), None)
    return call


route = _caller("bfq_moe_route", dict(logits=P, dt=2, bias=P, T=4, E=16, topk=4, score=0, n_groups=4, topk_groups=2,
                                      renorm=1, scale=1.0, ids=P, w=P))
route_bwd = _caller("bfq_moe_route_backward", dict(logits=P, dt=2, ids=P, dw=P, T=4, E=16, topk=4, score=0, renorm=1,
                                                   scale=1.0, dl=P))
sort = _caller("bfq_moe_sort", dict(ids=P, T=4800, topk=8, E=16, off=P, srt=P, places=P, ws=P, wsb=1 << 20))
dispatch = _caller("bfq_moe_dispatch", dict(x=P, xdt=0, xs=None, xl=0, xld=0, places=P, rows=None, q=P, qdt=3, s=P,
                                            layout=0, ld=2, eps=1e-10, fmt=0, T=4, topk=2, K=256, R=8))
COPY = dict(xdt=3, xs=P, xld=2)
combine = _caller("bfq_moe_combine", dict(rows=P, rdt=0, w=P, places=P, ids=None, E=0, base=P, out=P, odt=0, ckpt=P,
                                          cdt=3, cs=P, eps=1e-10, T=4, topk=2, K=256, R=8))
combine_bwd = _caller("bfq_moe_combine_backward", dict(dout=P, ddt=0, w=P, rows=P, rdt=0, rs=None, places=P, ids=None,
                                                       E=0, d_rows=P, q=P, qdt=3, s=P, layout=0, ld=2, eps=1e-10,
                                                       fmt=0, dw=P, T=4, topk=2, K=256, R=8))
ckpt = _caller("bfq_gated_checkpoint", dict(pre=P, act=0, h=P, q=P, qdt=3, s=P, layout=0, ld=2, eps=1e-10, fmt=0, ckpt=P,
                                            cdt=3, cs=P, live=P, M=4, F=256))
ckpt_bwd = _caller("bfq_gated_checkpoint_backward", dict(ckpt=P, cdt=3, cs=P, dh=P, act=0, dpre=P, q=P, qdt=3, s=P,
                                                         layout=0, ld=4, eps=1e-10, fmt=0, h=P, live=P, M=4, F=256))


def _refuses(bfq, call, status, *cases):
    for kw in cases:
        assert call(bfq, **kw) == status, kw
        assert bfq.last_error()


def test_route_refusals(bfq):
    E = bfq
    for call, needed in ((route, ("logits", "ids", "w")), (route_bwd, ("logits", "ids", "dw", "dl"))):
        _refuses(E, call, E.BFQ_ERR_NULL, *({n: None} for n in needed))
        _refuses(E, call, E.BFQ_ERR_DTYPE, dict(dt=3), dict(dt=5), dict(dt=77), dict(dt=-1))
        _refuses(E, call, E.BFQ_ERR_ARG, dict(score=2), dict(score=-1), dict(scale=NAN), dict(scale=INF), dict(scale=-INF))
        _refuses(E, call, E.BFQ_ERR_SHAPE, dict(T=-1), dict(T=1 << 22), dict(E=0), dict(E=1024), dict(topk=0), dict(topk=17),
                 dict(E=-1))
        _refuses(E, call, E.BFQ_ERR_ALIGN, *({n: P + 2} for n in needed))
        assert call(E, T=0, **{n: None for n in needed}) == E.BFQ_OK
    _refuses(E, route, E.BFQ_ERR_SHAPE, dict(E=256, topk=65, n_groups=1, topk_groups=1), dict(n_groups=0), dict(n_groups=3),
             dict(topk_groups=0), dict(topk_groups=5), dict(topk_groups=1, topk=5), dict(E=130, n_groups=65, topk_groups=60),
             dict(n_groups=-4))
    _refuses(E, route, E.BFQ_ERR_ALIGN, dict(bias=P + 1), dict(dt=0, logits=P + 1))
    assert route(E, T=0, bias=None) == E.BFQ_OK


def test_sort_refusals(bfq):
    E = bfq
    _refuses(E, sort, E.BFQ_ERR_NULL, *({n: None} for n in ("ids", "off", "srt", "places")))
    _refuses(E, sort, E.BFQ_ERR_SHAPE, dict(T=-1), dict(topk=0), dict(E=0), dict(E=1024), dict(T=1 << 28), dict(T=1 << 62))
    _refuses(E, sort, E.BFQ_ERR_ALIGN, *({n: P + 2} for n in ("ids", "off", "srt", "places", "ws")))
    need = E.bfq_moe_sort_workspace_bytes(4800, 8, 16)
    assert need == 38 * 17 * 4                      # 38 workgroups' histograms
    _refuses(E, sort, E.BFQ_ERR_WORKSPACE, dict(ws=None), dict(wsb=need - 1), dict(ws=None, wsb=0))
    assert sort(E, T=0, off=None) == E.BFQ_ERR_NULL   # an empty batch still writes the offsets


def test_sort_workspace_sizes(bfq):
    w = bfq.bfq_moe_sort_workspace_bytes
    assert w(1024, 8, 256) == 0 and w(0, 8, 256) == 0 and w(-1, 8, 256) == 0 and w(5, 0, 4) == 0 and w(5, 2, 0) == 0
    assert w(1025, 8, 256) == 9 * 257 * 4
    assert w(8192, 8, 256) == 64 * 257 * 4
    assert w(1 << 22, 64, 1023) == 256 * 1024 * 4     # never more than 256 workgroups
    assert w(1 << 62, 64, 1023) == 0                  # a batch that the sort refuses


def test_dispatch_refusals(bfq):
    E = bfq
    _refuses(E, dispatch, E.BFQ_ERR_NULL, dict(x=None), dict(places=None), dict(q=None, s=None), dict(s=None), dict(q=None),
             dict(xs=P), dict(COPY, xs=None), dict(COPY, rows=P), dict(COPY, q=None, s=None), dict(COPY, q=None, s=None, rows=P))
    _refuses(E, dispatch, E.BFQ_ERR_DTYPE, dict(xdt=1), dict(xdt=2), dict(xdt=5), dict(xdt=-1), dict(qdt=0), dict(qdt=5),
             dict(COPY, qdt=4), dict(COPY, xdt=4))
    _refuses(E, dispatch, E.BFQ_ERR_SHAPE, dict(T=-1), dict(T=1 << 22), dict(topk=0), dict(topk=65), dict(K=0), dict(K=-128),
             dict(K=136, ld=2), dict(K=252), dict(K=1 << 24), dict(R=-1), dict(R=1 << 31), dict(ld=1), dict(layout=1, ld=7),
             dict(layout=2, fmt=1, R=6, ld=7), dict(ld=1 << 41), dict(COPY, xld=1), dict(COPY, xl=1, xld=3), dict(COPY, xld=1 << 41),
             dict(COPY, xl=2, layout=2, fmt=1, ld=8, xld=3), dict(rows=P, q=None, s=None, K=12))
    _refuses(E, dispatch, E.BFQ_ERR_ARG, dict(layout=3), dict(layout=2, ld=8), dict(fmt=2), dict(eps=0.0), dict(eps=NAN), dict(eps=INF),
             dict(COPY, xl=2, xld=4), dict(COPY, layout=2, fmt=1, ld=8), dict(COPY, xl=7), dict(eps=-1.0))
    _refuses(E, dispatch, E.BFQ_ERR_ALIGN, dict(x=P + 8), dict(q=P + 8), dict(rows=P + 2), dict(s=P + 2), dict(places=P + 1),
             dict(COPY, xs=P + 2))
    assert dispatch(E, T=0, R=0, x=None, places=None, q=None, s=None) == E.BFQ_OK


def test_no_rows(bfq):
    """A GPU that was given no row: tensors over rows may be missing, and nothing is to be written to them."""
    E = bfq
    assert dispatch(E, R=0, q=None, s=None) == E.BFQ_OK and dispatch(E, COPY, R=0, q=None, s=None) == E.BFQ_OK
    _refuses(E, dispatch, E.BFQ_ERR_NULL, dict(R=0, x=None), dict(R=0, places=None))
    _refuses(E, combine, E.BFQ_ERR_NULL, dict(R=0, rows=None, out=None))
    _refuses(E, combine_bwd, E.BFQ_ERR_NULL, dict(R=0, dout=None))
    assert combine_bwd(E, R=0, rows=None, d_rows=None, q=None, s=None, dw=None) == E.BFQ_OK


def test_combine_refusals(bfq):
    E = bfq
    pair = dict(places=None, ids=P, E=16)
    _refuses(E, combine, E.BFQ_ERR_NULL, dict(rows=None), dict(out=None), dict(ckpt=None), dict(cs=None))
    _refuses(E, combine, E.BFQ_ERR_DTYPE, dict(rdt=3), dict(odt=4), dict(rdt=-1), dict(odt=77), dict(cdt=0), dict(cdt=5))
    _refuses(E, combine, E.BFQ_ERR_SHAPE, dict(T=-1), dict(T=1 << 22), dict(topk=0), dict(topk=65), dict(K=0), dict(K=12, ckpt=None, cs=None),
             dict(K=136), dict(K=1 << 24), dict(R=-1), dict(R=1 << 31), dict(pair, R=9), dict(pair, R=7), dict(pair, E=0),
             dict(pair, E=-5), dict(places=None, R=9))
    _refuses(E, combine, E.BFQ_ERR_ARG, dict(ids=P, E=16), dict(eps=0.0), dict(eps=NAN))
    _refuses(E, combine, E.BFQ_ERR_ALIGN, dict(rows=P + 8), dict(out=P + 4), dict(base=P + 8), dict(ckpt=P + 8), dict(cs=P + 2),
             dict(w=P + 2), dict(places=P + 2), dict(pair, ids=P + 1))
    assert combine(E, T=0, R=0, rows=None, out=None, ckpt=None, cs=None, w=None, base=None) == E.BFQ_OK


def test_combine_backward_refusals(bfq):
    E = bfq
    pair, codes = dict(places=None, ids=P, E=16), dict(rdt=3, rs=P)
    _refuses(E, combine_bwd, E.BFQ_ERR_NULL, dict(dout=None), dict(q=None), dict(s=None), dict(rows=None), dict(dw=None),
             dict(rows=None, dw=None, q=None, s=None, d_rows=None), dict(rs=P), dict(codes, rs=None))
    _refuses(E, combine_bwd, E.BFQ_ERR_DTYPE, dict(ddt=1), dict(ddt=3), dict(ddt=-1), dict(rdt=5), dict(rdt=77), dict(qdt=2))
    _refuses(E, combine_bwd, E.BFQ_ERR_SHAPE, dict(T=-1), dict(T=1 << 22), dict(topk=0), dict(topk=65), dict(K=0), dict(K=136),
             dict(codes, K=136, q=None, s=None), dict(K=1 << 24), dict(R=-1), dict(R=1 << 31), dict(pair, R=9), dict(pair, E=0), dict(ld=1),
             dict(layout=1, ld=7), dict(layout=2, fmt=1, R=5, ld=7))
    _refuses(E, combine_bwd, E.BFQ_ERR_ARG, dict(ids=P, E=16), dict(layout=3), dict(layout=2, ld=8), dict(fmt=2), dict(eps=0.0))
    _refuses(E, combine_bwd, E.BFQ_ERR_ALIGN, dict(dout=P + 8), dict(rows=P + 8), dict(d_rows=P + 8), dict(q=P + 4), dict(s=P + 2),
             dict(codes, rs=P + 2), dict(w=P + 2), dict(dw=P + 2), dict(places=P + 2))
    assert combine_bwd(E, T=0, R=0, dout=None, rows=None, d_rows=None, q=None, s=None, dw=None) == E.BFQ_OK


def test_checkpoint_refusals(bfq):
    E = bfq
    _refuses(E, ckpt, E.BFQ_ERR_NULL, dict(pre=None), dict(q=None), dict(s=None), dict(ckpt=None), dict(cs=None),
             dict(h=None, q=None, s=None, ckpt=None, cs=None))
    _refuses(E, ckpt_bwd, E.BFQ_ERR_NULL, dict(ckpt=None), dict(cs=None), dict(dh=None), dict(q=None), dict(s=None),
             dict(dpre=None, q=None, s=None, h=None))
    for call, ld in ((ckpt, 2), (ckpt_bwd, 4)):
        _refuses(E, call, E.BFQ_ERR_DTYPE, dict(cdt=0), dict(cdt=5), dict(qdt=1), dict(qdt=-1))
        _refuses(E, call, E.BFQ_ERR_SHAPE, dict(M=-1), dict(M=(1 << 24) - 4), dict(F=0), dict(F=64), dict(F=-128), dict(F=1 << 26),
                 dict(ld=ld - 1), dict(layout=1, ld=3), dict(layout=2, fmt=1, M=5, ld=7))
        _refuses(E, call, E.BFQ_ERR_ARG, dict(act=2), dict(act=-1), dict(layout=3), dict(layout=2, ld=8), dict(fmt=2), dict(eps=0.0),
                 dict(eps=NAN))
        _refuses(E, call, E.BFQ_ERR_ALIGN, dict(ckpt=P + 8), dict(cs=P + 2), dict(q=P + 8), dict(s=P + 2), dict(h=P + 8), dict(live=P + 2))
    _refuses(E, ckpt, E.BFQ_ERR_ALIGN, dict(pre=P + 8))
    _refuses(E, ckpt_bwd, E.BFQ_ERR_ALIGN, dict(dh=P + 8), dict(dpre=P + 8))
    assert ckpt(E, M=0, pre=None, h=None, q=None, s=None, ckpt=None, cs=None) == E.BFQ_OK
    assert ckpt_bwd(E, M=0, ckpt=None, cs=None, dh=None, dpre=None, q=None, s=None, h=None) == E.BFQ_OK


# --------------------------------------------------------------------------- the binding

def _t(*shape, dt=torch.bfloat16):
    return torch.zeros(shape, dtype=dt)


def _good(bfq):
    """One call an entry point whose arguments fit, with host tensors."""
    i32, f32, u8 = torch.int32, torch.float32, torch.uint8
    T, E, topk, K, F, R = 4, 16, 2, 256, 256, 8
    return {
        "bfq_moe_route": dict(logits=_t(T, E, dt=f32), topk_ids=_t(T, topk, dt=i32), topk_weights=_t(T, topk, dt=f32),
                              bias=_t(E, dt=f32)),
        "bfq_moe_route_backward": dict(logits=_t(T, E), topk_ids=_t(T, topk, dt=i32), d_weights=_t(T, topk, dt=f32),
                                       d_logits=_t(T, E)),
        "bfq_moe_sort": dict(topk_ids=_t(T, topk, dt=i32), E=E, expert_offsets=_t(E + 1, dt=i32), sorted_pairs=_t(T * topk, dt=i32),
                             pair_rows=_t(T, topk, dt=i32)),
        "bfq_moe_dispatch": dict(x=_t(T, K), pair_rows=_t(T, topk, dt=i32), rows=_t(R, K), q=_t(R, K, dt=u8),
                                 scales=_t(R, K // 128, dt=f32)),
        "bfq_moe_combine": dict(rows=_t(R, K), out=_t(T, K), topk=topk, weights=_t(T, topk, dt=f32), pair_rows=_t(T, topk, dt=i32),
                                base=_t(T, K), ckpt=_t(R, K, dt=u8), ckpt_scales=_t(R, K // 128, dt=f32)),
        "bfq_moe_combine_backward": dict(dout=_t(T, K), topk=topk, weights=_t(T, topk, dt=f32), rows=_t(R, K, dt=u8),
                                         rows_scales=_t(R, K // 128, dt=f32), pair_rows=_t(T, topk, dt=i32), d_rows=_t(R, K),
                                         q=_t(R, K, dt=u8), scales=_t(R, K // 128, dt=f32), d_weights=_t(T, topk, dt=f32)),
        "bfq_gated_checkpoint": dict(preact=_t(T, 2 * F), h=_t(T, F), q=_t(T, F, dt=u8), scales=_t(T, F // 128, dt=f32),
                                     ckpt=_t(T, 2 * F, dt=u8), ckpt_scales=_t(T, 2 * F // 128, dt=f32), live_rows=_t(1, dt=i32)),
        "bfq_gated_checkpoint_backward": dict(ckpt=_t(T, 2 * F, dt=u8), ckpt_scales=_t(T, 2 * F // 128, dt=f32), dh=_t(T, F),
                                              dpre=_t(T, 2 * F), q=_t(T, 2 * F, dt=u8), scales=_t(T, 2 * F // 128, dt=f32),
                                              h=_t(T, F), live_rows=_t(1, dt=i32)),
    }


@pytest.mark.parametrize("name", ["bfq_moe_route", "bfq_moe_route_backward", "bfq_moe_sort", "bfq_moe_dispatch", "bfq_moe_combine",
                                  "bfq_moe_combine_backward", "bfq_gated_checkpoint", "bfq_gated_checkpoint_backward"])
def test_binding_checks_every_tensor(bfq, name):
    """Fitting host tensors reach the device check; of each tensor another dtype, another size and a
    strided view are refused before it."""
    fn, good = getattr(bfq, name), _good(bfq)[name]
    with pytest.raises(bfq.BfqArgumentError, match="need a GPU tensor"):
        fn(**good)
    for arg, t in good.items():
        if not isinstance(t, torch.Tensor):
            continue
        for bad in (t.double(), torch.zeros([n + 1 for n in t.shape], dtype=t.dtype),
                    torch.zeros([2 * n for n in t.shape], dtype=t.dtype)[tuple(slice(None, None, 2) for _ in t.shape)], "text"):
            if isinstance(bad, torch.Tensor) and bad.dtype == t.dtype and (
                    bad.shape == t.shape if t.numel() == 1 else bad.shape != t.shape and arg in ("scales", "sorted_pairs")):
                continue                         # one element has no stride; these two may be larger
            with pytest.raises((bfq.BfqArgumentError, AttributeError)) as e:
                fn(**{**good, arg: bad})
            assert "GPU tensor" not in str(e.value), (arg, e.value)


def test_binding_pairs_of_arguments(bfq):
    g = _good(bfq)
    for name, gone, match in (("bfq_moe_dispatch", "scales", "go together"), ("bfq_moe_combine", "ckpt_scales", "go together"),
                              ("bfq_moe_combine_backward", "d_weights", "go together"),
                              ("bfq_moe_combine_backward", "rows_scales", "need rows_scales"),
                              ("bfq_gated_checkpoint", "ckpt", "go together")):
        with pytest.raises(bfq.BfqArgumentError, match=match):
            getattr(bfq, name)(**{**g[name], gone: None})
    with pytest.raises(bfq.BfqArgumentError, match="must be given"):
        bfq.bfq_moe_combine_backward(_t(4, 256), 2)


def test_conveniences_allocate_under_the_launch_stream(bfq, monkeypatch):
    """What an allocating call makes belongs to the stream it launches on; operands and outputs are
    marked as used by both."""
    import contextlib
    log, now = [], [11]

    class Stream:
        def __init__(self, h):
            self.cuda_stream = h

    @contextlib.contextmanager
    def under(s):
        now.append(s.cuda_stream)
        yield
        now.pop()

    def seen(fn):
        def call(*a, **kw):
            log.append(("alloc", now[-1]))
            return fn(*a, **kw)
        return call
    g = _good(bfq)
    bfq._torch_module()
    monkeypatch.setattr(torch.cuda, "is_initialized", lambda: True)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: Stream(now[-1]))
    monkeypatch.setattr(torch.cuda, "stream", under)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: now[-1], raising=False)
    monkeypatch.setattr(torch, "empty", seen(torch.empty))
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: log.append(("keep", s.cuda_stream)), raising=False)
    for name in g:
        monkeypatch.setattr(bfq, name, lambda *a, stream=None, **kw: log.append(("launch", bfq._stream(stream))))
    r, c, k, b = (g[n] for n in ("bfq_moe_route", "bfq_moe_combine", "bfq_gated_checkpoint", "bfq_moe_combine_backward"))
    big = torch.zeros((4800, 8), dtype=torch.int32)
    calls = [
        (2, 0, 2, lambda s: bfq.moe_route(r["logits"], 2, bias=r["bias"], stream=s)),
        (3, 0, 1, lambda s: bfq.moe_route_backward(r["logits"], r["topk_ids"], r["topk_weights"], stream=s)),
        (1, 1, 3, lambda s: bfq.moe_sort(big, 16, stream=s)),
        (2, 0, 1, lambda s: bfq.moe_dispatch(c["out"], c["pair_rows"], stream=s)),
        (2, 0, 2, lambda s: bfq.moe_dispatch(c["out"], c["pair_rows"], codes=True, stream=s)),
        (4, 0, 3, lambda s: bfq.moe_combine(c["rows"], 2, weights=c["weights"], pair_rows=c["pair_rows"], base=c["base"],
                                            ckpt_dtype=bfq.BFQ_INT8, stream=s)),
        (5, 0, 3, lambda s: bfq.moe_combine_backward(b["dout"], 2, weights=b["weights"], rows=b["rows"], rows_scales=b["rows_scales"],
                                                     pair_rows=b["pair_rows"], codes=True, stream=s)),
        (2, 0, 4, lambda s: bfq.gated_checkpoint(k["preact"], codes=True, live_rows=k["live_rows"], stream=s)),
        (3, 0, 2, lambda s: bfq.gated_checkpoint_backward(k["ckpt"], k["ckpt_scales"], k["h"], want_h=True, stream=s)),
    ]
    for operands, workspace, outputs, call in calls:
        log.clear()
        call(Stream(22))
        assert [h for kind, h in log if kind == "alloc"] == [22] * (outputs + workspace)
        assert [h for kind, h in log if kind == "launch"] == [22]
        kept = [h for kind, h in log if kind == "keep"]
        assert kept.count(22) == operands and kept.count(11) == outputs

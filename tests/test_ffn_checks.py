"""CPU tests of the feed-forward operators' host side: every refusal of the C entry points (before
any launch, so host addresses stand in for device pointers), the binding's argument checks, the
gated tile rule and the workspace sizes."""
import ctypes

import pytest
import torch

BUF = ctypes.create_string_buffer(1 << 16)
P = (ctypes.addressof(BUF) + 255) // 256 * 256       # an aligned address that nothing is read from


def _bs(a=128, b=128):
    return (ctypes.c_int32 * 2)(a, b)


def _gated(bfq, **kw):
    d = dict(a_q=P, a_scales=P, a_layout=0, a_ld=2, w_q=P, w_scales=P, w_layout=0, sfmt=0, act=0, out=P,
             out_scales=None, out_layout=0, out_ld=0, out_eps=1e-10, preact=None, M=4, F=256, K=256,
             bs=_bs(), in_dtype=bfq.BFQ_E4M3FN, out_dtype=bfq.BFQ_BF16, tile=None, ws=None, wsb=0)
    d.update(kw)
    return bfq.lib.bfq_gated_gemm(*d.values(), None)


def test_gated_gemm_refusals(bfq):
    E = bfq
    for name in ("a_q", "a_scales", "w_q", "w_scales", "out", "bs"):
        assert _gated(bfq, **{name: None}) == E.BFQ_ERR_NULL, name
    codes = dict(out_dtype=E.BFQ_E4M3FN, out_scales=P, out_ld=2)
    assert _gated(bfq, **{**codes, "out_scales": None}) == E.BFQ_ERR_NULL
    for dt in (E.BFQ_INT8, E.BFQ_BF16, 77):
        assert _gated(bfq, in_dtype=dt) == E.BFQ_ERR_DTYPE
    for dt in (E.BFQ_INT8, E.BFQ_INT32, 77):
        assert _gated(bfq, out_dtype=dt) == E.BFQ_ERR_DTYPE
    for kw in (dict(M=-1), dict(F=0), dict(F=64), dict(K=64), dict(K=0), dict(bs=_bs(1, 256)),
               dict(M=1 << 24), dict(F=1 << 26), dict(K=1 << 24, a_ld=1 << 17), dict(a_ld=1),
               dict(a_layout=1, a_ld=3), dict(a_ld=1 << 24), dict(M=1 << 22, F=1 << 18),
               dict(codes, out_ld=1), dict(codes, out_layout=1, out_ld=3),
               dict(codes, out_ld=1 << 41)):
        assert _gated(bfq, **kw) == E.BFQ_ERR_SHAPE, kw
    for kw in (dict(act=2), dict(act=-1), dict(w_layout=2), dict(sfmt=2), dict(a_layout=3),
               dict(a_layout=2, a_ld=4), dict(codes, out_eps=0.0), dict(codes, out_eps=float("nan")),
               dict(codes, out_layout=9), dict(codes, out_layout=2, out_ld=4)):
        assert _gated(bfq, **kw) == E.BFQ_ERR_ARG, kw
    for name in ("a_q", "w_q", "out"):
        assert _gated(bfq, **{name: P + 8}) == E.BFQ_ERR_ALIGN, name
    assert _gated(bfq, preact=P + 2) == E.BFQ_ERR_ALIGN
    assert _gated(bfq, a_scales=P + 2) == E.BFQ_ERR_ALIGN
    assert _gated(bfq, **{**codes, "out_scales": P + 1}) == E.BFQ_ERR_ALIGN
    # tiles: an unknown one, one of another scale format, a split past the K blocks
    t = bfq.bfq_gated_get_tile_candidate(0)
    bad = bfq.bfq_tile.from_dict({**t.as_dict(), "bn": 96})
    assert _gated(bfq, tile=ctypes.byref(bad)) == E.BFQ_ERR_TILE
    ue = next(c for c in (bfq.bfq_gated_get_tile_candidate(i, 0, 1)
                          for i in range(bfq.bfq_gated_num_tile_candidates(0, 1))) if c.sched == 3)
    assert _gated(bfq, tile=ctypes.byref(ue)) == E.BFQ_ERR_TILE
    for kw in (dict(split_k=3), dict(split_k=0), dict(group_m=0), dict(raster=2)):
        assert _gated(bfq, tile=ctypes.byref(bfq.bfq_tile.from_dict({**t.as_dict(), **kw}))) == E.BFQ_ERR_TILE, kw
    two = bfq.bfq_tile.from_dict({**t.as_dict(), "split_k": 2})
    n = bfq.bfq_gated_gemm_workspace_bytes(4, 256, 256, tile=two)
    assert n == 2 * 4 * 512 * 4
    assert _gated(bfq, tile=ctypes.byref(two)) == E.BFQ_ERR_WORKSPACE
    assert _gated(bfq, tile=ctypes.byref(two), ws=P, wsb=n - 1) == E.BFQ_ERR_WORKSPACE
    assert "required" in bfq.last_error()
    # an empty batch launches nothing
    assert _gated(bfq, M=0, a_q=None, a_scales=None, out=None) == E.BFQ_OK
    assert _gated(bfq, **{**codes, "M": 0, "out_scales": None, "out": None}) == E.BFQ_OK


def test_gated_queries(bfq):
    L = bfq.lib
    t = bfq.bfq_tile()
    for args, st in (((1, 256, 256, 0, 0, 0, None), bfq.BFQ_ERR_NULL), ((1, 256, 256, 4, 0, 0, ctypes.byref(t)), bfq.BFQ_ERR_DTYPE),
                     ((1, 100, 256, 0, 0, 0, ctypes.byref(t)), bfq.BFQ_ERR_SHAPE),
                     ((1 << 30, 256, 256, 0, 0, 0, ctypes.byref(t)), bfq.BFQ_ERR_SHAPE),
                     ((1, 256, 256, 0, 5, 0, ctypes.byref(t)), bfq.BFQ_ERR_ARG),
                     ((1, 256, 256, 0, 0, 5, ctypes.byref(t)), bfq.BFQ_ERR_ARG)):
        assert L.bfq_gated_select_tile(*args) == st, args
    assert bfq.bfq_gated_num_tile_candidates(3, 0) == 0
    n = bfq.bfq_gated_num_tile_candidates()
    assert L.bfq_gated_get_tile_candidate(0, 0, n, ctypes.byref(t)) == bfq.BFQ_ERR_ARG
    assert L.bfq_gated_get_tile_candidate(0, 0, -1, ctypes.byref(t)) == bfq.BFQ_ERR_ARG
    assert bfq.bfq_gated_gemm_workspace_bytes(0, 256, 256) == 0
    assert bfq.bfq_gated_gemm_workspace_bytes(1 << 30, 256, 256) == ctypes.c_size_t(-1).value


def test_gated_split_last_round_refusals(bfq):
    tiles = [bfq.bfq_gated_get_tile_candidate(i) for i in range(bfq.bfq_gated_num_tile_candidates())]
    codes = dict(out_dtype=bfq.BFQ_E4M3FN, out_scales=P, out_ld=2)
    for t in tiles:
        v2 = bfq.bfq_tile.from_dict({**t.as_dict(), "variant": 2})
        # a last round needs whole rounds before it: no workspace, and the next check is the alignment
        assert bfq.bfq_gated_gemm_workspace_bytes(4, 256, 256, tile=v2) == 0
        if t.variant == 1:
            assert _gated(bfq, tile=ctypes.byref(v2)) == bfq.BFQ_ERR_TILE       # strips have no such form
            continue
        for kw in (dict(split_k=2), dict(group_m=0), dict(raster=2)):
            bad = bfq.bfq_tile.from_dict({**v2.as_dict(), **kw})
            assert _gated(bfq, tile=ctypes.byref(bad)) == bfq.BFQ_ERR_TILE, kw
        if t.bn != 128:                              # codes need whole groups in a tile
            assert _gated(bfq, tile=ctypes.byref(v2), **codes) == bfq.BFQ_ERR_TILE
        M, F = 256 * t.bm + 1, t.bn if t.bn == 128 else 128
        n = bfq.bfq_gated_gemm_workspace_bytes(M, F, 7168, tile=v2)
        rest = -(-M // t.bm) * (F // t.bn) % 256
        assert n == rest * min(256 // rest, 16) * t.bm * 2 * t.bn * 4 > 0
        assert _gated(bfq, M=M, F=F, K=7168, a_ld=56, tile=ctypes.byref(v2)) == bfq.BFQ_ERR_WORKSPACE
        assert _gated(bfq, M=M, F=F, K=7168, a_ld=56, tile=ctypes.byref(v2), ws=P, wsb=n - 1) == bfq.BFQ_ERR_WORKSPACE


@pytest.mark.parametrize("wl", [0, 1])
@pytest.mark.parametrize("sfmt", [0, 1])
def test_gated_rule_names_compiled_tiles(bfq, wl, sfmt):
    """The rule's tile is a compiled one at every size, also for packed activation scales, and
    its workspace follows the documented formula."""
    for inv in (False, True):
        bfq.bfq_set_batch_invariant(inv)
        try:
            for M in (1, 2, 15, 16, 17, 32, 33, 64, 65, 128, 129, 200, 256, 511, 777, 1024, 2048, 4096, 30000):
                for F in (128, 256, 2048, 2304, 18432):
                    for K in (128, 512, 1536, 7168):
                        t = bfq.bfq_gated_select_tile(M, F, K, w_layout=wl, scale_fmt=sfmt)
                        assert 1 <= t.split_k <= max(1, K // 128 // 2) and t.bm > 0
                        assert not inv or t.split_k == 1
                        def kw(dt):
                            return dict(M=M, F=F, K=K, w_layout=wl, sfmt=sfmt, a_ld=K // 128, out_dtype=dt,
                                        out_scales=P, out_ld=F // 128)

                        for dt, codes in ((bfq.BFQ_BF16, False), (bfq.BFQ_E4M3FN, True)):
                            n = bfq.bfq_gated_gemm_workspace_bytes(M, F, K, dt, wl, sfmt)
                            tc = bfq.bfq_gated_select_tile(M, F, K, dt, wl, sfmt)
                            want = tc.split_k * M * 2 * F * 4 if tc.split_k > 1 or (codes and tc.bn != 128) else 0
                            if tc.variant == 2:      # the last round's tiles in parts that fill it
                                rest = -(-M // tc.bm) * (F // tc.bn) % 256
                                parts = min(256 // rest, K // 256, 16)
                                assert want == 0 and parts > 1 and not inv
                                want = rest * parts * tc.bm * 2 * tc.bn * 4
                                bad = tc.from_dict({**tc.as_dict(), "split_k": 2})
                                assert _gated(bfq, **kw(dt), tile=bad) == bfq.BFQ_ERR_TILE
                            assert n == want
                            # host pointers: refused for its missing workspace, or (none needed) for
                            # an alignment that is checked after the tile is known to be fine
                            if n:
                                assert _gated(bfq, **kw(dt)) == bfq.BFQ_ERR_WORKSPACE
                                if sfmt:
                                    assert _gated(bfq, **{**kw(dt), "a_layout": 2, "a_ld": M}) == bfq.BFQ_ERR_WORKSPACE
        finally:
            bfq.bfq_set_batch_invariant(False)


def test_gated_backward_and_transpose_refusals(bfq):
    E = bfq

    def bwd(**kw):
        d = dict(pre=P, dh=P, act=0, dpre=P, q=None, qd=E.BFQ_E4M3FN, scales=None, lay=0, ld=4, eps=1e-10,
                 fmt=0, h=None, M=4, F=256)
        d.update(kw)
        return E.lib.bfq_gated_backward(*d.values(), None)
    q = dict(q=P, scales=P)
    for kw in (dict(pre=None), dict(dh=None), dict(dpre=None), dict(q=P), dict(scales=P)):
        assert bwd(**kw) == E.BFQ_ERR_NULL, kw
    for kw in (dict(M=-1), dict(F=0), dict(F=12), dict(q, F=264), dict(M=1 << 24), dict(F=1 << 26),
               dict(q, ld=3), dict(q, lay=1, ld=3)):
        assert bwd(**kw) == E.BFQ_ERR_SHAPE, kw
    for kw in (dict(act=3), dict(q, eps=0.0), dict(q, fmt=2), dict(q, lay=5), dict(q, lay=2)):
        assert bwd(**kw) == E.BFQ_ERR_ARG, kw
    assert bwd(**dict(q, qd=E.BFQ_BF16)) == E.BFQ_ERR_DTYPE
    for kw in (dict(pre=P + 2), dict(dh=P + 8), dict(dpre=P + 4), dict(h=P + 2), dict(q, q=P + 8),
               dict(q, scales=P + 2)):
        assert bwd(**kw) == E.BFQ_ERR_ALIGN, kw
    assert bwd(M=0, pre=None, dh=None, dpre=None) == E.BFQ_OK

    def tr(w=P, s=P, N=128, K=128, dt=E.BFQ_E4M3FN, wt=P + (1 << 15), st=P):
        return E.lib.bfq_transpose_weights(w, s, N, K, dt, wt, st, None)
    assert tr(w=None) == tr(s=None) == tr(wt=None) == tr(st=None) == E.BFQ_ERR_NULL
    assert tr(dt=E.BFQ_BF16) == E.BFQ_ERR_DTYPE
    assert tr(N=64) == tr(K=100) == tr(N=-128) == tr(N=1 << 23) == tr(K=1 << 24) == E.BFQ_ERR_SHAPE
    assert tr(w=P + 8) == tr(st=P + 2) == E.BFQ_ERR_ALIGN
    assert tr(wt=P + 16) == E.BFQ_ERR_ARG
    assert tr(N=0) == E.BFQ_OK


def _norm(bfq, **kw):
    d = dict(y=P, r=P, rd=bfq.BFQ_BF16, w_post=P, gate=None, kind=0, alpha=1.0, w_pre=P, eps=1e-6, ro=P,
             normed=P, q=None, qd=bfq.BFQ_E4M3FN, group=128, scales=None, lay=0, ld=2, qeps=1e-10, fmt=0,
             M=4, K=256)
    d.update(kw)
    return bfq.lib.bfq_norm_residual(*d.values(), None)


def _norm_bwd(bfq, **kw):
    d = dict(y=P, r=P, rd=bfq.BFQ_BF16, w_post=P, gate=None, kind=0, alpha=1.0, w_pre=P, eps=1e-6, dn=P,
             dro=P, dr=P, dy=P, dwpre=None, dwpost=None, dgate=None, M=4, K=256, ws=None, wsb=0)
    d.update(kw)
    return bfq.lib.bfq_norm_residual_backward(*d.values(), None)


def test_norm_refusals(bfq):
    E = bfq
    q = dict(q=P, scales=P)
    for fn in (_norm, _norm_bwd):
        for kw in (dict(r=None), dict(kind=1), dict(gate=P), dict(kind=3), dict(y=None)):
            assert fn(bfq, **kw) == E.BFQ_ERR_NULL, kw
        for kw in (dict(M=-1), dict(K=0), dict(K=12), dict(K=16392), dict(M=1 << 24)):
            assert fn(bfq, **kw) == E.BFQ_ERR_SHAPE, kw
        for kw in (dict(kind=4, gate=P), dict(kind=-1, gate=P), dict(eps=0.0), dict(eps=-1.0), dict(eps=float("nan")),
                   dict(eps=float("inf"))):
            assert fn(bfq, **kw) == E.BFQ_ERR_ARG, kw
        for dt in (E.BFQ_FP16, E.BFQ_INT8):
            assert fn(bfq, rd=dt) == E.BFQ_ERR_DTYPE
        for kw in (dict(y=P + 8), dict(r=P + 2), dict(w_post=P + 2), dict(w_pre=P + 8),
                   dict(kind=1, gate=P + 2), dict(kind=2, gate=P + 1)):
            assert fn(bfq, **kw) == E.BFQ_ERR_ALIGN, kw
    for kw in (dict(ro=None), dict(normed=None), dict(w_pre=None), dict(q=P), dict(scales=P),
               dict(y=None, w_post=None), dict(y=None, w_post=None, ro=None, w_pre=None, normed=None)):
        assert _norm(bfq, **kw) == E.BFQ_ERR_NULL, kw
    for kw in (dict(q, K=264, group=264), dict(q, group=64), dict(q, group=0), dict(q, ld=1),
               dict(q, lay=1, ld=3)):
        assert _norm(bfq, **kw) == E.BFQ_ERR_SHAPE, kw
    for kw in (dict(q, qeps=0.0), dict(q, fmt=7), dict(q, lay=4), dict(q, lay=2, ld=4),
               dict(q, lay=2, ld=4, fmt=1, group=256)):
        assert _norm(bfq, **kw) == E.BFQ_ERR_ARG, kw
    assert _norm(bfq, **dict(q, qd=E.BFQ_BF16)) == E.BFQ_ERR_DTYPE
    for kw in (dict(ro=P + 8), dict(normed=P + 2), dict(q, q=P + 8), dict(q, scales=P + 2)):
        assert _norm(bfq, **kw) == E.BFQ_ERR_ALIGN, kw
    assert _norm(bfq, M=0, y=None, r=None, ro=None, normed=None) == E.BFQ_OK
    for kw in (dict(dr=None), dict(dy=None), dict(dn=None), dict(w_pre=None), dict(w_post=None, dwpost=P),
               dict(dgate=P), dict(w_pre=None, dn=None, dwpre=P)):
        assert _norm_bwd(bfq, **kw) == E.BFQ_ERR_NULL, kw
    for kw in (dict(dn=P + 8), dict(dro=P + 2), dict(dr=P + 8), dict(dy=P + 8), dict(dwpre=P + 2),
               dict(dwpost=P + 1), dict(kind=1, gate=P, dgate=P + 2)):
        assert _norm_bwd(bfq, **kw) == E.BFQ_ERR_ALIGN, kw
    n = bfq.bfq_norm_residual_backward_workspace_bytes(4, 256)
    assert n == 4 * 2 * 256 * 4
    for kw in (dict(dwpre=P), dict(dwpost=P), dict(kind=1, gate=P, dgate=P)):
        assert _norm_bwd(bfq, **kw) == E.BFQ_ERR_WORKSPACE
        assert _norm_bwd(bfq, **kw, ws=P, wsb=n - 1) == E.BFQ_ERR_WORKSPACE
    assert _norm_bwd(bfq, M=0, y=None, r=None, dr=None, dy=None, dn=None, dro=None) == E.BFQ_OK
    assert bfq.bfq_norm_residual_backward_workspace_bytes(1 << 30, 256) == ctypes.c_size_t(-1).value


def _err(bfq, match, fn, *a, **kw):
    with pytest.raises(bfq.BfqArgumentError, match=match):
        fn(*a, **kw)


def test_binding_checks(bfq):
    """Host tensors of the right form fail the device check last; anything else before it."""
    z = torch.zeros
    M, F, K = 4, 256, 512
    a, sa = z((M, K), dtype=torch.uint8), z((M, K // 128))
    w, sw = z((2 * F, K), dtype=torch.uint8), z((2 * F // 128, K // 128))
    out, pre = z((M, F), dtype=torch.bfloat16), z((M, 2 * F), dtype=torch.bfloat16)
    g = bfq.bfq_gated_gemm
    _err(bfq, "device", g, a, sa, w, sw, out, preact=pre)
    _err(bfq, "as many up rows", g, a, sa, w[:-1], sw, out)
    _err(bfq, "dtype int8", g, a.view(torch.int8), sa, w, sw, out)
    _err(bfq, "shape", g, a, sa, w, sw, out[:, :128])
    _err(bfq, "strides", g, a, sa, w, sw, pre[:, :F])
    _err(bfq, "elements", g, a, sa, w, sw[:2], out)
    _err(bfq, "needs at least", g, a, sa[:, :2], w, sw, out)
    _err(bfq, "out_scales goes with", g, a, sa, w, sw, out, out_scales=z((M, 2)))
    codes = z((M, F), dtype=torch.uint8)
    _err(bfq, "out_scales goes with", g, a, sa, w, sw, codes)
    _err(bfq, "needs at least", g, a, sa, w, sw, codes, out_scales=z((M, 1)))
    _err(bfq, "device", g, a, sa, w, sw, codes, out_scales=z((M, 2)))
    _err(bfq, "preact", g, a, sa, w, sw, out, preact=pre[:, :F])
    _err(bfq, "workspace", g, a, sa, w, sw, out, workspace=z(8, dtype=torch.uint8), workspace_bytes=64)
    b = bfq.bfq_gated_backward
    dh = out.clone()
    _err(bfq, "device", b, pre, dh, dpre=pre.clone())
    _err(bfq, "preact has shape", b, pre[:, :F], dh, dpre=pre)
    _err(bfq, "dtype float32", b, pre, dh.float(), dpre=pre)
    _err(bfq, "go together", b, pre, dh, q=z((M, 2 * F), dtype=torch.uint8))
    _err(bfq, "needs at least", b, pre, dh, q=z((M, 2 * F), dtype=torch.uint8), scales=z((M, 2)))
    _err(bfq, "h has shape", b, pre, dh, h=pre)
    t = bfq.bfq_transpose_weights
    _err(bfq, "device", t, w, sw, z((K, 2 * F), dtype=torch.uint8), sw)
    _err(bfq, "wt_q has shape", t, w, sw, codes, sw)
    _err(bfq, "different code types", t, w, sw, z((K, 2 * F), dtype=torch.int8), sw)
    n = bfq.bfq_norm_residual
    r, y, v = z((M, K)), z((M, K), dtype=torch.bfloat16), z(K, dtype=torch.bfloat16)
    full = dict(y=y, w_pre=v, res_out=r.clone(), normed=y.clone())
    _err(bfq, "device", n, r, **full)
    _err(bfq, "residual has dtype", n, r.half(), **full)
    _err(bfq, "res_out has dtype", n, r, **{**full, "res_out": y})
    _err(bfq, "y has shape", n, r, **{**full, "y": y[:2]})
    _err(bfq, "w_pre has dtype", n, r, **{**full, "w_pre": v.float()})
    _err(bfq, "w_post holds", n, r, **full, w_post=v[:8])
    _err(bfq, "gate goes with", n, r, **full, gate=v)
    _err(bfq, "gate goes with", n, r, **full, gate_kind=bfq.BFQ_GATE_TOKEN)
    _err(bfq, "gate holds", n, r, **full, gate=v, gate_kind=bfq.BFQ_GATE_TOKEN)
    _err(bfq, "gate has|gate must|expected", n, r, **full, gate=v, gate_kind=bfq.BFQ_GATE_FULL)
    _err(bfq, "go together", n, r, **full, q=z((M, K), dtype=torch.uint8))
    _err(bfq, "strides", n, z((M, 2 * K))[:, :K], **full)
    nb = bfq.bfq_norm_residual_backward
    full = dict(y=y, w_pre=v, d_normed=y, d_y=y.clone())
    _err(bfq, "device", nb, r, r.clone(), **full)
    _err(bfq, "d_res has dtype", nb, r, y, **full)
    _err(bfq, "d_res_out has dtype", nb, r, r, **full, d_res_out=y)
    _err(bfq, "d_w_pre has dtype", nb, r, r, **full, d_w_pre=v)
    _err(bfq, "d_gate has dtype", nb, r, r, **full, gate=v, gate_kind=1, d_gate=v)
    _err(bfq, "d_gate holds", nb, r, r, **full, gate=v, gate_kind=1, d_gate=z(M))

"""GPU tests of the mixture-of-experts layer's operators together, as a layer uses them: forward in both
row orders, backward to the tokens and the logits, on several streams, in a captured graph, with a part
of the experts."""
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
T, E, TOPK, K, F = 192, 8, 2, 512, 256
CODE = 2.0 ** -4                  # half a step of an e4m3 code, relative to its value


def _randn(seed, *shape):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return torch.randn(shape, generator=g, device=DEV)


class Layer:
    def __init__(self, bfq, experts=E):
        self.bfq = bfq
        w1, w2 = _randn(1, experts, 2 * F, K) * 0.05, _randn(2, experts, K, F) * 0.05
        self.E = experts

        def stack(w):
            q, s = zip(*(bfq.quant_weight_blocks(w[e]) for e in range(experts)))
            t, ts = zip(*(bfq.transpose_weights(a, b) for a, b in zip(q, s)))
            return torch.stack(q), torch.stack(s), torch.stack(t), torch.stack(ts)
        self.q1, self.s1, self.t1, self.ts1 = stack(w1)
        self.q2, self.s2, self.t2, self.ts2 = stack(w2)
        self.tile = bfq.bfq_moe_get_tile_candidate(0)      # one tile for every batch: equal sums

    def gemm(self, q, s, srt, off, topk, wq, ws, stream=None):
        return self.bfq.moe_block_gemm(q, s, srt, off, topk, wq, ws, tile=self.tile, stream=stream)

    def forward_pairs(self, x, ids, w, base=None):
        b = self.bfq
        off, srt = b.moe_align(ids, self.E)
        xq, xs = b.quant_tokens(x)
        pre = self.gemm(xq, xs, srt, off, ids.shape[1], self.q1, self.s1)
        hq, hs, ck, cs = b.gated_checkpoint(pre, codes=True)
        y = self.gemm(hq, hs, srt, off, 1, self.q2, self.s2)
        return b.moe_combine(y, ids.shape[1], weights=w, topk_ids=ids, E=self.E, base=base)

    def forward(self, x, logits, base=None, stream=None, shift=0):
        b, s = self.bfq, stream
        ids, w = b.moe_route(logits, TOPK, renorm=True, stream=s)
        if shift:
            with torch.cuda.stream(s or torch.cuda.current_stream()):
                ids = ids - shift
        off, srt, at = b.moe_sort(ids, self.E, stream=s)
        q, sc = b.moe_dispatch(x, at, codes=True, stream=s)
        R = q.shape[0]
        with torch.cuda.stream(s or torch.cuda.current_stream()):
            seq = torch.arange(R, device=DEV, dtype=torch.int32)
        pre = self.gemm(q, sc, seq, off, 1, self.q1, self.s1, s)
        hq, hs, ck, cs = b.gated_checkpoint(pre, codes=True, live_rows=off[self.E:], stream=s)
        y = self.gemm(hq, hs, seq, off, 1, self.q2, self.s2, s)
        out, yq, ys = b.moe_combine(y, TOPK, weights=w, pair_rows=at, base=base, ckpt_dtype=b.BFQ_E4M3FN, stream=s)
        return out, dict(ids=ids, w=w, at=at, off=off, seq=seq, ck=ck, cs=cs, yq=yq, ys=ys, logits=logits)

    def backward(self, dout, k, stream=None):
        b, s = self.bfq, stream
        g = b.moe_combine_backward(dout, TOPK, weights=k["w"], rows=k["yq"], rows_scales=k["ys"], pair_rows=k["at"],
                                   codes=True, stream=s)
        dh = self.gemm(g["q"], g["scales"], k["seq"], k["off"], 1, self.t2, self.ts2, s)
        pq, ps = b.gated_checkpoint_backward(k["ck"], k["cs"], dh, codes=True, live_rows=k["off"][self.E:], stream=s)
        drows = self.gemm(pq, ps, k["seq"], k["off"], 1, self.t1, self.ts1, s)
        dx = b.moe_combine(drows, TOPK, pair_rows=k["at"], stream=s)
        dl = b.moe_route_backward(k["logits"], k["ids"], g["d_weights"], renorm=True, stream=s)
        return dx, dl, g["d_weights"]

    def exact(self, x, ids, w, base):
        """The layer in 64 bits on the weights that the codes stand for."""
        def values(q, s):
            return q.view(torch.float8_e4m3fn).double() * s.double().repeat_interleave(128, 1).repeat_interleave(128, 2)
        w1, w2 = values(self.q1, self.s1), values(self.q2, self.s2)
        out = torch.zeros(x.shape, dtype=torch.float64, device=DEV) if base is None else base.double()
        for e in range(self.E):
            pre = x @ w1[e].t()
            y = (torch.nn.functional.silu(pre[:, :F]) * pre[:, F:]) @ w2[e].t()
            out = out + ((ids == e) * w).sum(dim=1, keepdim=True) * y
        return out


def _inputs(seed, n=T, experts=E):
    return _randn(seed, n, K).bfloat16(), _randn(seed + 1, n, experts), _randn(seed + 2, n, K).bfloat16()


def test_both_orders_give_the_same_layer(bfq):
    layer = Layer(bfq)
    x, logits, base = _inputs(3)
    out, k = layer.forward(x, logits, base)
    assert torch.equal(out.view(torch.int16), layer.forward_pairs(x, k["ids"], k["w"], base).view(torch.int16))


@pytest.mark.parametrize("n", [1, 5, T])
def test_forward_and_gradients(bfq, n):
    """Against the layer in 64 bits with unquantized activations. Each set of codes on the way is off by at most
    half a step of 2^-4 of a value, so a result by about that a set: forward x and h (2), the tokens' gradient the
    checkpoint, the rows' gradient and dpre besides (5); a weight's gradient is a product with rows of 3 sets."""
    layer = Layer(bfq)
    x, logits, base = _inputs(5, n)
    out, k = layer.forward(x, logits, base)
    dout = (_randn(9, n, K) * 0.1).bfloat16()
    dx, dl, dw = layer.backward(dout, k)
    x64, w64 = x.double().requires_grad_(), k["w"].double().requires_grad_()
    ref = layer.exact(x64, k["ids"], w64, base)
    ref.backward(dout.double())
    moved = ref.detach() - base.double()
    rows = (out.double() - base.double() - moved).norm() / moved.norm()
    assert rows <= 2 * CODE + 2.0 ** -8 * float(ref.detach().norm() / moved.norm())
    assert (dx.double() - x64.grad).norm() <= 5 * CODE * x64.grad.norm()
    assert (dw.double() - w64.grad).norm() <= 3 * CODE * (dout.double().norm(dim=1) * moved.norm(dim=1)).norm() / float(k["w"].min())
    # the logits' gradient is the router's, of these weights' gradient
    l64 = logits.double().requires_grad_()
    s = torch.softmax(l64, dim=1).gather(1, k["ids"].long())
    ((s / s.sum(dim=1, keepdim=True)) * dw.double()).sum().backward()
    assert bool(((dl.double() - l64.grad).abs() <= 2.0 ** -24 * 256 * dw.double().abs().sum(dim=1, keepdim=True)).all())


def test_experts_in_two_halves_add_up(bfq):
    """Two GPUs' shares of the experts, each with the pairs that are its own: the sum of their layers."""
    whole = Layer(bfq)
    x, logits, _ = _inputs(7)
    out, k = whole.forward(x, logits)
    parts = []
    for lo in (0, E // 2):
        half = Layer(bfq)
        half.E = E // 2
        for n in ("q1", "s1", "q2", "s2"):
            setattr(half, n, getattr(whole, n)[lo:lo + E // 2].contiguous())
        ids, w = bfq.moe_route(logits, TOPK, renorm=True)
        ids = ids - lo
        off, _, at = bfq.moe_sort(ids, E // 2)
        live = int(off[E // 2])
        assert 0 < live < T * TOPK and int((at >= 0).sum()) == live
        y, kept = half.forward(x, logits, shift=lo)
        ref = half.exact(x.double(), ids, w.double(), None)
        assert (y.double() - ref).norm() <= (2 * CODE + 2.0 ** -8) * ref.norm()
        assert torch.equal(y.view(torch.int16), half.forward_pairs(x, ids, w).view(torch.int16))
        parts.append(y.double())
    # three roundings to bf16
    assert bool(((parts[0] + parts[1] - out.double()).abs() <= 2.0 ** -8 * (parts[0].abs() + parts[1].abs() + out.double().abs())).all())


@pytest.mark.parametrize("raw", [False, True])
def test_streams(bfq, raw):
    """Layers in flight on three streams equal those made one by one."""
    layer = Layer(bfq)
    data = [_inputs(20 + 5 * i, n) for i, n in enumerate((T, 40, 1))]
    douts = [(_randn(50 + i, *x.shape) * 0.1).bfloat16() for i, (x, _, _) in enumerate(data)]
    want = []
    for (x, l, b), d in zip(data, douts):
        out, k = layer.forward(x, l, b)
        want.append((out, *layer.backward(d, k)))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in data]
    for _ in range(4):
        got = []
        for (x, l, b), d, s in zip(data, douts, streams):
            if raw:                                        # the handle of the stream, where every call takes one
                ids, w = bfq.moe_route(l, TOPK, renorm=True, stream=s.cuda_stream)
                off, srt, at = bfq.moe_sort(ids, E, stream=s.cuda_stream)
                got.append((bfq.moe_combine(bfq.moe_dispatch(x, at, stream=s.cuda_stream), TOPK, weights=w, pair_rows=at,
                                            base=b, stream=s.cuda_stream),))
            else:
                out, k = layer.forward(x, l, b, stream=s)
                got.append((out, *layer.backward(d, k, stream=s)))
        torch.cuda.synchronize()
        for (x, l, b), w, g in zip(data, want, got):
            if raw:
                ids, wt = bfq.moe_route(l, TOPK, renorm=True)
                rows = x.unsqueeze(1).expand(-1, TOPK, -1).reshape(-1, K).contiguous()
                assert torch.equal(g[0], bfq.moe_combine(rows, TOPK, weights=wt, base=b))
            else:
                assert all(torch.equal(a, c) for a, c in zip(w, g))


@pytest.mark.parametrize("n", [3, T])
def test_graph_replays(bfq, n):
    """Forward and backward captured once, replayed on new inputs with eager work between."""
    layer = Layer(bfq)
    x, l, b = _inputs(70, n)
    dout = (_randn(75, n, K) * 0.1).bfloat16()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        out, k = layer.forward(x, l, b)
        layer.backward(dout, k)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, k = layer.forward(x, l, b)
        dx, dl, dw = layer.backward(dout, k)
    for i in range(4):
        nx, nl, nb = _inputs(80 + i, n)
        if i == 2:
            nl[:, 3:] = -float("inf")                      # three experts take everything
        x.copy_(nx)
        l.copy_(nl)
        b.copy_(nb)
        dout.copy_((_randn(90 + i, n, K) * 0.1).bfloat16())
        graph.replay()
        torch.cuda.synchronize()
        wout, wk = layer.forward(x, l, b)
        want = (wout, *layer.backward(dout, wk))
        torch.cuda.synchronize()
        assert all(torch.equal(a, c) for a, c in zip((out, dx, dl, dw), want)), i


def test_equal_calls_give_equal_bits(bfq):
    layer = Layer(bfq)
    x, l, b = _inputs(100)
    dout = (_randn(101, T, K) * 0.1).bfloat16()
    runs = []
    for _ in range(3):
        out, k = layer.forward(x, l, b)
        runs.append((out, *layer.backward(dout, k)))
    assert all(torch.equal(a, c) for r in runs[1:] for a, c in zip(runs[0], r))


def test_tokens_do_not_depend_on_the_batch(bfq):
    """The router, the combine and its gradient treat a token alike in any batch."""
    x, l, _ = _inputs(110)
    ids, w = bfq.moe_route(l, TOPK, renorm=True)
    rows = _randn(111, T * TOPK, K).bfloat16()
    out = bfq.moe_combine(rows, TOPK, weights=w)
    g = bfq.moe_combine_backward(x, TOPK, weights=w, rows=rows, codes=True)
    for a, b in ((0, 1), (17, 90), (191, 192)):
        i2, w2 = bfq.moe_route(l[a:b], TOPK, renorm=True)
        assert torch.equal(i2, ids[a:b]) and torch.equal(w2, w[a:b])
        part = rows[a * TOPK:b * TOPK]
        assert torch.equal(bfq.moe_combine(part, TOPK, weights=w2), out[a:b])
        g2 = bfq.moe_combine_backward(x[a:b], TOPK, weights=w2, rows=part, codes=True)
        assert torch.equal(g2["q"], g["q"][a * TOPK:b * TOPK]) and torch.equal(g2["d_weights"], g["d_weights"][a:b])


def test_readme_example(bfq):
    """The README's blocks run as they stand, one after the other."""
    import os
    import re
    text = open(os.path.join(os.path.dirname(__file__), "..", "README.md")).read()
    env = {}
    for block in re.findall(r"```python\n(.*?)```", text, re.S):
        exec(block, env)
    assert env["moe"].shape == env["dx_moe"].shape == (64, 7168) and env["dlogits"].shape == (64, 16)
    assert all(bool(env[n].float().isfinite().all()) and bool(env[n].any()) for n in ("moe", "dx_moe", "dlogits"))


def test_host_and_other_device_tensors_are_refused(bfq):
    x = torch.zeros((4, 256), dtype=torch.bfloat16, device=DEV)
    at = torch.zeros((4, 2), dtype=torch.int32)
    with pytest.raises(bfq.BfqArgumentError, match="need a GPU tensor"):
        bfq.moe_dispatch(x, at)

"""GPU tests of the router weights' gradient through a whole mixture-of-experts layer: what the combine keeps
of the rows in 8 bits, the combine's gradient from it, and the router's gradient from that."""
import pytest
import torch

import test_gpu_moe_layer as layers

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U = 2.0 ** -24
K, TOPK = layers.K, layers.TOPK


def _run(bfq, n):
    layer = layers.Layer(bfq)
    x, logits, base = layers._inputs(5, n)
    out, k = layer.forward(x, logits, base)
    dout = (layers._randn(9, n, K) * 0.1).bfloat16()
    _, dl, dw = layer.backward(dout, k)
    return layer, x, logits, k, dout, dl, dw.double()


def _wrong(ref):
    """Gradients that a test has to tell from ref."""
    return {"none": torch.zeros_like(ref), "negated": -ref, "pairs swapped": ref.flip(1)}


@pytest.mark.parametrize("n", [1, 5, layers.T])
def test_weights_gradient_from_the_kept_rows(bfq, n):
    """The products of the gradient with the rows that the kept codes stand for, in 64 bits. From codes to codes a
    thread multiplies 16 columns, then by their scale; 512 columns take half a wave: 17 roundings, 6 additions."""
    _, _, _, k, dout, _, dw = _run(bfq, n)
    rows = k["yq"].view(torch.float8_e4m3fn).double() * k["ys"].double().repeat_interleave(128, dim=1)
    terms = rows[k["at"].long()] * dout.double().unsqueeze(1)
    ref, tol = terms.sum(dim=2), terms.abs().sum(dim=2) * U * 23 * (1 + 64 * U)
    assert bool(((dw - ref).abs() <= tol).all())
    for what, bad in _wrong(ref).items():
        assert float(((bad - ref).abs() > tol).float().mean()) > 0.9, what


def test_weights_gradient_of_the_unquantized_layer(bfq):
    """Against the layer in 64 bits whose activations were never quantized. Three sets of codes (x, h and the kept
    rows) lie between, each off by at most half a step of 2^-4 of a value: a row is off by at most 3 of them in its
    norm, and over 384 pairs so are the products with gradients that have nothing to do with the error. The logits'
    gradient is linear in them."""
    layer, x, logits, k, dout, dl, dw = _run(bfq, layers.T)
    w64 = k["w"].double().requires_grad_()
    layer.exact(x.double(), k["ids"], w64, None).backward(dout.double())
    ref = w64.grad
    bound = 3 * layers.CODE
    assert (dw - ref).norm() <= bound * ref.norm()
    for what, bad in _wrong(ref).items():
        assert (bad - ref).norm() > 2 * bound * ref.norm(), what
    l64 = logits.double().requires_grad_()
    s = torch.softmax(l64, dim=1).gather(1, k["ids"].long())
    ((s / s.sum(dim=1, keepdim=True)) * ref).sum().backward()
    assert (dl.double() - l64.grad).norm() <= bound * l64.grad.norm()


def test_empty_batch(bfq):
    """No tokens: the layer runs through, forward and backward."""
    layer = layers.Layer(bfq)
    x, logits, base = layers._inputs(3, 0)
    out, k = layer.forward(x, logits, base)
    dx, dl, dw = layer.backward(x, k)
    assert out.shape == dx.shape == (0, K) and dl.shape == (0, layers.E) and dw.shape == (0, TOPK)
    # beside rows of a larger buffer
    rows = layers._randn(1, 8, K).bfloat16()
    at = torch.empty((0, TOPK), dtype=torch.int32, device=DEV)
    assert bfq.moe_combine(rows, TOPK, pair_rows=at).shape == (0, K)
    assert bfq.moe_combine_backward(x, TOPK, rows=rows, pair_rows=at)["d_weights"].shape == (0, TOPK)

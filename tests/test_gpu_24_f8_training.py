"""GPU test of the 8-bit training operators together, as one layer's training
step: residual and layer norm into an F8 tensor, the product with a weight in
square blocks, the output's gradient quantised both ways, both gradients of
the product (the weight's from the activation's 8-bit checkpoint, read
transposed), and the norm's gradient from its own checkpoint.  Every stage is
compared with fp64 arithmetic on that stage's own inputs; the chain is then
captured into a graph and replayed.  And the gradient of the layer as a whole,
against differences of its function in fp64."""
import os
import sys

import numpy as np
import pytest

import communication_tensor_gemm_amd as dg
from oracle import f8, parity

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import f8_linear  # noqa: E402

pytestmark = pytest.mark.gpu


def f64(t):
    import torch
    return t.to(torch.float64).cpu().numpy()


def bits(t):
    import torch
    return t.view(torch.uint8).cpu().numpy()


def values(pair, cols=None):
    return f8.values(bits(pair[0]), bits(pair[1]), cols)


def product_close(got, a, b, bias=None, C=None):
    D = a @ b.T + (0 if bias is None else bias[None]) + (0 if C is None else C)
    ok, worst, tight, _ = parity.check(got, D, np.linalg.norm(a, axis=1), np.linalg.norm(b, axis=1), 1.0, 0.0 if C is None else 1.0, C,
                                       "e4m3", "bf16", bias)
    assert ok and tight, worst


def layer(tokens=300, width=520, out=392):
    import torch
    g = torch.Generator(device="cuda").manual_seed(3)
    n = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    L = f8_linear.NormLinear(tokens, width, out, seed=1)
    return L, n(tokens, width).bfloat16(), n(tokens, width).bfloat16(), (n(tokens, out) * 0.1).bfloat16(), (n(tokens, width) * 0.1).bfloat16()


def test_every_stage():
    import torch
    L, x, r, dy, dh = layer()
    tokens, width, out = L.tokens, L.width, L.out
    y = L.forward(x, r)
    torch.cuda.synchronize()
    # the stream, the norm's two 8-bit outputs and the product
    h = (x.float() + r.float()).bfloat16()
    assert torch.equal(L.h, h)
    y64, n64, _, rstd = f8.layer_norm(f64(h), f64(L.norm_weight), f64(L.norm_bias), L.eps)
    for pair, v in ((L.act, y64), (L.kept, n64)):
        assert np.all(np.abs(values(pair, width) - v) <= 2.0 ** -4 * np.abs(v) * (1 + 1e-4) + 2.0 ** -9 * np.abs(v).max(-1, keepdims=True) / 224)
    product_close(f64(y), values(L.act), values(L.w8), f64(L.bias))
    w, wt = values(L.w8, width), values(L.w8_t, out)
    assert np.array_equal(w, wt.T) and np.all(np.abs(w - f64(L.weight)) <= 2.0 ** -4 * np.abs(w) * (1 + 2.0 ** -4) + 2.0 ** -10)
    dx = L.backward(dy, dh)
    torch.cuda.synchronize()
    assert np.array_equal(bits(L.dy8[0]), f8.quantize(f64(dy))[0])
    assert np.array_equal(bits(L.dy8_t[0]), f8.quantize(f64(dy).T)[0])
    assert np.array_equal(bits(L.act_t[0]), f8.quantize(values(L.act, width).T)[0])
    product_close(f64(L.dact), values(L.dy8), values(L.w8_t))
    product_close(f64(L.dweight), values(L.dy8_t), values(L.act_t))
    n = values(L.kept, width)
    ref = f8.layer_norm_backward(f64(L.dact), n, f64(L.norm_weight), f64(L.rstd), f64(dh))
    g = f64(L.dact) * f64(L.norm_weight)
    size = f64(L.rstd)[:, None] * (np.abs(g) + np.abs(g).mean(-1, keepdims=True) + np.abs(n) * np.abs(g * n).mean(-1, keepdims=True))
    assert np.all(np.abs(f64(dx) - ref[0]) <= 2.0 ** -8 * np.abs(ref[0]) + 128 * 2.0 ** -24 * (size + np.abs(f64(dh))))
    chain = (tokens / 2 + 24) * 2.0 ** -24
    assert np.all(np.abs(f64(L.dnorm_weight) - ref[1]) <= chain * np.abs(f64(L.dact) * n).sum(0))
    assert np.all(np.abs(f64(L.dnorm_bias) - ref[2]) <= chain * np.abs(f64(L.dact)).sum(0))


def test_gradients_of_the_whole_step():
    """Against the fp64 gradient of the layer without any 8-bit rounding.  Each
    product's operands carry half a step of 2^-4 per element (and a floor
    below the blocks' normal range), errors that are independent from element to
    element: 2 * 2^-4 in the 2-norm bounds what two of them give with room, and
    the norm's own rounding adds another 2^-4."""
    L, x, r, dy, dh = layer()
    L.forward(x, r)
    dx = L.backward(dy, dh)
    h, w = f64((x.float() + r.float()).bfloat16()), f64(L.weight)
    a, n, _, rstd = f8.layer_norm(h, f64(L.norm_weight), f64(L.norm_bias), L.eps)
    g = f64(dy)
    rel = lambda p, q: np.linalg.norm(p - q) / np.linalg.norm(q)  # noqa: E731
    assert rel(f64(L.dweight), g.T @ a) <= 2 * 2.0 ** -4
    want = f8.layer_norm_backward(g @ w, n, f64(L.norm_weight), rstd, f64(dh))
    assert rel(f64(dx), want[0]) <= 3 * 2.0 ** -4
    assert rel(f64(L.dnorm_weight), want[1]) <= 3 * 2.0 ** -4 and rel(f64(L.dnorm_bias), want[2]) <= 3 * 2.0 ** -4
    # the oracle's gradient against differences of the layer's function along a direction
    t, v = 1e-4, np.random.default_rng(1).standard_normal(h.shape)
    f = lambda s: ((f8.layer_norm(s, f64(L.norm_weight), f64(L.norm_bias), L.eps)[0] @ w.T) * g).sum()  # noqa: E731
    assert abs((f(h + t * v) - f(h - t * v)) / (2 * t) - ((want[0] - f64(dh)) * v).sum()) <= 1e-5 * np.abs(want[0] * v).sum()


def test_captured():
    import torch
    L, x, r, dy, dh = layer(257, 384, 640)
    y = L.forward(x, r)
    dx = L.backward(dy, dh)
    torch.cuda.synchronize()
    results = lambda: [t.clone() for t in (y, dx, L.dweight, L.dnorm_weight, L.dnorm_bias, L.h)]  # noqa: E731
    want = results()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        L.forward(x, r)
        L.backward(dy, dh)
    for i in range(3):
        for t in (y, dx, L.dweight, L.dnorm_weight, L.dnorm_bias, L.h):
            t.fill_(i)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(results(), want))
        L.forward(x, r)
        L.backward(dy, dh)
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(results(), want))


def test_two_layers_at_once():
    """Two layers' steps on two streams, each with its own tensors and workspaces, equal the steps one after the other."""
    import torch
    made = [layer(300, 520, 392), layer(257, 384, 640)]
    want = []
    for L, x, r, dy, dh in made:
        y, dx = L.forward(x, r), L.backward(dy, dh)
        want.append([t.clone() for t in (y, dx, L.dweight, L.dnorm_weight, L.dnorm_bias)])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in made]
    for _ in range(5):
        for s, (L, x, r, dy, dh) in zip(streams, made):
            with torch.cuda.stream(s):
                L.forward(x, r)
                L.backward(dy, dh)
    torch.cuda.synchronize()
    for w, (L, *_) in zip(want, made):
        assert all(torch.equal(p, q) for p, q in zip(w, (L.y, L.dx, L.dweight, L.dnorm_weight, L.dnorm_bias)))


def test_weight_gradients_accumulate():
    """A second batch's gradient on top of the first, in fp32, with beta = 1."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(5)
    total, want, size = torch.zeros((200, 264), device="cuda"), 0, 0
    for tokens in (130, 300):
        pairs = []
        for cols in (200, 264):
            x = torch.randn(tokens, cols, generator=g, device="cuda").bfloat16()
            t = f8_linear.f8_empty(cols, tokens)
            dg.dist_gemm_f8_quantize(x, codes_t=t[0], scales_t=t[1])
            pairs.append(t)
        (a, a_s), (b, b_s) = pairs
        ws = f8_linear.product_workspace(200, 264, a.size(1))
        dg.dist_gemm_f8_product(a, a_s, b, b_s, total, C=total, beta=1.0, workspace=ws)
        va, vb = values((a, a_s)), values((b, b_s))
        want = want + va @ vb.T
        size = size + np.linalg.norm(va, axis=1)[:, None] * np.linalg.norm(vb, axis=1)[None]
    assert np.all(np.abs(f64(total) - want) <= 1e-4 * size)


def test_example_runs():
    f8_linear.main(tokens=200, width=384, out=256)

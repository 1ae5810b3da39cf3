"""GPU test of the low-precision operators run together (examples/mx_experts.py).

Each stage is checked against fp64 from the bytes that the stage before it
wrote, with that operator's own bar, so no tolerance covers a chain."""
import os
import sys

import numpy as np
import pytest

from gpu_helpers import log
from oracle import codecs, mx, parity

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu

BF16 = 2.0 ** -8    # half an ulp, relative
NORM = 2.0 ** -20   # fp32 sums of a few hundred terms, rsqrt and two products


def f64(t):
    import torch
    return t.to(torch.float64).cpu().numpy()


def values(pair, fmt, cols):
    return mx.values(pair[0].cpu().numpy(), pair[1].cpu().numpy(), fmt, cols)


def product_ok(got, a, b, out):
    ok, worst, tight, _ = parity.check(got, a @ b.T, np.linalg.norm(a, axis=1), np.linalg.norm(b, axis=1), 1.0, 0.0, None,
                                       "e4m3", out, None)
    assert ok and tight, worst


def by_expert(got, a, w, offsets):
    rows = w.shape[0] // (len(offsets) - 1)
    for e in range(len(offsets) - 1):
        r = slice(offsets[e], offsets[e + 1])
        if r.stop > r.start:
            product_ok(got[r], a[r], w[e * rows:(e + 1) * rows], "bf16")


def blocks_of(pair, fmt, ref):
    """The norm's blocks lie within half a step of `ref`, at the scale that was written."""
    scales = pair[1].cpu().numpy()[:, :ref.shape[1] // 32].astype(int) - 127
    got = values(pair, fmt, ref.shape[1])
    top = np.repeat(np.ldexp(1.0, scales), 32, axis=1)
    m = np.abs(ref) / top
    # spacing of the format at that value; past its largest value, values saturate
    if fmt == "E4M3":
        step, most = np.exp2(np.maximum(np.floor(np.log2(np.maximum(m, 2.0 ** -20))), -6) - 3), 448.0
    else:
        step, most = np.exp2(np.maximum(np.floor(np.log2(np.maximum(m, 2.0 ** -20))), 0) - 1), 6.0
    want = np.minimum(m, most) * np.sign(ref)
    # the next binade's step at its edge; the value itself to the norm's accuracy
    assert (np.abs(got / top - want) <= step * 0.5 + m * NORM * 2 + 1e-30).all()
    amax = np.abs(ref).reshape(*scales.shape, 32).max(-1)
    e = np.floor(np.log2(amax)) - mx.EMAX[fmt]
    near = np.abs(np.log2(amax) - np.round(np.log2(amax))) < 1e-5   # the norm's last bits decide
    assert ((scales == e) | near).all()


@pytest.mark.parametrize("tokens", [1, 7, 70, 300])
def test_experts(tokens):
    import torch
    import mx_experts
    experts, width, hidden, vocab = 5, 320, 544, 264
    log("experts", tokens)
    layer = mx_experts.Experts(300, experts, width, hidden, vocab, seed=3)
    g = torch.Generator(device="cuda").manual_seed(tokens)
    x, res, dn, dh = (torch.randn(tokens, width, device="cuda", generator=g).bfloat16() for _ in range(4))
    offsets = [0, tokens // 3, tokens // 3, tokens - tokens // 4, tokens, tokens]   # two of them empty
    s = layer.forward(x, res, torch.tensor(offsets, dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    h = f64(x) + f64(res)
    assert (np.abs(f64(s["h"]) - h) <= np.abs(h) * BF16).all()
    n, rstd = mx.rms_norm(f64(s["h"]), f64(layer.gain), 1e-6)[:2]
    blocks_of(s["n"], "E4M3", n)
    by_expert(f64(s["u"]), values(s["n"], "E4M3", width), values(layer.up, "E2M1", width), offsets)
    codes, scales = mx.quantize(f64(s["r"]), "E4M3")
    assert np.array_equal(s["a"][0].cpu().numpy(), codes) and np.array_equal(s["a"][1].cpu().numpy(), scales)
    by_expert(f64(s["o"]), values(s["a"], "E4M3", hidden), values(layer.down, "E2M1", hidden), offsets)
    m = mx.rms_norm(f64(s["h2"]), f64(layer.head_gain), 1e-6)[0]
    blocks_of(s["m"], "E2M1", m)
    product_ok(f64(s["logits"]), values(s["m"], "E2M1", width), values(layer.head, "E2M1", width), "f32")
    dx, dgain = layer.norm_gradient(dn, s, dh)
    torch.cuda.synchronize()
    rx, rw = mx.rms_norm_backward(f64(dn), f64(s["h"]), f64(layer.gain), rstd, f64(dh))
    big = np.abs(rx) + np.abs(f64(dh)) + np.abs(f64(dn)) * rstd.reshape(-1, 1) * np.abs(f64(layer.gain))
    assert (np.abs(f64(dx) - rx) <= np.abs(rx) * BF16 + big * 2.0 ** -16).all()
    terms = (np.abs(f64(dn) * f64(s["h"])) * rstd.reshape(-1, 1)).sum(0)
    assert (np.abs(f64(dgain) - rw) <= terms * 2.0 ** -16 + 1e-30).all()


def test_tensor_parallel_step():
    import torch
    import mx_experts
    tokens, width, N = 256, 512, 320
    log("tensor parallel", tokens, width, N)
    g = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randn(tokens, width, device="cuda", generator=g).bfloat16()
    gain = torch.rand(width, device="cuda", generator=g).add_(0.5).bfloat16()
    weight = torch.randint(0, 0x50, (N, width), dtype=torch.uint8, device="cuda", generator=g)
    scale = 1 / 64
    y, out = mx_experts.tensor_parallel(x, gain, weight, scale)
    n = mx.rms_norm(f64(x), f64(gain), 1e-6)[0] / scale
    a = codecs.e4m3_to_f64(y.cpu().numpy())
    step = np.exp2(np.maximum(np.floor(np.log2(np.maximum(np.abs(n), 2.0 ** -20))), -6) - 3)
    assert (np.abs(a - np.clip(n, -448, 448)) <= step * 0.5 + np.abs(n) * NORM).all()
    product_ok(f64(out), a * scale, codecs.e4m3_to_f64(weight.cpu().numpy()), "bf16")

"""CPU pins of oracle/mx.py: the element codes against exhaustive nearest-value
search, the block scale, and the norm's gradient against differences."""
import numpy as np
import pytest

from oracle import codecs, mx


def test_e2m1_is_the_nearest_value_ties_to_even():
    x = np.concatenate([np.linspace(-8, 8, 4097), [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 5.0001, 100.0]])
    got = mx.f64_to_e2m1(x)
    for v, c in zip(x, got):
        d = np.abs(mx.E2M1_VALUES - min(abs(v), 6.0))
        best = np.flatnonzero(d == d.min())
        want = best[0] if len(best) == 1 else [b for b in best if b % 2 == 0][0]
        assert c & 7 == want, v
    assert list(mx.f64_to_e2m1(np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0]))) == [0, 2, 2, 4, 4, 6, 6]
    assert mx.f64_to_e2m1(np.array([-0.0]))[0] == 8


def test_pack_puts_the_even_element_low():
    c = np.array([[1, 2, 3, 15]], dtype=np.uint8)
    assert mx.pack(c).tolist() == [[0x21, 0xF3]]
    assert (mx.unpack(mx.pack(c)) == c).all()


@pytest.mark.parametrize("fmt", ["E2M1", "E4M3"])
def test_quantize_by_hand(fmt):
    x = np.zeros((1, 64))
    x[0, 0], x[0, 1] = 5.0, -1.0          # floor(log2 5) = 2
    x[0, 32] = 2.0 ** -140                # below what E8M0 holds: X = -127
    codes, scales = mx.quantize(x, fmt)
    e = {"E2M1": 2, "E4M3": 8}[fmt]
    assert scales.shape == (1, 16) and scales[0, 0] == 127 + 2 - e and scales[0, 1] == 0 and not scales[0, 2:].any()
    v = mx.values(codes, scales, fmt, 64)
    assert v[0, 1] == -1.0 and v[0, 0] == {"E2M1": 4.0, "E4M3": 5.0}[fmt]


@pytest.mark.parametrize("fmt,most", [("E2M1", 2.0 / 8), ("E4M3", 64.0 / 512)])
def test_quantize_error_and_saturation(fmt, most):
    """Every value within its block's largest error: the top of the range
    saturates from 8 to 6 (E2M1) or 512 to 448 (E4M3)."""
    g = np.random.default_rng(3)
    x = g.standard_normal((50, 256)) * np.exp2(g.integers(-30, 30, (50, 1)))
    v = mx.values(*mx.quantize(x, fmt), fmt, 256)
    amax = np.abs(x).reshape(50, 8, 32).max(-1)
    top = np.exp2(np.floor(np.log2(amax)) + 1)
    assert (np.abs(v - x).reshape(50, 8, 32) <= most * top[..., None]).all()


def test_nonfinite_blocks_are_nan():
    x = np.ones((1, 96))
    x[0, 3], x[0, 40] = np.inf, np.nan
    codes, scales = mx.quantize(x, "E4M3")
    v = mx.values(codes, scales, "E4M3", 96)
    assert scales[0, :3].tolist() == [255, 255, 127 - 8] and np.isnan(v[0, :64]).all() and (v[0, 64:] == 1).all()
    assert not codes[0, :64].any()


def test_e4m3_elements_are_the_codecs():
    x = np.linspace(256, 511, 32)[None]
    codes, _ = mx.quantize(x, "E4M3")
    assert (codes == codecs.f64_to_e4m3(x)).all()


def test_norm_gradient_against_differences():
    g = np.random.default_rng(5)
    h, w, dy = g.standard_normal((3, 7)), g.standard_normal(7), g.standard_normal((3, 7))
    eps = 1e-3
    _, rstd = mx.rms_norm(h, w, eps)
    dx, dw = mx.rms_norm_backward(dy, h, w, rstd)
    t = 1e-6
    for i in range(3):
        for j in range(7):
            p, m = h.copy(), h.copy()
            p[i, j] += t
            m[i, j] -= t
            num = ((mx.rms_norm(p, w, eps)[0] - mx.rms_norm(m, w, eps)[0]) * dy).sum() / (2 * t)
            assert abs(num - dx[i, j]) < 1e-8
    for j in range(7):
        p, m = w.copy(), w.copy()
        p[j] += t
        m[j] -= t
        num = ((mx.rms_norm(h, p, eps)[0] - mx.rms_norm(h, m, eps)[0]) * dy).sum() / (2 * t)
        assert abs(num - dw[j]) < 1e-8

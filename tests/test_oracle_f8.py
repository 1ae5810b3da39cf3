"""CPU pins of oracle/f8.py: scales and codes by hand and by search, and the
layer norm's gradient against differences."""
import numpy as np
import pytest

from oracle import codecs, f8


@pytest.mark.parametrize("cols,pitch,scales", [(1, 128, 16), (128, 128, 16), (129, 256, 16), (2048, 2048, 16),
                                               (2049, 2176, 32), (16384, 16384, 128)])
def test_pitches(cols, pitch, scales):
    assert f8.pitch(cols) == pitch and f8.scale_pitch(cols) == scales


def test_quantize_by_hand():
    x = np.zeros((1, 300))
    x[0, 0], x[0, 1] = 448.0, -1.0        # 448 = 448 * 2^0
    x[0, 128], x[0, 129] = 449.0, 2.0     # one power further
    x[0, 256] = 2.0 ** -140               # below what E8M0 holds: X = -127
    codes, scales = f8.quantize(x)
    assert codes.shape == (1, 384) and scales.shape == (1, 16)
    assert scales[0, :4].tolist() == [127, 128, 0, 0]
    v = f8.values(codes, scales, 300)
    assert v[0, :2].tolist() == [448.0, -1.0] and v[0, 128:130].tolist() == [448.0, 2.0]
    assert not codes[0, 300:].any()


def test_the_scale_is_the_least_that_does():
    g = np.random.default_rng(1)
    x = g.standard_normal((40, 128)) * np.exp2(g.integers(-100, 100, (40, 1)))
    x[:8, 3] = np.ldexp([448, 448.0001, 447.9, 449, 224, 224.0001, 223.9, 256], 3) * np.sign(x[:8, 3])
    x[:8] = np.clip(x[:8], -np.abs(x[:8, 3:4]), np.abs(x[:8, 3:4]))
    _, scales = f8.quantize(x)
    amax = np.abs(x).max(-1)
    s = np.ldexp(1.0, scales[:, 0].astype(int) - 127)
    assert (amax <= 448 * s).all() and (amax > 224 * s).all()


def test_square_blocks_share_a_scale_and_transpose():
    x = np.random.default_rng(2).standard_normal((200, 300))
    codes, scales = f8.quantize(x, square=True)
    codes_t, scales_t = f8.quantize(x.T, square=True)
    assert np.array_equal(f8.values(codes, scales, 300), f8.values(codes_t, scales_t, 200).T)
    assert (scales[:128, :3] == scales[0, :3]).all() and (scales[128:, :3] == scales[128, :3]).all()


def test_nonfinite_blocks_are_nan():
    x = np.ones((1, 384))
    x[0, 3], x[0, 140] = np.inf, np.nan
    codes, scales = f8.quantize(x)
    v = f8.values(codes, scales, 384)
    assert scales[0, :3].tolist() == [255, 255, 127 - 8] and np.isnan(v[0, :256]).all() and (v[0, 256:] == 1).all()
    assert not codes[0, :256].any()


def test_requantising_only_rounds_below_the_normal_range():
    g = np.random.default_rng(4)
    x = g.standard_normal((256, 256)) * np.exp2(g.integers(-6, 6, (256, 1)))
    v = f8.values(*f8.quantize(x))
    codes_t, scales_t = f8.quantize(v.T)
    back = f8.values(codes_t, scales_t).T
    s = np.repeat(np.ldexp(1.0, scales_t[:, :2].astype(int) - 127), 128, axis=1).T
    normal = np.abs(v) >= s * 2.0 ** -6
    assert np.array_equal(back[normal], v[normal]) and (np.abs(back - v) <= s * 2.0 ** -10).all()
    assert (np.abs(codecs.e4m3_to_f64(codes_t)) <= 448).all()


def test_layer_norm_gradient_against_differences():
    g = np.random.default_rng(5)
    h, w, b, dy = g.standard_normal((3, 7)) + 2, g.standard_normal(7), g.standard_normal(7), g.standard_normal((3, 7))
    eps, t = 1e-3, 1e-6
    _, n, _, rstd = f8.layer_norm(h, w, b, eps)
    dx, dw, db = f8.layer_norm_backward(dy, n, w, rstd)

    def slope(change):
        return ((f8.layer_norm(*change(t), eps)[0] - f8.layer_norm(*change(-t), eps)[0]) * dy).sum() / (2 * t)

    def bump(a, at, d):
        a = a.copy()
        a[at] += d
        return a

    for i in range(3):
        for j in range(7):
            assert abs(slope(lambda d: (bump(h, (i, j), d), w, b)) - dx[i, j]) < 1e-8
    for j in range(7):
        assert abs(slope(lambda d: (h, bump(w, j, d), b)) - dw[j]) < 1e-8
        assert abs(slope(lambda d: (h, w, bump(b, j, d))) - db[j]) < 1e-8

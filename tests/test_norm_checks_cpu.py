"""CPU check of the comparison that the norms' statistics are held to: it
refuses a NaN or an infinity in the place of a number, and a number in theirs."""
import numpy as np
import pytest

from gpu_helpers import within
from oracle import f8, mx


def statistics():
    h = np.random.default_rng(1).standard_normal((6, 40))
    h[1, 3], h[2, 5] = np.nan, np.inf
    with np.errstate(invalid="ignore"):
        _, _, mean, rstd = f8.layer_norm(h, np.ones(40), None, 1e-5)
        _, rms = mx.rms_norm(h, np.ones(40), 1e-5)
    return mean, rstd, rms


@pytest.mark.parametrize("which", range(3))
def test_a_planted_mistake_is_refused(which):
    ref = statistics()[which]
    assert within(ref, ref, 0.0) and within(ref * (1 + 2.0 ** -30), ref, 1e-6)
    for row in range(len(ref)):
        for v in (np.nan, np.inf, -np.inf, 0.5):
            got = ref.copy()
            got[row] = v
            assert within(got, ref, 1e-6 * np.abs(ref)) == (got[row] == ref[row] or (np.isnan(got[row]) and np.isnan(ref[row]))), (row, v)


def test_tolerances_by_row():
    ref = np.array([1.0, 2.0])
    assert within([1.1, 2.0], ref, [0.2, 0.0]) and not within([1.1, 2.1], ref, [0.2, 0.0])

"""The scoring oracle against scipy, closed forms and a brute-force order."""
import numpy as np
import pytest
from scipy.special import log_softmax
from scipy.stats import entropy

from oracle import score as OS


@pytest.mark.parametrize("V, tau", [(1, 1.0), (2, 0.5), (17, 2.0), (1000, 0.7)])
def test_logp_and_entropy_match_scipy(V, tau):
    z = np.random.default_rng(V).normal(0, 3, V)
    ls = log_softmax(z / tau)
    for y in {0, V // 2, V - 1}:
        logp, H, idx, top = OS.score_row(z, y, V, tau)
        assert abs(logp - ls[y]) < 1e-12 and abs(H - entropy(np.exp(ls))) < 1e-11
        assert np.allclose(top, ls[idx], atol=1e-12)


def test_order_is_descending_then_by_index():
    rng = np.random.default_rng(1)
    for _ in range(50):
        z = rng.integers(-3, 4, 40).astype(float)
        z[rng.random(40) < 0.2] = -np.inf
        z[0] = 0.0
        _, _, idx, _ = OS.score_row(z, None, 40)
        assert idx.tolist() == sorted(range(40), key=lambda v: (-z[v], v))


def test_uniform_and_one_hot_rows():
    logp, H, idx, top = OS.score_row(np.zeros(8), 3, 4)
    assert np.isclose(logp, -np.log(8)) and np.isclose(H, np.log(8)) and idx.tolist() == [0, 1, 2, 3]
    z = np.full(8, -np.inf)
    z[5] = 2.0
    logp, H, idx, top = OS.score_row(z, 5, 3)
    assert logp == 0 and H == 0 and idx.tolist() == [5, 0, 1] and top.tolist() == [0.0, -np.inf, -np.inf]


@pytest.mark.parametrize("bad", [np.nan, np.inf])
def test_rows_without_a_distribution(bad):
    z = np.zeros(6)
    z[2] = bad
    logp, H, idx, top = OS.score_row(z, 0, 2)
    assert np.isnan(logp) and np.isnan(H) and idx.tolist() == [-1, -1] and np.isnan(top).all()
    logp, H, idx, _ = OS.score_row(np.full(4, -np.inf), 0, 1)
    assert np.isnan(logp) and np.isnan(H) and idx.tolist() == [-1]
    assert np.isnan(OS.score_row(np.zeros(4), 4, 1)[0])


def test_the_types_lowest_value_masks_like_minus_infinity():
    z = np.full(6, float(np.finfo(np.float32).min))
    z[2:4] = [1.0, 0.0]
    w = np.where(z < -1e38, -np.inf, z)
    a, b = OS.score_row(z, 5, 6), OS.score_row(w, 5, 6)
    assert a[0] == b[0] == -np.inf and a[1] == b[1] and np.array_equal(a[3], b[3])
    assert a[2].tolist() == b[2].tolist() == [2, 3, 0, 1, 4, 5]
    assert np.isnan(OS.score_row(np.full(4, z[0]), 0, 1)[1])
    assert not np.isnan(OS.score_row(np.full(4, z[0]), 0, 1, tau=2.0)[1])  # within the range again

"""Pins of the float64 cross entropy and clipping oracle: scipy's log-softmax, the usual closed forms and
central differences."""
import numpy as np
import pytest
from scipy.special import log_softmax, logsumexp

from oracle import ce as OC

OPTIONS = [dict(), dict(eps=0.1), dict(lam=1e-2), dict(cap=3.0), dict(eps=0.3, lam=1e-2, cap=2.0), dict(eps=1.0)]


@pytest.mark.parametrize("kw", OPTIONS)
def test_loss_is_the_mixed_cross_entropy(kw):
    rng = np.random.default_rng(0)
    x = rng.normal(0, 3, 37)
    eps, lam, cap = kw.get("eps", 0.0), kw.get("lam", 0.0), kw.get("cap", 0.0)
    z = cap * np.tanh(x / cap) if cap else x
    q = np.full(37, eps / 37)
    q[5] += 1 - eps
    want = -np.sum(q * log_softmax(z)) + lam * logsumexp(z) ** 2
    assert np.isclose(OC.row_loss(x, 5, **kw)[0], want, rtol=1e-13)


@pytest.mark.parametrize("kw", OPTIONS)
def test_gradients_against_central_differences(kw):
    rng = np.random.default_rng(1)
    T, V, H = 5, 11, 4
    h, W = rng.normal(0, 1, (T, H)), rng.normal(0, 1, (V, H))
    y, mask, w = rng.integers(0, V, T), np.array([1, 0, 1, 1, 1]), rng.random(T) + 0.5
    f = lambda h, W: 0.25 * np.sum(OC.lmhead(h, W, y, mask, 0.25, w, **kw)["loss"] * w)
    got = OC.lmhead(h, W, y, mask, 0.25, w, **kw)
    for a, grad, of in ((h, got["d_h"], lambda a: f(a, W)), (W, got["dW"], lambda a: f(h, a))):
        for i in np.ndindex(a.shape):
            up, dn = a.copy(), a.copy()
            up[i] += 1e-6
            dn[i] -= 1e-6
            assert abs((of(up) - of(dn)) / 2e-6 - grad[i]) <= 1e-8
    assert np.all(got["d_h"][1] == 0) and got["loss"][1] == 0


def test_masked_rows_may_hold_anything_and_bad_targets_are_nan():
    rng = np.random.default_rng(2)
    h, W = rng.normal(0, 1, (3, 4)), rng.normal(0, 1, (9, 4))
    a = OC.lmhead(h, W, [1, 2, 3], [1, 0, 1], 1.0)
    h[1] = np.nan
    b = OC.lmhead(h, W, [1, -100, 3], [1, 0, 1], 1.0)
    assert np.array_equal(a["dW"], b["dW"]) and np.array_equal(a["loss"], b["loss"])
    assert np.isnan(OC.lmhead(h, W, [1, 2, 9], [1, 0, 1], 1.0)["loss"][2])


def test_clip_factor():
    g = [np.array([3.0]), np.array([0.0, 4.0])]
    assert OC.clip(g, 10.0)[:2] == (5.0, 1.0) and OC.clip(g, 5.0)[:2] == (5.0, 1.0)
    assert np.isclose(OC.clip(g, 1.0)[1], 0.2) and np.allclose(OC.clip(g, 1.0)[2], [3, 4])
    n, f, each = OC.clip(g, 1.0, scale=0.5)
    assert np.isclose(n, 2.5) and np.isclose(f, 0.2) and np.allclose(each, [1.5, 2.0])
    assert OC.clip([np.array([np.inf])], 1.0)[1] == 0.0 and OC.clip([], 1.0)[:2] == (0.0, 1.0)

"""The distillation oracle where the student's remainder underflows as a share of its row."""
import numpy as np
import pytest

from oracle import distill as OD


@pytest.mark.parametrize("gap", [50.0, 100.0, 700.0, 1e3, 1e4])
def test_closed_form_of_two_levels(gap):
    V, n, q = 1000, 4, 0.2
    z = np.full(V, -gap)
    z[:n] = 0.0
    loss, dx, _ = OD.row_loss(z, np.arange(n), np.full(n, np.log(q)), OD.FORWARD_TAIL)
    qr = 1 - n * q
    log_s = np.log(n) + np.log1p((V - n) / n * np.exp(-gap))
    want = n * q * (np.log(q) + log_s) + qr * (np.log(qr) - (np.log(V - n) - gap - log_s))
    assert abs(loss - want) <= 1e-12 * abs(want)
    p = np.exp(-gap - log_s)
    assert np.allclose(dx[n:], p - qr / (V - n), rtol=1e-12, atol=0)
    # the logarithm of the remainder is a number of the gap's size, off by half a step (2^-53 of it) or two
    assert abs(dx.sum()) < 1e-13 + qr * gap * 2.0 ** -52


@pytest.mark.parametrize("gap", [10.0, 95.0, 1e3])
def test_gradient_matches_central_differences(gap):
    rng = np.random.default_rng(3)
    z = rng.normal(0, 1, 9) - gap
    z[:3] += gap
    idx, lq = np.array([1, 0, 2]), np.log([0.3, 0.2, 0.25])
    _, g, _ = OD.row_loss(z, idx, lq, OD.FORWARD_TAIL, 0.7)
    h = 1e-5 * max(1.0, gap / 100)
    for v in range(9):
        a, b = z.copy(), z.copy()
        a[v] += h
        b[v] -= h
        num = (OD.row_loss(a, idx, lq, OD.FORWARD_TAIL, 0.7)[0] - OD.row_loss(b, idx, lq, OD.FORWARD_TAIL, 0.7)[0]) / (2 * h)
        assert abs(num - g[v]) < 1e-6

"""GPU cross entropy from hidden states at its edges. Tolerances as in test_gpu_lmhead_ce.py where its checks are
used; the others stand at their tests."""
import numpy as np
import pytest
import torch

from rl_post_token_gb300 import _lib
from tests.test_gpu_lmhead_ce import BF16, DEV, _built, _call, _check64, _inputs, cta_group  # noqa: F401

pytestmark = pytest.mark.gpu
# reduce and dlogits in one launch; logits kept; formed again; formed again in two pieces. The last column is alone
# in its tile
PATHS = {"joint": (70, 769, 64), "kept": (300, 8961, 64), "again": (700, 8961, 64), "pieces": (4200, 34817, 64)}


@pytest.mark.parametrize("cap", [0.0, 0.5, 30.0])
@pytest.mark.parametrize("what", ["h inf", "h -inf", "h nan", "W inf", "W -inf", "W nan", "W -inf alone"])
@pytest.mark.parametrize("column", [-1, -9])
@pytest.mark.parametrize("path", PATHS)
def test_a_logit_that_is_infinite_or_nan_counts_as_non_finite(path, column, what, cap):
    T, V, H = PATHS[path]
    h, Wt, y, _ = _inputs(T, V, H, 8, None)
    y[y >= V - 9] = 0
    where, value = what.split()[:2]
    if what.endswith("alone"):
        h[:, 5] = h[:, 5].abs() + 0.125  # every token's logit there is -inf, and no other is infinite
    clean = _call(h, Wt, y, None, 1.0, soft_cap=cap, z_loss=1e-3)
    bad = torch.ones(T, dtype=torch.bool, device=DEV)
    if where == "h":
        h[3, 5] = float(value)
        bad[:] = False
        bad[3] = True
    else:
        Wt[column, 5] = float(value)
    for grads in (False, True):
        out = _call(h, Wt, y, None, 1.0, soft_cap=cap, z_loss=1e-3, grads=grads)
        for k in ("loss", "logp", "lse"):
            assert torch.equal(torch.isnan(out[k]), bad) and torch.equal(out[k][~bad], clean[k][~bad]), k
    assert torch.isnan(out["d_h"][bad]).all() and torch.equal(out["d_h"][~bad], clean["d_h"][~bad])
    res = _lib.grpo_finish_step(out["acc"], out["loss"], expected_N=T, grad_bufs=[out["d_h"], out["dW"]])
    assert res["status"] == _lib.STEP_SKIPPED_NONFINITE and res["n_nonfinite"] == int(bad.sum())
    assert torch.all(out["d_h"] == 0) and torch.all(out["dW"] == 0)


@pytest.mark.parametrize("path", PATHS)
def test_a_non_finite_token_of_weight_zero_has_a_nan_gradient(path):
    T, V, H = PATHS[path]
    h, Wt, y, _ = _inputs(T, V, H, 9, None)
    y[3] = V
    w = np.ones(T, np.float32)
    w[3] = 0.0
    out = _call(h, Wt, y, None, 1.0, w=w)
    assert torch.isnan(out["loss"][3]) and torch.isnan(out["d_h"][3]).all() and torch.isnan(out["dW"]).all()
    assert torch.isfinite(out["d_h"][4:]).all()
    assert _lib.grpo_finish_step(out["acc"], out["loss"], expected_N=T)["n_nonfinite"] == 1


@pytest.mark.parametrize("H", [2048, 8192, 16384, 65536])
def test_exact_products_of_large_hidden_sizes(H):
    # Eight entries of a hidden state are not 0, and they and W are powers of two: no partial sum is rounded.
    # The factor on the products is at most 1 + 2^-30 8192 = 1 + 2^-17, so lse is off by 2^-17 of the largest
    # logit; exponentials, their sum and the logarithm add less than 2^-20 max(1, |lse|).
    T, V = 300, 1000
    rng = np.random.default_rng(H)
    h = torch.zeros((T, H), device=DEV)
    at = torch.from_numpy(np.stack([rng.choice(H, 8, replace=False) for _ in range(T)])).to(DEV)
    h.scatter_(1, at, torch.from_numpy(2.0 ** rng.integers(0, 4, (T, 8))).float().to(DEV))
    g = torch.Generator(device=DEV)
    g.manual_seed(H)
    Wt = torch.randint(0, 2, (V, H), generator=g, device=DEV) * 2.0 - 1.0
    x = h.double() @ Wt.double().T
    out = _call(h.to(BF16), Wt.to(BF16), rng.integers(0, V, T).astype(np.int32), None, 1.0, grads=False)
    lse, top = torch.logsumexp(x, 1), x.abs().max(1).values
    assert float(top.max()) > 24
    assert torch.all((out["lse"].double() - lse).abs() <= 2.0 ** -17 * top + 2.0 ** -20 * lse.abs().clamp(min=1.0))


@pytest.mark.parametrize("terms", [dict(), dict(label_smoothing=0.1, z_loss=1e-3, soft_cap=5.0)])
@pytest.mark.parametrize("T, V, H", [(200, 3000, 4096), (300, 4000, 8192), (70, 4000, 16384)])
def test_large_hidden_sizes(cta_group, T, V, H, terms):
    # (at most 1e-5 of a logit is left of what the products lose; the logits are a few units, so that is below the
    # bar, 1e-5 of log-probs and lse of 8 and more)
    a = _inputs(T, V, H, 5, 0.2)
    _check64(a, 1.0, _call(*a, 1.0, **terms), **terms)


@pytest.mark.parametrize("H", [2048, 8192])
def test_what_dense_products_lose_is_given_back(H):
    # with one entry in the vocabulary lse is the logit: in the mean over many it loses 0.93 to 1.04 times 2^-30 H
    # of its size, and less than half of that may be left
    T, lost, size = 8192, 0.0, 0.0
    for seed in range(8):
        h, Wt, y, _ = _inputs(T, 1, H, seed, None, std=20.0)
        x = (h.double() @ Wt.double().T)[:, 0]
        out = _call(h, Wt, y, None, 1.0, grads=False)
        lost += float(((out["lse"].double() - x) * x.sign()).sum())
        size += float(x.abs().sum())
    assert abs(lost) <= 0.5 * 2.0 ** -30 * H * size


@pytest.mark.parametrize("terms", [dict(label_smoothing=0.1), dict(z_loss=1e-3, soft_cap=5.0)])
@pytest.mark.parametrize("T, V, H, masked", [
    (1000, 50257, 1000, 0.3), (1000, 50257, 1024, None), (1000, 50257, 1088, 0.3),  # by H, on and off 64
    (250, 50257, 1000, None), (251, 50257, 1000, None), (250, 50257, 512, None),    # few tokens
    (568, 9200, 64, None), (569, 9200, 64, 0.1),                                    # 20 MB
    (1328, 50257, 1088, None), (1340, 50257, 1088, None),                           # 256 MB
    (91, 9200, 64, None), (92, 9200, 64, None)])                                    # one launch for both
def test_the_limits_of_keeping_the_logits(T, V, H, masked, terms):
    a = _inputs(T, V, H, 6, masked)
    _check64(a, 1.0 / T, _call(*a, 1.0 / T, **terms), **terms)


def test_float32_gradients_over_micro_batches_at_a_large_hidden_size():
    T, V, H = 300, 6000, 4096
    a, b = _inputs(T, V, H, 21, 0.3), _inputs(T, V, H, 22, None)
    b = (b[0], a[1], b[2], b[3])
    one, two = _call(*a, 1.0), _call(*b, 1.0)
    dW = _call(*a, 1.0)["dW"]
    got = _call(*b, 1.0, dW=dW, dw_accumulate=True)["dW"]
    assert got is dW and torch.equal(got, one["dW"] + two["dW"])

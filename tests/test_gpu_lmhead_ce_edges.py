"""GPU cross entropy from hidden states at its edges. Tolerances as in test_gpu_lmhead_ce.py where its checks are
used; the others stand at their tests."""
import numpy as np
import pytest
import torch

from rl_post_token_gb300 import _lib
from tests.test_gpu_lmhead_ce import DEV, _built, _call, _inputs  # noqa: F401

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

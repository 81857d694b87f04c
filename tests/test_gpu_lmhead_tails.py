"""GPU calls from hidden states at a vocabulary's last tile: one that ends on an odd group of 32 columns while the
same CTAs go on to further tiles (the dlogits' staging buffers are then taken out of their turn), and one whose
only column is NaN. Checks and tolerances of test_gpu_lmhead.py."""
import numpy as np
import pytest
import torch

from rl_post_token_gb300 import _lib
from tests import test_gpu_lmhead_distill as D
from tests.test_gpu_lmhead import DEV, _built, _case, _check, cta_group  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("V", [20, 256 + 70, 256 + 140])
def test_an_odd_tail_followed_by_other_tiles(cta_group, V):
    # 40000 tokens: 157 pairs' tiles (313 of one CTA) to a column of tiles, two and more to each pair (CTA)
    _check(40000, V, 64, seed=V, valid_lo=0.1, old=False)


@pytest.mark.parametrize("V", [1, 257, 4097])
@pytest.mark.parametrize("entropy", [False, True])
def test_a_nan_column_alone_in_its_tile_counts(cta_group, V, entropy):
    T, Hd = 70, 64
    wl, h, Wt, hb, wb, mask, a_tok, old_logp = _case(T, V, Hd, seed=5, valid_lo=0.2)
    Wt[V - 1, 3] = float("nan")
    t = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(DEV)
    d_h, dW, loss, logp = (torch.full(s, 7.0, device=DEV) for s in ((T, Hd), (V, Hd), (T,), (T,)))
    acc = _lib.new_step_acc(DEV)
    ws = torch.empty(_lib.grpo_lmhead_workspace_size(T, V, Hd), dtype=torch.uint8, device=DEV)
    terms = dict(ent_coef=0.05, entropy_tok=torch.empty(T, device=DEV)) if entropy else None
    _lib.grpo_lmhead_loss_fwd_bwd(h, Wt, t(wl.target), t(old_logp), t(a_tok), t(mask), wl.eps, 1.0, d_h, dW, loss, logp,
                                  acc, ws, terms=terms)
    valid = t(mask) != 0
    assert torch.equal(torch.isnan(logp), valid)
    res = _lib.grpo_finish_step(acc, loss, expected_N=int(mask.sum()), grad_bufs=[d_h, dW])
    assert res["status"] == _lib.STEP_SKIPPED_NONFINITE and res["n_nonfinite"] == int(mask.sum()) > 0
    assert torch.all(d_h == 0) and torch.all(dW == 0)


@pytest.mark.parametrize("V", [257, 4097])
def test_a_nan_column_alone_in_its_tile_counts_in_the_distillation(cta_group, V):
    T = 70
    h, Wt, idx, lq, mask = D._inputs(T, V, 64, 8, 6)
    idx[idx == V - 1] = 0
    Wt[V - 1, 3] = float("nan")
    ws = torch.empty(_lib.grpo_lmhead_distill_workspace_size(T, V, 64, 8), dtype=torch.uint8, device=DEV)
    loss, acc = torch.empty(T, device=DEV), _lib.new_step_acc(DEV)
    _lib.grpo_lmhead_distill_topk_fwd_bwd(h, Wt, D._t(idx), D._t(lq), D._t(mask), 1.0, None, None, loss, acc, ws)
    res = _lib.grpo_finish_step(acc, loss, expected_N=int(mask.sum()))
    used = (mask != 0) & (idx >= 0).any(1)  # (a token without a list has loss 0)
    assert res["status"] == _lib.STEP_SKIPPED_NONFINITE and res["n_nonfinite"] >= int(used.sum()) > 0

"""The distillation oracle against closed forms, full KL divergences and central differences."""
import numpy as np
import pytest
from scipy.special import log_softmax, rel_entr

from oracle import distill as OD

KINDS = [OD.FORWARD_TOPK, OD.FORWARD_TAIL, OD.REVERSE_TAIL]


def _case(seed, V=11, K=4, unused=1):
    rng = np.random.default_rng(seed)
    z = rng.normal(0, 2, V)
    idx = np.concatenate([rng.permutation(V)[:K], np.full(unused, -1)])
    lq = np.concatenate([log_softmax(rng.normal(0, 1, K + 1))[:K], np.zeros(unused)])
    order = rng.permutation(K + unused)
    return z, idx[order], lq[order]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("tau", [1.0, 0.5, 2.0])
@pytest.mark.parametrize("seed", range(6))
def test_gradient_matches_central_differences(kind, tau, seed):
    z, idx, lq = _case(seed)
    _, g, _ = OD.row_loss(z, idx, lq, kind, tau)
    h = 1e-6
    for v in range(z.shape[0]):
        a, b = z.copy(), z.copy()
        a[v] += h
        b[v] -= h
        num = (OD.row_loss(a, idx, lq, kind, tau)[0] - OD.row_loss(b, idx, lq, kind, tau)[0]) / (2 * h)
        assert abs(num - g[v]) < 1e-8
    assert abs(g.sum()) < 1e-12  # the softmax does not see a shift of the row


@pytest.mark.parametrize("tau", [1.0, 1.7])
def test_a_list_of_the_whole_vocabulary_is_the_full_divergence(tau):
    rng = np.random.default_rng(3)
    z, lq = rng.normal(0, 1, 9), log_softmax(rng.normal(0, 1, 9))
    p, q = np.exp(log_softmax(z / tau)), np.exp(lq)
    for kind, want in ((OD.FORWARD_TOPK, rel_entr(q, p).sum()), (OD.FORWARD_TAIL, rel_entr(q, p).sum()),
                       (OD.REVERSE_TAIL, rel_entr(p, q).sum())):
        assert abs(OD.row_loss(z, np.arange(9), lq, kind, tau)[0] - want) < 1e-7, kind


def test_tail_kinds_are_the_divergence_of_the_merged_distributions():
    z, idx, lq = _case(5)
    p = np.exp(log_softmax(z))
    S = idx[idx >= 0]
    q = np.exp(lq[idx >= 0])
    pm, qm = np.append(p[S], 1 - p[S].sum()), np.append(q, 1 - q.sum())
    assert abs(OD.row_loss(z, idx, lq, OD.FORWARD_TAIL)[0] - rel_entr(qm, pm).sum()) < 1e-12
    assert abs(OD.row_loss(z, idx, lq, OD.REVERSE_TAIL)[0] - rel_entr(pm, qm).sum()) < 1e-12


@pytest.mark.parametrize("kind", KINDS)
def test_equal_distributions_give_zero(kind):
    z = np.random.default_rng(7).normal(0, 1, 12)
    lp = log_softmax(z / 0.8)
    idx = np.array([3, 0, 11, 5])
    # FORWARD_TOPK compares the renormalised list with the full student: equal where it is everything
    idx = np.arange(12) if kind == OD.FORWARD_TOPK else idx
    loss, g, _ = OD.row_loss(z, idx, lp[idx], kind, 0.8)
    assert abs(loss) < 1e-12 and np.abs(g).max() < 1e-12


def test_topk_takes_the_list_up_to_a_constant():
    z, idx, lq = _case(9)
    a, b = OD.row_loss(z, idx, lq, 0), OD.row_loss(z, idx, lq + 40.0, 0)
    assert abs(a[0] - b[0]) < 1e-12 and np.abs(a[1] - b[1]).max() < 1e-12


@pytest.mark.parametrize("kind", KINDS)
def test_empty_and_bad_lists(kind):
    z = np.random.default_rng(1).normal(0, 1, 6)
    loss, g, _ = OD.row_loss(z, [-1, -1], [0.0, 0.0], kind)
    assert abs(loss) < 2.0 ** -23 and np.abs(g).max() < 2.0 ** -23
    for idx, lq in (([1, 1], [-1.0, -1.0]), ([1, 6], [-1.0, -1.0]), ([-2, 1], [-1.0, -1.0]),
                    ([0, 1], [np.nan, -1.0]), ([0, 1], [np.inf, -1.0])):
        loss, g, _ = OD.row_loss(z, idx, lq, kind)
        assert np.isnan(loss) and np.isnan(g).all()

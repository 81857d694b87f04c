"""GPU parity of the LM-head distillation call against the float64 oracle: per-token loss, d_h and
dW over ragged extents, several vocabulary chunks, masked tokens, unused list entries, weights,
both tile shapes and the flags.

Tolerances. Loss: every log-prob within the LM-head bar 1e-5 max(1, |log p|) (the other LM-head
tests'), weighted by the renormalised teacher's probabilities, and 4 roundings of 2^-24 of each
term's parts. d_h and dW are products of dlogits rounded to bf16 (half a step: 2^-8 of each), with
float32 sums of at most 16,896 terms per chunk: |d| <= (2^-8 + 2^-10) (|dz| |W|) + the same for the
listed tokens' |p - q|, whose error is (1e-5 max(1, |log p|) + 2^-22) p + 2^-22 q."""
import numpy as np
import pytest
import torch

from oracle import distill as OD
from oracle import loss as OL
from rl_post_token_gb300 import _lib
from rl_post_token_gb300 import workloads as W

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _built(grpo_lib):
    assert torch.cuda.is_available()
    return grpo_lib


@pytest.fixture(params=[2, 1], ids=["pair", "one_cta"])
def cta_group(request, monkeypatch):
    monkeypatch.setenv("GRPO_LMHEAD_CTA_GROUP", str(request.param))
    return request.param


def _t(a):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def _inputs(T, V, H, K, seed, masked=0.2, unused=0.3, std=0.05):
    rng = np.random.default_rng(seed)
    h = torch.from_numpy(rng.standard_normal((T, H)).astype(np.float32)).to(torch.bfloat16).to(DEV)
    Wt = torch.from_numpy((std * rng.standard_normal((V, H))).astype(np.float32)).to(torch.bfloat16).to(DEV)
    idx = np.stack([rng.permutation(V)[:K] for _ in range(T)]).astype(np.int32)
    lq = np.log(rng.dirichlet(np.ones(K + 1), T)[:, :K] + 1e-6).astype(np.float32)
    cut = rng.random((T, K)) < unused
    idx[cut], lq[cut] = -1, 0.25
    mask = (rng.random(T) >= masked).astype(np.uint8)
    return h, Wt, idx, lq, mask


def _call(h, Wt, idx, lq, mask, scale, w=None, grads=True, dW=None, ws=None, **kw):
    T, H = h.shape
    V, K = Wt.shape[0], idx.shape[1]
    d_h = torch.full((T, H), 7.0, device=DEV) if grads else None
    if grads and dW is None:
        dW = torch.full((V, H), 7.0, device=DEV)
    loss = torch.full((T,), -7.0, device=DEV)
    acc = _lib.new_step_acc(DEV)
    if ws is None:
        ws = torch.empty(_lib.grpo_lmhead_distill_workspace_size(T, V, H, K), dtype=torch.uint8, device=DEV)
    _lib.grpo_lmhead_distill_topk_fwd_bwd(h, Wt, _t(idx), _t(lq), _t(mask), scale, d_h, dW, loss, acc, ws, w_tok=_t(w),
                                          **kw)
    torch.cuda.synchronize()
    return loss, d_h, dW, acc


def _reference(h, Wt, idx, lq, mask, scale, w=None):
    """(loss, loss bar, dz, dz bar) in float64."""
    hd, wd = h.double().cpu().numpy(), Wt.double().cpu().numpy()
    z = hd @ wd.T
    T, V = z.shape
    loss, bar, dz, bz = np.zeros(T), np.zeros(T), np.zeros((T, V)), np.zeros((T, V))
    for t in range(T):
        if not mask[t]:
            continue
        g = scale * (1.0 if w is None else float(w[t]))
        loss[t], d, parts = OD.row_loss(z[t], idx[t], lq[t], OD.FORWARD_TOPK)
        dz[t] = d * g
        S = idx[t][idx[t] != -1]
        lp, p, q = parts["lp"], parts["p"], parts["q"]
        e = 1e-5 * np.maximum(1.0, np.abs(lp))
        lqn = np.log(np.where(q > 0, q, 1.0))
        lqt = lq[t][idx[t] != -1].astype(np.float64)
        lqt = np.where(q > 0, lqt, 0.0)  # an entry without mass adds nothing (its log-prob may be -inf)
        bar[t] = np.sum(q * (e[S] + 2.0 ** -22 * (np.abs(lqn) + np.abs(lqt) + np.abs(lp[S]) + 1))) + 1e-7
        bz[t] = abs(g) * p * (e + 2.0 ** -22) * (1.0 if parts["alpha"] else 0.0)
        bz[t, S] += abs(g) * 2.0 ** -21 * q
    return hd, wd, loss, bar, dz, bz


def _check(args, scale, out, w=None, dw0=None):
    h, Wt, idx, lq, mask = args
    loss, d_h, dW, acc = out
    hd, wd, rl, bar, dz, bz = _reference(h, Wt, idx, lq, mask, scale, w)
    err = np.abs(loss.double().cpu().numpy() - rl)
    assert np.all(err <= bar), (int(np.argmax(err - bar)), err.max())
    if d_h is None:
        return
    m = (2.0 ** -8 + 2.0 ** -10) * np.abs(dz) + 1.01 * bz
    for got, ref, tol in ((d_h, dz @ wd, m @ np.abs(wd)), (dW, dz.T @ hd, m.T @ np.abs(hd))):
        if got is dW and dw0 is not None:
            ref = ref + dw0
            tol = tol + 2.0 ** -23 * np.abs(ref)
        e = np.abs(got.double().cpu().numpy() - ref)
        assert np.all(e <= tol + 1e-12), (e.max(), float((e - tol).max()))


@pytest.mark.parametrize("T, V, H, K", [(1, 5, 64, 5), (2, 300, 64, 1), (130, 3000, 128, 20), (257, 1027, 192, 256),
                                        (300, 40000, 512, 33), (64, 17153, 1088, 64)])
def test_parity(cta_group, T, V, H, K):
    a = _inputs(T, V, H, K, T + V)
    _check(a, 0.7, _call(*a, 0.7))
    w = np.random.default_rng(0).random(T).astype(np.float32)
    _check(a, 1.0 / T, _call(*a, 1.0 / T, w=w), w=w)


def test_skipping_masked_tokens_accumulating_and_loss_only_keep_the_bits():
    a = _inputs(300, 20000, 256, 16, 4, masked=0.5)
    loss, d_h, dW, acc = _call(*a, 1.0)
    res = _lib.grpo_finish_step(acc, loss, expected_N=int(a[4].sum()))
    assert res["status"] == 0 and res["n_tokens"] == 300
    l2, h2, w2, _ = _call(*a, 1.0, skip_masked=True)
    assert torch.equal(loss, l2) and torch.equal(d_h, h2) and torch.equal(dW, w2)
    l3, _, _, _ = _call(*a, 1.0, grads=False)
    assert torch.equal(loss, l3)
    base = torch.randn_like(dW)
    acc_w = base.clone()
    l4, h4, _, _ = _call(*a, 1.0, dW=acc_w, dw_accumulate=True)
    assert torch.equal(h4, d_h) and torch.equal(acc_w, base + dW)
    assert torch.all(d_h[torch.from_numpy(a[4] == 0).to(DEV)] == 0)
    # a workspace holding another call's values and NaN bytes
    ws = torch.full((_lib.grpo_lmhead_distill_workspace_size(300, 20000, 256, 16),), 255, dtype=torch.uint8, device=DEV)
    _call(*_inputs(300, 20000, 256, 16, 5), 1.0, ws=ws)
    l5, h5, w5, _ = _call(*a, 1.0, ws=ws)
    assert torch.equal(loss, l5) and torch.equal(d_h, h5) and torch.equal(dW, w5)


def test_agrees_with_the_row_call_on_the_stored_logits():
    h, Wt, idx, lq, mask = a = _inputs(96, 5000, 128, 24, 9)
    loss, d_h, _, _ = _call(*a, 1.0)
    z = (h.double() @ Wt.double().T).float()
    l2, dz = torch.empty(96, device=DEV), torch.empty_like(z)
    _lib.grpo_distill_topk_fwd_bwd(z, _t(idx), _t(lq), _t(mask), _lib.DISTILL_FORWARD_TOPK, 1.0, dz, l2,
                                   _lib.new_step_acc(DEV))
    # both within the log-prob bar of the exact loss
    assert torch.all((loss - l2).abs() <= 2e-5 * torch.clamp(l2.abs(), min=1.0) + 2e-5)
    ref, scale = dz.double() @ Wt.double(), dz.double().abs() @ Wt.double().abs()
    assert torch.all((d_h.double() - ref).abs() <= (2.0 ** -8 + 2.0 ** -10 + 1e-4) * scale + 1e-9)


def test_bad_lists_and_rows_are_counted_and_zeroed():
    h, Wt, idx, lq, mask = _inputs(40, 3000, 64, 8, 2, masked=0.0, unused=0.0)
    idx[3, 1] = idx[3, 5]
    idx[4, 0] = 3000
    idx[5, 0] = -7
    lq[6, 0] = np.nan
    idx[7] = -1
    lq[8] = -np.inf
    lq[9, 2] = -np.inf
    lq[10] += 300.0  # the list up to a constant
    h[11] = float("nan")
    a = (h, Wt, idx, lq, mask)
    loss, d_h, dW, acc = _call(*a, 1.0)
    bad = [3, 4, 5, 6, 11]
    lh = loss.cpu().numpy()
    assert np.isnan(lh[bad]).all() and np.isfinite(np.delete(lh, bad)).all() and lh[7] == 0 and lh[8] == 0
    assert torch.isnan(d_h[bad]).all() and torch.all(d_h[[7, 8]] == 0)
    res = _lib.grpo_finish_step(acc, loss, grad_bufs=[d_h, dW])
    assert res["status"] == _lib.STEP_SKIPPED_NONFINITE and res["n_nonfinite"] == len(bad)
    assert not d_h.any() and not dW.any()
    ok = np.array([t for t in range(40) if t not in bad])
    b = (h[torch.from_numpy(ok).to(DEV)].contiguous(), Wt, idx[ok], lq[ok], mask[ok])
    _check(b, 1.0, _call(*b, 1.0))


def test_every_token_masked():
    h, Wt, idx, lq, mask = _inputs(70, 2000, 64, 8, 2)
    for skip in (False, True):
        loss, d_h, dW, acc = _call(h, Wt, idx, lq, mask * 0, 1.0, skip_masked=skip)
        assert not loss.any() and not d_h.any() and not dW.any()
        assert _lib.grpo_finish_step(acc, loss, expected_N=0)["status"] == 0


def test_captured_into_a_graph():
    a, b = _inputs(200, 20000, 128, 16, 1), _inputs(200, 20000, 128, 16, 2, masked=0.6)
    want = [_call(*x, 1.0) for x in (a, b)]
    bufs = [a[0].clone(), a[1].clone(), _t(a[2]), _t(a[3]), _t(a[4])]
    d_h, dW = torch.empty((200, 128), device=DEV), torch.empty((20000, 128), device=DEV)
    loss, acc = torch.empty(200, device=DEV), _lib.new_step_acc(DEV)
    ws = torch.empty(_lib.grpo_lmhead_distill_workspace_size(200, 20000, 128, 16), dtype=torch.uint8, device=DEV)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        _lib.grpo_lmhead_distill_topk_fwd_bwd(*bufs, 1.0, d_h, dW, loss, acc, ws)
    for x, e in zip((a, b), want):
        for dst, src in zip(bufs, x):
            dst.copy_(src if isinstance(src, torch.Tensor) else _t(src))
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(loss, e[0]) and torch.equal(d_h, e[1]) and torch.equal(dW, e[2])


def test_product_sizes_on_sampled_rows():
    T, V, H, K = 640, W.V_QWEN, 2048, 64
    h, Wt, idx, lq, mask = _inputs(T, V, H, K, 3, std=0.02)
    scale = 1.0 / max(int(mask.sum()), 1)
    loss, d_h, dW, _ = _call(h, Wt, idx, lq, mask, scale)
    rows = np.r_[0:6, 300:304, T - 3:T]
    sub = (h[torch.from_numpy(rows).to(DEV)].contiguous(), Wt, idx[rows], lq[rows], mask[rows])
    _check(sub, scale, (loss[rows], None, None, None))
    hd, wd, _, _, dz, bz = _reference(*sub, scale)
    m = (2.0 ** -8 + 2.0 ** -10) * np.abs(dz) + 1.01 * bz
    e = np.abs(d_h[rows].double().cpu().numpy() - dz @ wd)
    assert np.all(e <= m @ np.abs(wd) + 1e-12), float(e.max())


def test_binding_refuses_what_the_call_cannot_take():
    h, Wt, idx, lq, mask = a = _inputs(8, 300, 64, 4, 0)
    with pytest.raises(_lib.GrpoError) as e:
        _call(*a, 1.0, ws=torch.empty(_lib.grpo_lmhead_distill_workspace_size(8, 300, 64, 4) - 256, dtype=torch.uint8,
                                      device=DEV))
    assert e.value.code == _lib.ERR_CAPACITY
    with pytest.raises(ValueError):
        _call(h, Wt[:, :32], idx, lq, mask, 1.0)
    with pytest.raises(ValueError):
        _call(h.float(), Wt, idx, lq, mask, 1.0)
    with pytest.raises(ValueError):
        _call(h, Wt, idx[:4], lq[:4], mask, 1.0)
    with pytest.raises(_lib.GrpoError):
        _call(h, Wt, idx, lq, mask, float("nan"))

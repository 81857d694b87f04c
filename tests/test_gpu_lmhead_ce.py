"""GPU parity of the cross entropy from hidden states against the float64 oracle: per-token loss, log-prob
and lse, d_h and dW over ragged extents, one and several vocabulary pieces, masks, weights, label
smoothing, z-loss, soft cap, both tile shapes and both gradient types.

Tolerances. Log-probs and lse within 1e-5 max(1, |value|), the LM-head tests' bar; the loss the sum of its
terms' bars. dx before its rounding: p's relative error is its log-prob's bar and 2^-21, the other parts
2^-21 of theirs, the cap's derivative 1e-5. dx enters the products as bf16, half a step (2^-8) of each
entry, with float32 sums (2^-10 for the longest): |d| <= ((2^-8 + 2^-10) |dx| + bar) |W|, and 2^-8 of the
result once more where that is bf16."""
import math

import numpy as np
import pytest
import torch

from oracle import ce as OC
from rl_post_token_gb300 import _lib

pytestmark = pytest.mark.gpu
DEV = "cuda"
F32, BF16 = torch.float32, torch.bfloat16


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


def _inputs(T, V, H, seed, masked=0.2, std=1.0):
    rng = np.random.default_rng(seed)
    h = torch.from_numpy(rng.standard_normal((T, H)).astype(np.float32)).to(BF16).to(DEV)
    Wt = torch.from_numpy((std / math.sqrt(H) * rng.standard_normal((V, H))).astype(np.float32)).to(BF16).to(DEV)
    y = rng.integers(0, V, T).astype(np.int32)
    mask = None if masked is None else (rng.random(T) >= masked).astype(np.uint8)
    return h, Wt, y, mask


def _call(h, Wt, y, mask, scale, w=None, dt=(F32, F32), grads=True, dW=None, ws=None, d_h=None, **kw):
    T, H = h.shape
    V = Wt.shape[0]
    if grads and d_h is None:
        d_h = torch.full((T, H), 7.0, device=DEV, dtype=dt[0])
    if grads and dW is None:
        dW = torch.full((V, H), 7.0, device=DEV, dtype=dt[1])
    loss, logp, lse = (torch.full((T,), -7.0, device=DEV) for _ in range(3))
    acc = _lib.new_step_acc(DEV)
    if ws is None:
        ws = torch.full((_lib.grpo_lmhead_ce_workspace_size(T, V, H),), 255, dtype=torch.uint8, device=DEV)
    _lib.grpo_lmhead_ce_fwd_bwd(h, Wt, _t(y), _t(mask), scale, d_h, dW, loss, acc, ws, w_tok=_t(w), logp_tok=logp,
                                lse_tok=lse, **kw)
    torch.cuda.synchronize()
    return dict(loss=loss, logp=logp, lse=lse, d_h=d_h, dW=dW, acc=acc)


def _np(t):
    return t.double().cpu().numpy()


def _check(args, scale, out, w=None, dw0=None, label_smoothing=0.0, z_loss=0.0, soft_cap=0.0):
    h, Wt, y, mask = args
    hd, wd = _np(h), _np(Wt)
    eps, lam = label_smoothing, z_loss
    ref = OC.lmhead(hd, wd, y, mask, scale, w, eps, lam, soft_cap)
    T, V = len(y), wd.shape[0]
    bar = {k: np.zeros(T) for k in ("loss", "logp", "lse")}
    bdx = np.zeros((T, V))
    for t in range(T):
        p = ref["parts"][t]
        if p is None:
            hd[t] = 0.0
            continue
        rel = lambda v: 1e-5 * np.maximum(1.0, np.abs(v))
        lse, lp = p["lse"], p["logp"]
        bar["logp"][t], bar["lse"][t] = rel(lp[y[t]]), rel(lse)
        bar["loss"][t] = (1 - eps) * rel(lp[y[t]]) + eps * rel(np.mean(lp)) + lam * 2 * abs(lse) * rel(lse) \
            + 2.0 ** -22 * abs(ref["loss"][t])
        g = abs(scale) * (1.0 if w is None else float(w[t]))
        cp = abs(1 + 2 * lam * lse) * p["p"]
        hot = np.zeros(V)
        hot[y[t]] = 1 - eps
        bdx[t] = g * p["d"] * (cp * (rel(lp) + 2.0 ** -21) + 2 * lam * rel(lse) * p["p"]
                               + 2.0 ** -21 * (hot + eps / V))
        if soft_cap:
            bdx[t] += 1e-5 * np.abs(ref["dx"][t])
    for k in ("loss", "logp", "lse"):
        err = np.abs(_np(out[k]) - ref[k])
        assert np.all(err <= bar[k]), (k, int(np.argmax(err - bar[k])), err.max())
    if out["d_h"] is None:
        return
    m = (2.0 ** -8 + 2.0 ** -10) * np.abs(ref["dx"]) + 1.01 * bdx
    for k, want, tol in (("d_h", ref["d_h"], m @ np.abs(wd)), ("dW", ref["dW"], m.T @ np.abs(hd))):
        got = out[k]
        if k == "dW" and dw0 is not None:
            want = want + _np(dw0)
            tol = tol + 2.0 ** -23 * np.abs(want)
        if got.dtype == BF16:
            tol = tol + 2.0 ** -8 * (np.abs(want) + tol)
        e = np.abs(_np(got) - want)
        assert np.all(e <= tol + 1e-30), (k, e.max(), float((e - tol).max()))
    if mask is not None:
        assert np.all(_np(out["d_h"])[mask == 0] == 0)


TERMS = [dict(), dict(label_smoothing=0.1), dict(z_loss=1e-3, soft_cap=3.0),
         dict(label_smoothing=0.25, z_loss=1e-2, soft_cap=30.0), dict(label_smoothing=1.0)]


@pytest.mark.parametrize("terms", TERMS)
@pytest.mark.parametrize("T, V, H, masked", [(1, 1, 8, None), (1, 5, 64, None), (2, 300, 72, 0.5), (130, 3000, 128, 0.2),
                                             (257, 1027, 200, None), (300, 17153, 264, 0.3), (64, 40000, 1032, 0.2)])
def test_parity(cta_group, terms, T, V, H, masked):
    a = _inputs(T, V, H, T + V, masked)
    w = np.random.default_rng(0).random(T).astype(np.float32)
    _check(a, 0.7, _call(*a, 0.7, **terms), **terms)
    _check(a, 1.0 / T, _call(*a, 1.0 / T, w=w, dt=(BF16, BF16), **terms), w=w, **terms)


@pytest.mark.parametrize("T, V, masked", [(700, 35000, 0.4), (1100, 35000, None), (150, 6000, 0.4)])
def test_logits_kept_and_formed_again(cta_group, T, V, masked):
    # (the kept ones take 48 MB at most; few of them are joined and turned into dlogits by one kernel)
    a = _inputs(T, V, 64, 3, masked)
    kw = dict(label_smoothing=0.1, z_loss=1e-3)
    _check(a, 1.0, _call(*a, 1.0, **kw), **kw)
    _check(a, 1.0, _call(*a, 1.0, dt=(BF16, F32), **kw), **kw)


def _check64(args, scale, out, w=None, label_smoothing=0.0, z_loss=0.0, soft_cap=0.0):
    """_check on the GPU in float64, all tokens at once (for calls too large for the row oracle)."""
    h, Wt, y, mask = args
    live = torch.ones(len(y), dtype=torch.bool, device=DEV) if mask is None else _t(mask) != 0
    hd, wd, at = h.double()[live], Wt.double(), _t(y).long()[live][:, None]
    V = wd.shape[0]
    x = hd @ wd.T
    z = soft_cap * torch.tanh(x / soft_cap) if soft_cap else x
    d = 1 / torch.cosh(x / soft_cap) ** 2 if soft_cap else 1.0
    lse = torch.logsumexp(z, 1, keepdim=True)
    lp = z - lse
    logp, mean = lp.gather(1, at), lp.mean(1, keepdim=True)
    loss = -(1 - label_smoothing) * logp - label_smoothing * mean + z_loss * lse ** 2
    rel = lambda v: 1e-5 * v.abs().clamp(min=1.0)
    bar = (1 - label_smoothing) * rel(logp) + label_smoothing * rel(mean) + 2 * z_loss * lse.abs() * rel(lse) + 2.0 ** -22 * loss.abs()
    for k, want, tol in (("logp", logp, rel(logp)), ("lse", lse, rel(lse)), ("loss", loss, bar)):
        assert torch.all((out[k].double()[live] - want[:, 0]).abs() <= tol[:, 0]), k
        assert torch.all(out[k][~live] == 0), k
    g = torch.full_like(lse, abs(scale)) if w is None else abs(scale) * _t(w).double()[live][:, None]
    p, hot = lp.exp(), torch.zeros_like(lp).scatter_(1, at, 1 - label_smoothing)
    dx = g * d * ((1 + 2 * z_loss * lse) * p - hot - label_smoothing / V)
    m = (2.0 ** -8 + 2.0 ** -10) * dx.abs() + 1.01 * g * d * (
        (1 + 2 * z_loss * lse).abs() * p * (rel(lp) + 2.0 ** -21) + 2 * z_loss * rel(lse) * p
        + 2.0 ** -21 * (hot + label_smoothing / V)) + (1e-5 * dx.abs() if soft_cap else 0.0)
    full = torch.zeros(h.shape, dtype=torch.float64, device=DEV)
    d_h, tol_h = full.clone(), full
    d_h[live], tol_h[live] = dx @ wd, m @ wd.abs()
    for k, want, tol in (("d_h", d_h, tol_h), ("dW", dx.T @ hd, m.T @ hd.abs())):
        if out[k].dtype == BF16:
            tol = tol + 2.0 ** -8 * (want.abs() + tol)
        e = (out[k].double() - want).abs()
        assert torch.all(e <= tol + 1e-30), (k, float(e.max()), float((e - tol).max()))


@pytest.mark.parametrize("terms", [dict(), dict(label_smoothing=0.1, z_loss=1e-3, soft_cap=5.0)])
@pytest.mark.parametrize("masked", [None, 0.5])
def test_several_vocabulary_pieces(cta_group, masked, terms):
    # a piece has 256 MB of dlogits: 124 tiles of 256 columns at 4200 tokens; two pieces, the second's last
    # tile and K block ragged
    a = _inputs(4200, 35001, 72, 3, masked)
    w = np.random.default_rng(1).random(4200).astype(np.float32)
    _check64(a, 0.3, _call(*a, 0.3, **terms), **terms)
    _check64(a, 0.3, _call(*a, 0.3, w=w, dt=(BF16, BF16), **terms), w=w, **terms)
    base = torch.randn((35001, 72), device=DEV)
    one, buf = _call(*a, 1.0, **terms), base.clone()
    two = _call(*a, 1.0, dW=buf, dw_accumulate=True, dt=(BF16, F32), **terms)
    assert torch.equal(buf, base + one["dW"]) and torch.equal(two["d_h"], one["d_h"].to(BF16))


@pytest.mark.parametrize("T, V, H", [(70_001, 300, 24), (400_003, 70, 8)])
def test_many_tokens(T, V, H):
    # (several rounds of the compaction's blocks)
    a = _inputs(T, V, H, 16, 0.3)
    a[3][a[3] != 0] = np.random.default_rng(2).integers(1, 256, int(a[3].sum()))  # any value but 0 counts
    w = (np.random.default_rng(1).random(T) - 0.3).astype(np.float32)
    kw = dict(label_smoothing=0.1, z_loss=1e-3)
    _check64(a, 1.0 / T, _call(*a, 1.0 / T, **kw), **kw)
    _check64(a, 1.0 / T, _call(*a, 1.0 / T, w=np.abs(w), **kw), w=np.abs(w), **kw)
    plus, minus = _call(*a, 1.0 / T, w=w, **kw), _call(*a, -1.0 / T, w=-w, **kw)
    assert torch.equal(plus["d_h"], minus["d_h"]) and torch.equal(plus["dW"], minus["dW"])


def test_offsets_past_2_to_the_31():
    # W and dW of 2.2e9 elements, targets among the last rows
    T, V, H = 64, 1_100_000, 2048
    g = torch.Generator(device=DEV)
    g.manual_seed(0)
    Wt = torch.empty((V, H), dtype=BF16, device=DEV)
    for a in range(0, V, 100_000):
        Wt[a:a + 100_000] = (torch.randn((100_000, H), generator=g, device=DEV) / math.sqrt(H)).to(BF16)
    h = torch.randn((T, H), generator=g, device=DEV).to(BF16)
    y = (V - 1 - np.arange(T) * 331).astype(np.int32)
    out = _call(h, Wt, y, None, 1.0, dt=(BF16, BF16))
    x = torch.cat([h.double() @ Wt[a:a + 100_000].double().T for a in range(0, V, 100_000)], 1)
    lse = torch.logsumexp(x, 1, keepdim=True)
    logp = (x - lse).gather(1, _t(y).long()[:, None])[:, 0]
    assert torch.all((out["logp"].double() - logp).abs() <= 1e-5 * logp.abs())
    dx = (x - lse).exp()
    dx[torch.arange(T, device=DEV), _t(y).long()] -= 1
    rows = torch.tensor([0, 1, V // 2, 1_048_575, 1_048_576, V - 332, V - 2, V - 1], device=DEV)
    hd = h.double()
    want, tol = dx[:, rows].T @ hd, dx[:, rows].abs().T @ hd.abs()
    e = (out["dW"][rows].double() - want).abs()
    assert torch.all(e <= (2.0 ** -8 + 2.0 ** -9) * tol + 2.0 ** -8 * want.abs())
    want = sum(dx[:, a:a + 100_000] @ Wt[a:a + 100_000].double() for a in range(0, V, 100_000))
    size = sum(dx[:, a:a + 100_000].abs() @ Wt[a:a + 100_000].double().abs() for a in range(0, V, 100_000))
    assert torch.all((out["d_h"].double() - want).abs() <= (2.0 ** -8 + 2.0 ** -9) * size + 2.0 ** -8 * want.abs())


def _random_case(seed):
    rng = np.random.default_rng(1000 + seed)
    log = lambda lo, hi: int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    T, V, H = log(1, 3000), log(1, 30000), 8 * log(1, 100)
    kw = dict(label_smoothing=float(rng.choice([0, 0, 0.1, 0.6])), z_loss=float(rng.choice([0, 1e-4, 0.05])),
              soft_cap=float(rng.choice([0, 0, 2.0, 30.0])))
    dt = (F32, BF16)
    return (T, V, H), kw, (dt[rng.integers(2)], dt[rng.integers(2)]), rng.choice([None, 0.0, 0.3, 0.9]), rng


@pytest.mark.parametrize("seed", range(40))
def test_random_calls(seed, monkeypatch):
    (T, V, H), kw, dt, masked, rng = _random_case(seed)
    if seed % 3:
        monkeypatch.setenv("GRPO_LMHEAD_CTA_GROUP", str(seed % 3))
    a = _inputs(T, V, H, seed, masked, std=float(rng.choice([0.3, 1.0, 4.0])))
    w = rng.random(T).astype(np.float32) if rng.random() < 0.4 else None
    scale = float(rng.choice([1.0, 1.0 / T, 3e-5]))
    _check64(a, scale, _call(*a, scale, w=w, dt=dt, **kw), w=w, **kw)


def test_masked_tokens_may_hold_anything(cta_group):
    h, Wt, y, mask = _inputs(150, 2000, 136, 5, 0.5)
    a = _call(h, Wt, y, mask, 1.0, label_smoothing=0.1)
    h2, y2 = h.clone(), y.copy()
    h2[torch.from_numpy(mask == 0)] = float("nan")
    y2[mask == 0] = np.where(np.arange((mask == 0).sum()) % 2, -100, 2 ** 31 - 1)
    b = _call(h2, Wt, y2, mask, 1.0, label_smoothing=0.1)
    for k in ("loss", "logp", "lse", "d_h", "dW"):
        assert torch.equal(a[k], b[k]), k
    res = _lib.grpo_finish_step(b["acc"], b["loss"], expected_N=int(mask.sum()))
    assert res["status"] == 0 and res["n_tokens"] == 150 and res["n_clipped"] == 0


@pytest.mark.parametrize("T", [1, 63, 64, 65, 300])
def test_nothing_unmasked(cta_group, T):
    h, Wt, y, _ = _inputs(T, 700, 64, 6)
    out = _call(h, Wt, y, np.zeros(T, np.uint8), 1.0, dt=(BF16, F32), z_loss=1e-3)
    assert all(torch.all(out[k] == 0) for k in ("loss", "logp", "lse", "d_h", "dW"))
    res = _lib.grpo_finish_step(out["acc"], out["loss"], expected_N=0)
    assert res["status"] == 0 and res["n_valid"] == 0


def test_full_mask_weights_of_zero_and_loss_only():
    h, Wt, y, _ = _inputs(200, 3000, 128, 7, None)
    a = _call(h, Wt, y, None, 1.0)
    b = _call(h, Wt, y, np.ones(200, np.uint8), 1.0)
    c = _call(h, Wt, y, None, 1.0, grads=False)
    for k in ("loss", "logp", "lse", "d_h", "dW"):
        assert torch.equal(a[k], b[k]), k
        assert k[0] == "d" or torch.equal(a[k], c[k]), k
    w = np.ones(200, np.float32)
    w[50:] = 0
    d = _call(h, Wt, y, None, 1.0, w=w)
    assert torch.equal(d["loss"], a["loss"]) and torch.all(d["d_h"][50:] == 0)
    assert torch.equal(d["d_h"][:50], a["d_h"][:50])
    only = [_call(h, Wt, y, None, 1.0, grads=False, dW=torch.empty_like(a["dW"])),
            _call(h, Wt, y, None, 1.0, grads=False, d_h=torch.empty_like(a["d_h"]))]
    assert torch.equal(only[0]["dW"], a["dW"]) and torch.equal(only[1]["d_h"], a["d_h"])


def test_accumulating_dw_sums_the_calls():
    a = _inputs(300, 20000, 256, 4, 0.5)
    one = _call(*a, 1.0)
    base = torch.randn_like(one["dW"])
    buf = base.clone()
    two = _call(*a, 1.0, dW=buf, dw_accumulate=True)
    assert torch.equal(two["d_h"], one["d_h"]) and torch.equal(buf, base + one["dW"])


def test_no_tokens():
    dW = torch.full((40, 64), 7.0, device=DEV, dtype=BF16)
    e = lambda *s, dt=F32: torch.empty(s, dtype=dt, device=DEV)
    args = (e(0, 64, dt=BF16), e(40, 64, dt=BF16), e(0, dt=torch.int32), None, 1.0, e(0, 64))
    _lib.grpo_lmhead_ce_fwd_bwd(*args, dW, e(0), _lib.new_step_acc(DEV), e(0, dt=torch.uint8))
    assert torch.all(dW == 0)
    keep = torch.full((40, 64), 7.0, device=DEV)
    _lib.grpo_lmhead_ce_fwd_bwd(*args, keep, e(0), _lib.new_step_acc(DEV), e(0, dt=torch.uint8), dw_accumulate=True)
    assert torch.all(keep == 7)


@pytest.mark.parametrize("what", ["target", "negative", "nan", "inf", "range"])
def test_a_non_finite_token_skips_the_step(what):
    h, Wt, y, mask = _inputs(70, 900, 64, 8, None)
    if what == "target":
        y[3] = 900
    elif what == "negative":
        y[3] = -2 ** 31
    elif what == "nan":
        h[3, 5] = float("nan")
    elif what == "inf":
        h[3, 5] = float("inf")
    else:
        h[3] = 20000 * torch.sign(Wt[11])
    out = _call(h, Wt, y, mask, 1.0, z_loss=1e-3, label_smoothing=0.1)
    assert torch.isnan(out["loss"][3]) and torch.isfinite(out["loss"][4:]).all()
    res = _lib.grpo_finish_step(out["acc"], out["loss"], expected_N=70, grad_bufs=[out["d_h"], out["dW"]])
    assert res["status"] == _lib.STEP_SKIPPED_NONFINITE and res["n_nonfinite"] == 1
    assert torch.all(out["d_h"] == 0) and torch.all(out["dW"] == 0)


@pytest.mark.parametrize("cap", [1e-6, 0.5, 1e6])
def test_saturated_caps(cap):
    # every logit at the cap, or none near it
    a = _inputs(40, 600, 64, 9, None, std=30.0)
    kw = dict(soft_cap=cap, z_loss=1e-4)
    _check(a, 1.0, _call(*a, 1.0, **kw), **kw)


@pytest.mark.parametrize("T", [64, 600])
def test_a_token_does_not_see_its_neighbours_logits(T):
    # (the cap's short form is taken where a warp's rows allow it: the same bits as the long one's)
    h, Wt, y, _ = _inputs(T, 3000, 128, 15, None)
    kw = dict(soft_cap=30.0, z_loss=1e-4, label_smoothing=0.1)
    a = _call(h, Wt, y, None, 1.0, **kw)
    h2 = h.clone()
    h2[5] *= 200
    h2[40, 3] = float("nan")
    b = _call(h2, Wt, y, None, 1.0, **kw)
    same = torch.ones(T, dtype=torch.bool, device=DEV)
    same[[5, 40]] = False
    assert b["loss"][5] != a["loss"][5] and torch.isnan(b["loss"][40])
    for k in ("loss", "logp", "lse", "d_h"):
        assert torch.equal(a[k][same], b[k][same]), k


def test_large_and_peaked_logits():
    # log-probs next to 0 and lse far from it
    h, Wt, y, _ = _inputs(96, 4000, 128, 10, None, std=4.0)
    h = (h.float() + 3 * Wt[torch.from_numpy(y).long().to(DEV)].float()).to(BF16)
    for kw in (dict(), dict(label_smoothing=0.1, z_loss=1e-4)):
        _check((h, Wt, y, None), 1.0, _call(h, Wt, y, None, 1.0, **kw), **kw)


def test_streams_and_graph_replay_give_the_bits():
    T, V, H = 4200, 35000, 64  # two pieces: both streams
    a, b = _inputs(T, V, H, 11, 0.3), _inputs(T, V, H, 12, 0.6)
    wa, wb = _call(*a, 1.0, dt=(BF16, BF16)), _call(*b, 1.0, dt=(BF16, BF16))
    h, Wt, y, mask = (x.clone() if torch.is_tensor(x) else _t(x) for x in a)
    ws = torch.empty(_lib.grpo_lmhead_ce_workspace_size(T, V, H), dtype=torch.uint8, device=DEV)
    loss, d_h, dW, acc = torch.empty(T, device=DEV), torch.empty_like(h), torch.empty_like(Wt), _lib.new_step_acc(DEV)
    run = lambda: _lib.grpo_lmhead_ce_fwd_bwd(h, Wt, y, mask, 1.0, d_h, dW, loss, acc, ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
    side.synchronize()
    assert torch.equal(loss, wa["loss"]) and torch.equal(d_h, wa["d_h"]) and torch.equal(dW, wa["dW"])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run()
    for src, want in ((b, wb), (a, wa), (b, wb)):
        for to, x in zip((h, Wt, y, mask), src):
            to.copy_(x if torch.is_tensor(x) else _t(x))
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(loss, want["loss"]) and torch.equal(d_h, want["d_h"]) and torch.equal(dW, want["dW"])


def test_an_eager_call_during_another_streams_capture():
    # the capture holds the second stream until it ends; the eager call keeps to its own
    T, V, H = 4200, 35000, 64
    a, b = _inputs(T, V, H, 11, 0.3), _inputs(T, V, H, 12, 0.6)
    wa, wb = _call(*a, 1.0), _call(*b, 1.0)

    def buffers(x):
        h, Wt, y, mask = x
        return [h, Wt, _t(y), _t(mask), torch.zeros((T, H), device=DEV), torch.zeros((V, H), device=DEV),
                torch.zeros(T, device=DEV), _lib.new_step_acc(DEV),
                torch.empty(_lib.grpo_lmhead_ce_workspace_size(T, V, H), dtype=torch.uint8, device=DEV)]

    def call(z):
        _lib.grpo_lmhead_ce_fwd_bwd(*z[:4], 1.0, *z[4:])

    za, zb = buffers(a), buffers(b)
    side, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, capture_error_mode="relaxed"):
        call(za)
        with torch.cuda.stream(side):
            call(zb)
    side.synchronize()
    assert torch.equal(zb[6], wb["loss"]) and torch.equal(zb[4], wb["d_h"]) and torch.equal(zb[5], wb["dW"])
    assert torch.all(za[6] == 0)
    g.replay()
    call(zb)
    torch.cuda.synchronize()
    for z, want in ((za, wa), (zb, wb)):
        assert torch.equal(z[6], want["loss"]) and torch.equal(z[4], want["d_h"]) and torch.equal(z[5], want["dW"])


def test_micro_batches_sum_to_the_whole_step():
    T, V, H = 512, 5000, 128
    h, Wt, y, mask = _inputs(T, V, H, 13, 0.3)
    N = int(mask.sum())
    whole = _call(h, Wt, y, mask, 1.0 / N)
    dW = torch.zeros_like(whole["dW"])
    for a in range(0, T, 128):
        out = _call(h[a:a + 128], Wt, y[a:a + 128], mask[a:a + 128], 1.0 / N, dW=dW, dw_accumulate=True)
        assert torch.equal(out["loss"], whole["loss"][a:a + 128])
    # the same bf16 products summed in two orders: n float32 additions are off by at most n 2^-23 of the sum
    # of the terms' sizes each (2^-23: rounded towards zero or to nearest), n < 516 with the four calls'
    # joining, so the two differ by 2 x 516 x 2^-23 < 2^-12.9 of it (a bound of 2^-20 took no account of n)
    tol = 2.0 ** -12.9 * (torch.from_numpy(np.abs(OC.lmhead(_np(h), _np(Wt), y, mask, 1.0 / N)["dx"]).T @ np.abs(_np(h))))
    assert torch.all((dW - whole["dW"]).abs().double().cpu() <= tol)


def test_refusals():
    h, Wt, y, mask = _inputs(16, 100, 64, 14)
    with pytest.raises(_lib.GrpoError):
        _call(h, Wt, y, mask, 1.0, label_smoothing=1.5)
    for bad in (dict(dw_accumulate=True, dt=(F32, BF16)), dict(z_loss=-1.0), dict(soft_cap=-1.0),
                dict(soft_cap=float("nan")), dict(z_loss=float("inf")),
                dict(ws=torch.empty(256, dtype=torch.uint8, device=DEV))):
        with pytest.raises(_lib.GrpoError):
            _call(h, Wt, y, mask, 1.0, **bad)
    with pytest.raises(_lib.GrpoError):
        _call(h, Wt, y, mask, float("nan"))
    with pytest.raises(_lib.GrpoError):
        _call(h[:, :60].contiguous(), Wt[:, :60].contiguous(), y, mask, 1.0)
    with pytest.raises(ValueError):
        _call(h[:, :32], Wt[:, :32], y, mask, 1.0)
    with pytest.raises(ValueError):
        _call(h, Wt, y.astype(np.int64), mask, 1.0)
    with pytest.raises(ValueError):
        _call(h, Wt, y, mask[:8], 1.0)
    with pytest.raises(ValueError):
        _call(h, Wt, y, mask, 1.0, dt=(torch.float16, F32))

"""The remainder of the tail kinds at its ends: rows without a list, and FORWARD_TAIL where nearly all of
the student's mass is on the listed tokens: the remainder p_R, far below the float32 range as a share of
the row, still has a finite logarithm, and the tokens outside the list still share the gradient -q_R by
their shares of p_R.

Tolerances (t, E and dS as in test_gpu_distill: U = 2^-24, dS = 2^-22 + 50 U + 2 U E|t| ln2 of a sum of
exponentials). Outside the list the kernel forms dlogits = (mass p_R - q_R) g/s 2^t with t taken from the
largest logit outside, d = |t| ln2, and s their sum there:
  2^t / s             relative dS_out + 2^-22 + 2 U d + 2 U
  p_R                 relative dS_out + dS + 2^-22 + 2 U |log p_R| + 4 U, absolute 2^-126 (underflow)
  mass p_R - q_R      mass (p_R's error) + 2 U (mass p_R + q_R); the scale adds four roundings
Loss: the listed terms as in test_gpu_distill, and q_R times the error of log p_R, which is
((m_out - m) + log2 s - log2 S) ln2: dS_out + dS + 2 U (log s + log S) + 4 U |log p_R| (log2(e)/tau
rounded twice, the difference and the product) + 3 U |log q_R/p_R|. The output type adds half a step;
2^-126 (1 + |g|) covers what underflows."""
import numpy as np
import pytest
import torch

from oracle import distill as OD
from oracle import loss as OL
from rl_post_token_gb300 import _lib
from rl_post_token_gb300 import workloads as W
from tests import test_gpu_distill as D

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = D.U


@pytest.fixture(scope="module", autouse=True)
def _built(grpo_lib):
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return grpo_lib


def _check_row(got_loss, got_dz, z, idx, lq, tau, g, dtype):
    loss, dx, parts = OD.row_loss(z, idx, lq, OD.FORWARD_TAIL, tau)
    assert np.isfinite(loss) and np.isfinite(dx).all()
    z = OL.as_f64(np.asarray(z))
    on = idx != -1
    S, lq = idx[on], lq[on].astype(np.float64)
    out = np.ones(z.shape[0], bool)
    out[S] = False
    p, lp, q, qr = parts["p"], parts["lp"], parts["q"], parts["qr"]
    d = (z.max() - z) / tau
    dS = 2.0 ** -22 + 50 * U + 2 * U * float((p * d).sum())
    do = (z[out].max() - z[out]) / tau
    eo = np.exp(-do)
    s = eo.sum()
    dSo = 2.0 ** -22 + 50 * U + 2 * U * float((eo * do).sum() / s)
    lr = -(z.max() - z[out].max()) / tau + np.log(s) - np.log(parts["tot"])
    pr, mass = np.exp(lr), q.sum() + qr
    lq0 = np.where(np.isfinite(lq), lq, 0.0)
    dlp = dS + U * np.log(parts["tot"]) + 2 * U * (d[S] + np.abs(lp[S]))
    dp = dS + 2.0 ** -22 + 2 * U * d[S] + 6 * U
    bl = np.sum(q * (dlp + 16 * U * np.abs(lq0 - lp[S]) + U * (np.abs(lq0) + np.abs(lp[S]))))
    if qr > 0:
        bl += qr * (dSo + dS + 2 * U * (np.log(s) + np.log(parts["tot"])) + 4 * U * abs(lr) + 3 * U * abs(np.log(qr) - lr))
    bl += 2 * U * abs(loss)
    assert abs(got_loss - loss) <= bl, (got_loss, loss, bl)
    b = np.empty(z.shape[0])
    head = mass * (pr * (dSo + dS + 2.0 ** -22 + 2 * U * abs(lr) + 4 * U) + 2.0 ** -126) + 2 * U * (mass * pr + qr)
    b[out] = eo / s * (head + abs(mass * pr - qr) * (dSo + 2.0 ** -22 + 2 * U * do + 6 * U))
    b[S] = p[S] * mass * (dp + 2 * U) + 3 * U * q + U * np.abs(p[S] - q)
    b *= abs(g) / tau
    ref = dx * g
    tol = b + (D.HALF[dtype] + 5 * U) * (np.abs(ref) + b) + 2.0 ** -126 * (1.0 + abs(g))
    err = np.abs(got_dz - ref)
    v = int(np.argmax(err - tol))
    assert np.all(err <= tol), (v, got_dz[v], ref[v], err[v], tol[v], v in S)


# the kernels: a CTA per row (few rows, and many), a cluster; the last column is a temperature
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T, V, tau", [(10, 1000, 1.0), (10, 5003, 0.25), (320, 1000, 1.0), (10, 40000, 1.0),
                                       (170, 40001, 0.25), (10, 151936, 1.0), (4, 800008, 1.0)])
def test_a_remainder_below_the_float32_range(T, V, tau, dtype):
    K, n = 6, 10
    rng = np.random.default_rng(V)
    z = np.empty((n, V), np.float32)
    gap = np.array([80.0, 86.0, 87.0, 88.0, 95.0, 100.0, 120.0, 1000.0, 1e4, 3e5]) * (0.28 if tau < 1 else 1.0)
    idx = np.stack([rng.permutation(V)[:K] for _ in range(n)]).astype(np.int32)
    for r in range(n):
        z[r] = -gap[r] + rng.standard_normal(V)
        if r == 4:  # two levels outside: 2/V of the tokens hold most of the remainder, the others a third or so
            z[r] = -gap[r] - 4.5 * tau
            z[r, rng.permutation(V)[:max(V // 50, 1)]] = -gap[r]
        z[r, idx[r]] = 0.5 * rng.standard_normal(K)
    lq = np.log(rng.dirichlet(np.ones(K + 1), n)[:, :K] + 1e-4).astype(np.float32)
    lq[1] = np.log(0.2 / 6)
    lq[2] = np.log((1.0 - 1e-5) / 6)
    idx[3, 2], lq[3, 2] = -1, 0.0
    rows = np.arange(T) % n
    lg = torch.from_numpy(z).to(DEV).to(D.DT[dtype])[torch.from_numpy(rows).to(DEV)].contiguous()
    zh = W.logits_to_host(lg[:min(T, n)])
    w = (0.5 + rng.random(T)).astype(np.float32)
    scale = 1.0 / 7
    loss, dz, acc = D._call(lg, idx[rows], lq[rows], _lib.DISTILL_FORWARD_TAIL, scale, temperature=tau, w=w)
    res = _lib.grpo_finish_step(acc, loss, expected_N=T, grad_bufs=[dz])
    assert res["n_nonfinite"] == 0 and res["status"] == 0
    lh = loss.double().cpu().numpy()
    for r in sorted(set(range(min(T, n))) | {T - 1}):
        _check_row(lh[r], dz[r].double().cpu().numpy(), zh[r % n], idx[r % n], lq[r % n], tau, scale * float(w[r]), dtype)
    only, _, _ = D._call(lg, idx[rows], lq[rows], _lib.DISTILL_FORWARD_TAIL, scale, temperature=tau, w=w, dz=None)
    assert torch.equal(only, loss)


def test_tokens_far_below_the_largest_outside_keep_their_gradient():
    # four listed logits at 0 and 20 of the others at -84, 900 at -88.5: a third of the remainder is theirs
    z = torch.full((1, 924), -88.5, device=DEV)
    z[0, :4] = 0.0
    z[0, 4:24] = -84.0
    idx = np.arange(4, dtype=np.int32)[None]
    lq = np.full((1, 4), np.log(0.2), np.float32)
    loss, dz, _ = D._call(z, idx, lq, _lib.DISTILL_FORWARD_TAIL, 1.0)
    q = 0.8
    share = np.exp(-4.5) / (20 + 900 * np.exp(-4.5))
    got = dz[0, 24:].double().cpu().numpy()
    assert np.all(np.abs(got + (1 - q) * share) <= 1e-5 * share)
    assert abs(dz.double().sum().item()) <= 924 * 2.0 ** -24
    assert np.isfinite(loss.item())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T, V", [(5, 300), (400, 1000), (300, 5003), (40, 40000), (3, 151936), (400, 36001)])
def test_rows_without_a_list_have_loss_and_gradient_zero(T, V, dtype):
    # the remainder is everything: 1 log(1/1) and a gradient of 0, not what s/s rounds to
    lg, idx, lq = D._inputs(T, V, 7, dtype, V)
    none = np.arange(T) % 5 != 3
    idx[none] = -1
    for kind in D.KINDS:
        for tau in (1.0, 0.3):
            loss, dz, acc = D._call(lg, idx, lq, kind, 1.0, temperature=tau)
            at = torch.from_numpy(none).to(DEV)
            assert not loss[at].any() and not dz[at].any()
            assert torch.all(dz[~at].abs().amax(1) > 0)
            res = _lib.grpo_finish_step(acc, loss, expected_N=T)
            assert res["n_nonfinite"] == 0 and res["n_valid"] == T
            only, _, _ = D._call(lg, idx, lq, kind, 1.0, temperature=tau, dz=None)
            assert torch.equal(only, loss)
    # such a row is still one that can be bad
    lg[0, 1] = float("nan")
    for kind in D.KINDS:
        loss, dz, acc = D._call(lg, idx, lq, kind, 1.0)
        assert torch.isnan(loss[0]) and torch.isnan(dz[0]).all()
        assert _lib.grpo_finish_step(acc, loss)["n_nonfinite"] == 1


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T, V, K, most", [(400, 4000, 20, 20), (60, 50264, 64, 64), (500, 36001, 256, 200)])
def test_a_teacher_and_a_student_restricted_to_the_same_tokens(T, V, K, most, dtype):
    # every allowed token is listed: the teacher's masses sum to 1 up to the rounding of their log-probs,
    # and the student has nothing outside the list to put a remainder on
    g = torch.Generator(device=DEV).manual_seed(V)
    allow = torch.rand((T, V), device=DEV, generator=g).argsort(1) < torch.randint(2, most + 1, (T, 1), generator=g, device=DEV)
    masks = torch.tensor([-float("inf"), torch.finfo(D.DT[dtype]).min, -1e4, -1e9, -1e30], device=DEV)
    floor = masks[torch.randint(0, 5, (T, 1), generator=g, device=DEV)]
    rows = [torch.where(allow, 2 * torch.randn((T, V), generator=g, device=DEV), floor).to(D.DT[dtype]) for _ in range(2)]
    ti, tl = torch.empty((T, K), dtype=torch.int32, device=DEV), torch.empty((T, K), device=DEV)
    _lib.grpo_token_topk_logprobs(rows[0], K, top_idx=ti, top_logp=tl)
    rest = 1.0 - tl.double().exp().sum(1)
    assert int((rest >= 2.0 ** -24).sum()) > 0 and float(rest.abs().max()) < 2.0 ** -16
    idx, lq = ti.cpu().numpy(), tl.cpu().numpy()
    for kind in D.KINDS:
        loss, dz, acc = D._check(rows[1], idx, lq, kind, scale=1.0 / T, dtype=dtype, rows=range(0, T, 7))
        res = _lib.grpo_finish_step(acc, loss, expected_N=T, grad_bufs=[dz])
        assert res["n_nonfinite"] == 0 and res["status"] == 0 and torch.isfinite(dz).all()
        assert not dz[~allow].any()
    # a remainder worth the name still has no place to go
    lq[:, 0] -= 0.01
    loss, _, acc = D._call(rows[1], idx, lq, _lib.DISTILL_FORWARD_TAIL, 1.0)
    short = 1.0 - np.exp(lq.astype(np.float64)).sum(1) >= 2.0 ** -15
    away = (floor[:, 0] < -3e38).cpu().numpy()
    assert torch.isinf(loss[torch.from_numpy(short & away).to(DEV)]).all() and (short & away).any()
    assert torch.isfinite(loss[torch.from_numpy(~away).to(DEV)]).all()


@pytest.mark.parametrize("gap, none", [(80.0, False), (87.0, False), (88.0, True), (100.0, True)])
def test_many_tokens_just_past_the_limit_of_the_float32_range(gap, none):
    # 100,000 tokens hold e^11 times the share of one: what counts is how far each of them lies below the
    # largest (126 ln 2 = 87.34), in the oracle and in the kernel
    V, K = 100000, 8
    z = torch.full((6, V), -gap, device=DEV)
    idx = np.tile(np.arange(K, dtype=np.int32), (6, 1))
    z[:, :K] = torch.linspace(0, -2, K, device=DEV)
    q = np.full(K, 1 / K)
    lq = np.log(np.stack([q * (1 - r) for r in (0.3, 1e-3, 2e-5, 1e-5, 2e-6, 0.0)])).astype(np.float32)
    loss, dz, _ = D._call(z, idx, lq, _lib.DISTILL_FORWARD_TAIL, 1.0)
    zh = W.logits_to_host(z)
    for r in range(6):
        _check_row(loss[r].item(), dz[r].double().cpu().numpy(), zh[r], idx[r], lq[r], 1.0, 1.0, "f32")
        # the gradient outside sums to -q_R where it counts (p_R itself is below 2^-100)
        counts = r < 3 or not none
        qr = 1.0 - np.exp(lq[r].astype(np.float64)).sum()
        assert r == 5 or abs(dz[r, K:].double().sum().item() + (qr if counts else 0.0)) <= 1e-5 * qr

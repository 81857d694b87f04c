"""GPU parity of the distillation call against the float64 oracle, every element of dlogits.

Tolerances, from the arithmetic (t = (z - max) log2(e)/tau, E over the student's distribution):
  dS = 2^-22 + 50 2^-24 + 2^-23 ln2 E|t|    relative error of a sum of exponentials (ex2 within
       2^-22; at most 16 additions in a lane, 2 + 5 over the tile, 12 joins and 5 additions over the
       tiles, 8 + 5 over the list, one to add its part, and two rescalings: by the join, and to the
       largest of all logits, 2^-22 each and a product)
  dlp = dS + 2^-24 |log S| + 2^-23 (|z - max|/tau + |log p|)     of a log-prob (natural units)
  dp  = dS + 2^-22 + 2^-23 |t| ln2 + 4 2^-24                     relative, of a probability
       = what 2^t carries, the reciprocal of S and three products
Loss: each term's parts with their errors, and 8 + 5 additions over the list: 13 2^-24 of the terms'
magnitudes; FORWARD_TOPK's q/Q is within 2^-22 (expf within 2^-22 at these arguments, the sum, the reciprocal). dlogits: |alpha p| (relative error of p) + p d(alpha), on
the list p dp + q 2^-22 (FORWARD), p (dp |f - L| + d(f) + dL) (REVERSE); the grad scale adds three
roundings. The output type adds half a step: 2^-8 (bf16) or 2^-24 (float32) of the value, and results
below 2^-126 of the multiplier may be flushed."""
import numpy as np
import pytest
import torch

from oracle import distill as OD
from oracle import loss as OL
from rl_post_token_gb300 import _lib
from rl_post_token_gb300 import workloads as W

pytestmark = pytest.mark.gpu
DEV = "cuda"
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}
KINDS = [_lib.DISTILL_FORWARD_TOPK, _lib.DISTILL_FORWARD_TAIL, _lib.DISTILL_REVERSE_TAIL]
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _built(grpo_lib):
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return grpo_lib


def _bars(z, idx, lq, kind, tau, g, parts, loss):
    """(loss bar, dlogits bar before the output rounding) of a row, float64."""
    V = z.shape[0]
    on = idx != -1
    S, lq = idx[on], lq[on].astype(np.float64)
    p, lp, pr, q, alpha = parts["p"], parts["lp"], parts["pr"], parts["q"], parts["alpha"]
    d = np.where(p > 0, (parts["m"] - z) / tau, 0.0)  # |t| ln2
    dS = 2.0 ** -22 + 50 * U + 2 * U * float((p * d).sum())
    safe_lp = np.where(p > 0, lp, 0.0)
    dlp = dS + U * abs(np.log(parts["tot"])) + 2 * U * (d + np.abs(safe_lp))
    dp = dS + 2.0 ** -22 + 2 * U * d + 6 * U
    dpr = 2 * dS + 4 * U
    pS, lpS = p[S], safe_lp[S]
    lq0 = np.where(np.isfinite(lq), lq, 0.0)
    dz = np.empty(V)
    if kind == OD.FORWARD_TOPK:
        norm = abs(np.log(np.exp(lq - np.max(lq)).sum()) + np.max(lq)) if np.any(lq > -np.inf) else 0.0
        lqn = np.where(q > 0, np.log(np.where(q > 0, q, 1.0)), 0.0)
        dq = 8 * U + 13 * U
        bl = np.sum(q * (dlp[S] + dq + U * (2 * norm + 2 * np.abs(lq0) + 2 * np.abs(lqn))
                         + (3 * U + dq + 13 * U) * np.abs(lqn - lpS)))
        da = 0.0
        dz[:] = abs(alpha) * p * dp
        dz[S] = pS * dp[S] + (dq + 3 * U) * q + U * np.abs(pS - q)
        if alpha == 0.0:
            dz[:] = 0.0
    elif kind == OD.FORWARD_TAIL:
        qr = parts["qr"]
        r = qr / pr if qr > 0 else 0.0
        bl = np.sum(q * (dlp[S] + 16 * U * np.abs(lq0 - lpS) + U * (np.abs(lq0) + np.abs(lpS))))
        bl += qr * (dpr + 3 * U + 3 * U * abs(np.log(r))) if qr > 0 else 0.0
        da = r * (dpr + 3 * U) + 3 * U * (q.sum() + qr)
        dz[:] = abs(alpha) * p * dp + p * da
        dz[S] = pS * (q.sum() + qr) * (dp[S] + 2 * U) + 3 * U * q + U * np.abs(pS - q)
    else:
        f, fr, qr = parts["f"], parts["fr"], parts["qr"]
        df = dlp[S] + 2 * U * np.abs(f) + U * (np.abs(lq0) + np.abs(lpS))
        dfr = dpr + 3 * U + 3 * U * abs(fr)
        bl = np.sum(pS * (df + (dp[S] + 16 * U) * np.abs(f))) + pr * (dfr + (dpr + 3 * U) * abs(fr))
        da = dfr + bl + 3 * U * (abs(fr) + abs(loss))
        dz[:] = np.abs(alpha) * p * dp + p * da
        dz[S] = pS * ((dp[S] + 3 * U) * np.abs(f - loss) + df + bl + 3 * U * (np.abs(f) + abs(loss)))
    bl += 2 * U * abs(loss) + 1e-12
    return bl, dz * abs(g) / tau


def _check_row(got_loss, got_dz, z, idx, lq, kind, tau, g, dtype):
    """g: grad_scale times the token's weight."""
    loss, dx, parts = OD.row_loss(z, idx, lq, kind, tau)
    if np.isnan(loss):
        assert np.isnan(got_loss) and (got_dz is None or np.isnan(got_dz).all())
        return
    if np.isinf(loss):
        assert got_loss == loss
        return
    z = OL.as_f64(np.asarray(z))
    with np.errstate(invalid="ignore", divide="ignore"):
        bl, bz = _bars(z, idx, lq, kind, tau, g, parts, loss)
    assert abs(got_loss - loss) <= bl, (got_loss, loss, bl)
    if got_dz is None:
        return
    ref = dx * g
    mult = abs(parts["alpha"] * g / tau)
    tol = bz + (HALF[dtype] + 5 * U) * (np.abs(ref) + bz) + 2.0 ** -126 * (1.0 + mult)
    err = np.abs(got_dz - ref)
    if not np.all(err <= tol):
        v = int(np.argmax(err - tol))
        raise AssertionError((v, got_dz[v], ref[v], err[v], tol[v], v in idx.tolist(), int((err > tol).sum())))


def _inputs(T, V, K, dtype, seed, tau=1.0, pad=0, offset=0, unused=0.3):
    rng = np.random.default_rng(seed)
    z = rng.standard_normal((T, V)) * 3.0
    idx = np.stack([rng.permutation(V)[:K] for _ in range(T)]).astype(np.int32)
    u = rng.standard_normal((T, K + 1)) * 2
    lq = (u - np.log(np.exp(u).sum(1, keepdims=True)))[:, :K].astype(np.float32)
    np.put_along_axis(z, idx.astype(np.int64), tau * (lq + np.log(V) + 6 + 0.5 * rng.standard_normal((T, K))), 1)
    cut = rng.random((T, K)) < unused
    idx[cut], lq[cut] = -1, 0.5
    buf = torch.full((T * (V + pad) + offset + 8,), 50.0, dtype=DT[dtype], device=DEV)
    lg = buf[offset:offset + T * (V + pad)].view(T, V + pad)[:, :V]
    lg.copy_(torch.from_numpy(z))
    return lg, idx, lq


def _call(lg, idx, lq, kind, scale, mask=None, dz=True, w=None, **kw):
    T = kw.pop("rows", lg.shape[0])
    t = lambda a: a if a is None or isinstance(a, torch.Tensor) else torch.from_numpy(np.ascontiguousarray(a)).to(DEV)
    if dz is True:
        dz = torch.full(lg.shape, 7.0, dtype=lg.dtype, device=DEV)
    loss = torch.full((T,), -7.0, device=DEV)
    acc = _lib.new_step_acc(DEV)
    mask = torch.ones(T, dtype=torch.uint8, device=DEV) if mask is None else t(mask)
    _lib.grpo_distill_topk_fwd_bwd(lg, t(idx), t(lq), mask, kind, scale, dz, loss, acc, w_tok=t(w), **kw)
    torch.cuda.synchronize()
    return loss, dz, acc


def _check(lg, idx, lq, kind, scale=1.0, tau=1.0, w=None, dtype="bf16", rows=None, dz=True):
    loss, d, acc = _call(lg, idx, lq, kind, scale, temperature=tau, w=w, dz=dz)
    zh = W.logits_to_host(lg)
    lh = loss.double().cpu().numpy()
    for r in range(lg.shape[0]) if rows is None else rows:
        _check_row(lh[r], d[r].double().cpu().numpy(), zh[r], idx[r], lq[r], kind, tau,
                   scale * (1.0 if w is None else float(w[r])), dtype)
    return loss, d, acc


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V, K", [(1, 1), (2, 1), (9, 9), (40, 7), (256, 256), (1000, 64), (2047, 256), (4104, 20),
                                  (16384, 16), (30011, 37), (50257, 128)])
def test_sizes(V, K, dtype, kind):
    _check(*_inputs(3, V, K, dtype, V + K), kind, dtype=dtype, scale=0.37)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V", [151936, 163841, 400008])
def test_long_rows(V, dtype, kind):
    _check(*_inputs(3, V, 64, dtype, V), kind, dtype=dtype, scale=1.0 / 37)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("pad, offset", [(0, 1), (1, 0), (3, 5), (8, 0), (8, 8), (8, 3)])
@pytest.mark.parametrize("V", [5003, 20481])
def test_strides_and_alignments_give_the_same_bits(V, pad, offset, dtype):
    lg, idx, lq = _inputs(4, V, 33, dtype, 9, pad=pad, offset=offset)
    base = torch.zeros((4, (V + 63) // 8 * 8), dtype=DT[dtype], device=DEV)[:, :V]
    base.copy_(lg)
    for kind in KINDS:
        loss, dz, _ = _check(lg, idx, lq, kind, dtype=dtype)
        for out_pad, out_off in ((0, 0), (8, 0), (1, 1), (5, 2)):
            buf = torch.full((4 * (V + out_pad) + out_off + 8,), 9.0, dtype=DT[dtype], device=DEV)
            d = buf[out_off:out_off + 4 * (V + out_pad)].view(4, V + out_pad)
            l2, _, _ = _call(base, idx, lq, kind, 1.0, dz=d[:, :V])
            assert torch.equal(l2, loss) and torch.equal(d[:, :V], dz)
            assert torch.all(d[:, V:] == 9) and torch.all(buf[:out_off] == 9) and torch.all(buf[-8:] == 9)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("tau", [0.25, 1.0, 2.0, 8.0])
def test_temperatures_and_weights(tau, kind):
    for dtype in ("bf16", "f32"):
        lg, idx, lq = _inputs(4, 3001, 20, dtype, 4, tau=tau)
        _check(lg, idx, lq, kind, scale=0.01, tau=tau, dtype=dtype, w=np.array([1.0, 0.25, 0.0, 3.0], np.float32))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V", [700, 50257, 151936])
def test_confident_masked_and_bad_rows(V, dtype, kind):
    K = 24
    lg, idx, lq = _inputs(16, V, K, dtype, V + 5, unused=0.0)
    inf = float("inf")
    lg[0, int(idx[0, 0])] = 80.0                     # the student all but certain: a remainder far below 2^-24
    lg[1, 3] = 60.0                                  # certain of a token
    lq[2] = -30.0
    lq[2, 0] = -1e-7                                 # the teacher certain
    idx[3], lq[3] = -1, 0.0                          # no list
    keep = torch.zeros(V, dtype=torch.bool, device=DEV)
    keep[torch.from_numpy(idx[4].astype(np.int64)).to(DEV)] = True
    lg[4, ~keep] = -inf                              # nothing outside the list
    lg[5, int(idx[5, 2])] = -inf                     # a listed token the student cannot produce
    lq[6, 3] = -inf                                  # ... the teacher cannot
    lg[7, V // 2] = float("nan")
    lg[8, V - 1] = inf
    lg[9] = -inf
    idx[10, 4] = idx[10, 9]                          # a token twice
    idx[11, 1] = V
    idx[12, 1] = -5
    lq[13, 0] = float("nan")
    lg[14] = torch.where(keep, lg[14].float(), torch.finfo(DT[dtype]).min).to(DT[dtype])
    lg[14, torch.from_numpy(idx[14].astype(np.int64)).to(DEV)] = 1.0
    lq[15] -= 3.0
    loss, dz, acc = _check(lg, idx, lq, kind, dtype=dtype)
    lh = loss.double().cpu().numpy()
    res = _lib.grpo_finish_step(acc, loss, grad_bufs=[dz])
    assert res["n_tokens"] == res["n_valid"] == 16 and res["status"] == _lib.STEP_SKIPPED_NONFINITE
    assert res["n_nonfinite"] == int((~np.isfinite(lh)).sum()) and torch.all(dz == 0)


def test_masked_rows_padding_rows_and_token_index():
    T, V, K = 12, 20008, 16
    rows = T - 2
    lg, _, _ = _inputs(T, V, K, "bf16", 3)
    rng = np.random.default_rng(0)
    src = np.concatenate([rng.permutation(rows), [-1, -4]]).astype(np.int64)
    mask = (rng.random(rows) < 0.6).astype(np.uint8)
    _, idx, lq = _inputs(rows, V, K, "bf16", 8)
    w = rng.random(rows).astype(np.float32)
    zh = W.logits_to_host(lg)
    for kind in KINDS:
        loss, dz, acc = _call(lg, idx, lq, kind, 0.5, mask=mask, w=w, rows=rows,
                              tok_src=torch.from_numpy(src).to(DEV))
        for r in range(T):
            i = int(src[r])
            if i >= 0 and mask[i]:
                _check_row(loss[i].item(), dz[r].double().cpu().numpy(), zh[r], idx[i], lq[i], kind, 1.0,
                           0.5 * float(w[i]), "bf16")
            else:
                assert torch.all(dz[r] == 0) and (i < 0 or loss[i] == 0)
        res = _lib.grpo_finish_step(acc, loss, expected_N=int(mask.sum()))
        assert res["status"] == 0 and res["n_tokens"] == T and res["n_clipped"] == 0
        assert abs(res["loss"] - loss.double().sum().item() / mask.sum()) < 1e-12


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_loss_only_and_the_number_of_rows_change_no_bit(dtype):
    T, V = 330, 151936
    lg, idx, lq = _inputs(20, V, 64, dtype, 2)
    lg = lg.repeat(17, 1)[:T].contiguous()
    idx, lq = np.tile(idx, (17, 1))[:T], np.tile(lq, (17, 1))[:T]
    for kind in KINDS:
        loss, dz, _ = _call(lg, idx, lq, kind, 1.0)
        only, _, _ = _call(lg, idx, lq, kind, 1.0, dz=None)
        assert torch.equal(only, loss)
        for a, b in [(0, 1), (1, 4), (4, 30), (30, 120), (120, T)]:
            l2, d2, _ = _call(lg[a:b], idx[a:b], lq[a:b], kind, 1.0)
            assert torch.equal(l2, loss[a:b]) and torch.equal(d2, dz[a:b]), (kind, a, b)


def test_wider_lists_are_read_at_their_stride():
    lg, idx, lq = _inputs(5, 3000, 40, "bf16", 11)
    ti, tl = torch.from_numpy(idx).to(DEV), torch.from_numpy(lq).to(DEV)
    for kind in KINDS:
        a = _call(lg, ti[:, :9], tl[:, :9], kind, 1.0)
        b = _call(lg, idx[:, :9].copy(), lq[:, :9].copy(), kind, 1.0)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_captured_into_a_graph():
    lg, idx, lq = _inputs(6, 50264, 20, "bf16", 2)
    lg2, idx2, lq2 = _inputs(6, 50264, 20, "bf16", 3)
    t = lambda a: torch.from_numpy(a).to(DEV)
    for kind in KINDS:
        want = [_call(*x, kind, 1.0) for x in ((lg, idx, lq), (lg2, idx2, lq2))]
        z, i, q = lg.clone(), t(idx), t(lq)
        dz, loss, acc = torch.zeros_like(z), torch.zeros(6, device=DEV), _lib.new_step_acc(DEV)
        mask = torch.ones(6, dtype=torch.uint8, device=DEV)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            _lib.grpo_distill_topk_fwd_bwd(z, i, q, mask, kind, 1.0, dz, loss, acc)
        for x, e in zip(((lg, idx, lq), (lg2, idx2, lq2)), want):
            z.copy_(x[0]); i.copy_(t(x[1])); q.copy_(t(x[2]))
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(loss, e[0]) and torch.equal(dz, e[1])


def test_offsets_past_32_bits():
    T, V, K = 45000, 50256, 8
    z = torch.zeros((T, V), dtype=torch.bfloat16, device=DEV)
    lg, idx, lq = _inputs(3, V, K, "bf16", 6)
    z[-3:] = lg
    mask = torch.zeros(T, dtype=torch.uint8, device=DEV)
    mask[-3:] = 1
    ti = torch.full((T, K), -1, dtype=torch.int32, device=DEV)
    tl = torch.zeros((T, K), device=DEV)
    ti[-3:], tl[-3:] = torch.from_numpy(idx).to(DEV), torch.from_numpy(lq).to(DEV)
    loss, dz, _ = _call(z, ti, tl, _lib.DISTILL_FORWARD_TAIL, 1.0, mask=mask)
    zh = W.logits_to_host(lg)
    for r in range(3):
        _check_row(loss[T - 3 + r].item(), dz[T - 3 + r].double().cpu().numpy(), zh[r], idx[r], lq[r], 1, 1.0, 1.0,
                   "bf16")
    assert not dz[:-3].any()


def test_a_teachers_scores_train_a_student():
    # the run as it is used: the teacher's rows scored, the student's loss and gradient, the step
    # finish, one gradient step on the logits; every loss must be the oracle's before and after
    T, V, K = 24, 20000, 32
    g = torch.Generator(device=DEV).manual_seed(1)
    teacher = torch.randn((T, V), generator=g, device=DEV) * 3
    student = (0.8 * teacher + torch.randn((T, V), generator=g, device=DEV)).contiguous()
    top_idx = torch.empty((T, K), dtype=torch.int32, device=DEV)
    top_logp = torch.empty((T, K), device=DEV)
    _lib.grpo_token_topk_logprobs(teacher, K, top_idx=top_idx, top_logp=top_logp)
    idx, lq = top_idx.cpu().numpy(), top_logp.cpu().numpy()
    for kind in KINDS:
        z = student.clone()
        for _ in range(2):
            loss, dz, acc = _check(z, idx, lq, kind, scale=1.0 / T, dtype="f32")
            res = _lib.grpo_finish_step(acc, loss, expected_N=T)
            assert res["status"] == 0 and abs(res["loss"] - loss.double().mean().item()) < 1e-9
            z -= 20.0 * dz


def test_binding_refuses_what_the_kernel_cannot_take():
    lg, idx, lq = _inputs(2, 64, 8, "f32", 0)
    t = lambda a: torch.from_numpy(a).to(DEV)
    with pytest.raises(_lib.GrpoError):
        _call(lg, idx, lq, 3, 1.0)
    with pytest.raises(_lib.GrpoError):
        _call(lg, idx, lq, 0, 1.0, temperature=-1.0)
    with pytest.raises(_lib.GrpoError):
        _call(lg, idx, lq, 0, 1.0, dz=lg)  # in place
    with pytest.raises(ValueError):
        _call(lg, t(idx).long(), lq, 0, 1.0)
    with pytest.raises(ValueError):
        _call(lg, idx[:1], lq[:1], 0, 1.0)
    with pytest.raises(ValueError):
        _call(lg, idx, lq[:, :4].copy(), 0, 1.0)
    with pytest.raises(ValueError):
        _call(lg, idx, lq, 0, 1.0, dz=torch.zeros((2, 64), dtype=torch.bfloat16, device=DEV))

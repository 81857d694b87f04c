"""GPU scoring and distillation where z log2(e)/tau is so large that its float32 rounding is many units of
the exponent: finite masks over whole tiles of a row, rows of huge logits, temperatures next to 0. Against
the oracles with the bars of the single-call tests; the log-prob of a far token carries five roundings of
2^-24 of its value (log2(e)/tau, the difference, the scale, ln2 and their products). Just below the
point where the scale changes, t of the row's largest logit may be 64: half a step of that (2^-18) in log2 S
and in q/S, times ln2, are 5.3e-6 of an entropy or a log-prob next to 0."""
import numpy as np
import pytest
import torch

from oracle import distill as OD
from oracle import loss as OL
from oracle import score as OS
from rl_post_token_gb300 import _lib
from rl_post_token_gb300 import workloads as W
from tests import test_gpu_distill as D
from tests import test_gpu_distill_remainder as R
from tests import test_gpu_score as S

pytestmark = pytest.mark.gpu
DEV = "cuda"
MASKS = [-1e4, -1e9, -2.1e9, -3e9, -1e10, -3.3e12, -1e20, -1.7e30, -1e30, -1.5e38, -3e38]
FORMS = [(11, 9000), (11, 40001), (480, 36008), (11, 151936), (11, 800008)]


@pytest.fixture(scope="module", autouse=True)
def _built(grpo_lib):
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return grpo_lib


def _far_top(o, r, z, tau, n):
    """The log-probs of a row's n best tokens, bar by bar."""
    logp, H, idx, top = OS.score_row(z, None, n, tau)
    got = o["top_logp"][r, :n].double().cpu().numpy()
    assert np.array_equal(o["top_idx"][r, :n].cpu().numpy(), idx)
    fin = np.isfinite(top) & (np.abs(top) < 3e38)
    assert np.all(np.abs(got - top)[fin] <= 1e-5 + 5 * 2.0 ** -24 * np.abs(top)[fin]), (r, got, top)
    assert np.all(got[~fin] < -3e38)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T, V", FORMS)
def test_finite_masks_over_whole_tiles(T, V, dtype):
    z, idx, lq = D._inputs(T, V, 12, dtype, V, unused=0.2)
    for r in range(T):
        m = MASKS[r % len(MASKS)]
        a, b = [(0, V // 2), (V // 3, V), (V // 4, 3 * V // 4)][r % 3]
        keep = z[r].clone()
        z[r, a:b] = max(m * (1.0 + 0.05 * (r % 7)), torch.finfo(D.DT[dtype]).min)
        at = torch.from_numpy(idx[r][idx[r] >= 0].astype(np.int64)).to(DEV)
        z[r, at] = keep[at]
    rows = sorted(set(range(11)) | {T - 1})
    S._check(z, 12, rows=rows)
    S._check(z, 3, tau=0.01, rows=rows)
    for kind in D.KINDS:
        _, dz, acc = D._check(z, idx, lq, kind, dtype=dtype, rows=rows)
        assert torch.isfinite(dz).all()
        assert int(acc[16:24].view(torch.int64)[0]) == 0  # no token counts as non-finite


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T, V", FORMS)
def test_a_student_whose_unlisted_tokens_are_all_masked(T, V, dtype):
    K = 8
    rng = np.random.default_rng(V)
    z = torch.empty((T, V), dtype=D.DT[dtype], device=DEV)
    idx = np.stack([rng.permutation(V)[:K] for _ in range(T)]).astype(np.int32)
    lq = np.log(0.9 * rng.dirichlet(np.ones(K + 1), T)[:, :K] + 1e-4).astype(np.float32)
    for r in range(T):
        z[r] = MASKS[r % 10]
        z[r, torch.from_numpy(idx[r].astype(np.int64)).to(DEV)] = torch.from_numpy(rng.standard_normal(K)).to(DEV).to(z.dtype)
    loss, dz, acc = D._call(z, idx, lq, _lib.DISTILL_FORWARD_TAIL, 1.0)
    zh = W.logits_to_host(z[:11])
    for r in list(range(10)):
        R._check_row(loss[r].item(), dz[r].double().cpu().numpy(), zh[r], idx[r], lq[r], 1.0, 1.0, dtype)
    assert torch.isfinite(loss[:10]).all()
    for kind in (_lib.DISTILL_FORWARD_TOPK, _lib.DISTILL_REVERSE_TAIL):
        D._check(z, idx, lq, kind, dtype=dtype, rows=range(10))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T, V", [(10, 9000), (10, 40001), (480, 36008)])
def test_rows_of_huge_logits(T, V, dtype):
    # the largest of them, tied or not, has all the mass; its neighbours in the type are next
    g = torch.Generator(device=DEV).manual_seed(V)
    base = torch.tensor([1e9, 3e9, 1e10, 2.0 ** 33, 1e20, 1.7e30, 1e38, -1e9, -1e10, -1.3e30], device=DEV)
    at = torch.arange(T, device=DEV) % 10
    u = torch.randint(0, 6, (T, V), generator=g, device=DEV).float()
    eps = 2.0 ** -22 if dtype == "f32" else 2.0 ** -6
    z = (base[at][:, None] * (1.0 - eps * u)).to(D.DT[dtype])
    zh = W.logits_to_host(z[:10])
    o = S._call(z, 6, torch.zeros(T, dtype=torch.int32, device=DEV))
    for r in range(10):
        logp, H, _, _ = OS.score_row(zh[r], 0, 6)
        assert abs(o["entropy_tok"][r].item() - H) <= 2e-5 * max(1.0, H)
        assert abs(o["logp_tok"][r].item() - logp) <= 1e-5 + 5 * 2.0 ** -24 * abs(logp)
        _far_top(o, r, zh[r], 1.0, 6)
    idx = np.stack([np.random.default_rng(r).permutation(V)[:5] for r in range(T)]).astype(np.int32)
    lq = np.full((T, 5), np.log(0.15), np.float32)
    for kind in D.KINDS:
        loss, dz, _ = D._call(z, idx, lq, kind, 1.0)
        assert torch.isfinite(dz).all()
        for r in range(10):
            ref, dx, parts = OD.row_loss(zh[r], idx[r], lq[r], kind)
            zr = OL.as_f64(np.asarray(zh[r]))
            with np.errstate(invalid="ignore", divide="ignore"):
                bl, bz = D._bars(zr, idx[r], lq[r], kind, 1.0, 1.0, parts, ref)
            # listed tokens whose share underflows in 64 bits, too, have log-probs of up to 1e36: q within
            # 21 U, five roundings of the log-prob, the difference, the product, 13 U of the sum
            if kind != _lib.DISTILL_REVERSE_TAIL:
                bl += 41 * D.U * float(np.sum(parts["q"] * np.abs(parts["lp"][idx[r]])))
            assert abs(loss[r].item() - ref) <= bl, (kind, r, loss[r].item(), ref, bl)
            err = np.abs(dz[r].double().cpu().numpy() - dx)
            assert np.all(err <= bz + (D.HALF[dtype] + 5 * D.U) * (np.abs(dx) + bz) + 2.0 ** -126), (kind, r)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T, V", [(6, 9000), (6, 40001), (480, 36008)])
@pytest.mark.parametrize("tau", [1e-6, 1e-8, 1e-9, 1e-12, 1e-20, 1e-30])
def test_temperatures_next_to_zero(T, V, tau, dtype):
    z = S._logits(T, V, dtype, 3.0, 4)
    z[2, 5] = z[2, V - 9] = z[2].max()
    o = S._call(z, 4, z.float().argmax(1).int(), temperature=tau)
    zh = W.logits_to_host(z[:6])
    for r in range(6):
        logp, H, _, _ = OS.score_row(zh[r], int(zh[r].argmax()) if dtype == "f32" else None, 4, tau)
        ties = (z[r] == z[r].max()).sum().item()
        assert abs(o["logp_tok"][r].item() + np.log(ties)) <= 1e-5 and abs(o["entropy_tok"][r].item() - H) <= 1e-5
        _far_top(o, r, zh[r], tau, 4)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T, V", [(8, 900), (8, 40001), (330, 36008)])
@pytest.mark.parametrize("tau, top", [(1e-6, 29952.0), (1e-6, 600.0), (1e-3, 1e7), (1.0, 1e10), (1e-8, 40.0)])
def test_a_listed_token_far_above_a_row_of_ordinary_ones(T, V, tau, top, dtype):
    # the shifts of the row and of the tokens outside the list are under different scales
    z, idx, lq = D._inputs(T, V, 7, dtype, V, unused=0.0)
    for r in range(T):
        z[r, int(idx[r, r % 7])] = top
    lq -= 0.1
    loss, dz, acc = D._call(z, idx, lq, _lib.DISTILL_FORWARD_TAIL, 0.5, temperature=tau)
    assert int(acc[16:24].view(torch.int64)[0]) == 0
    zh = W.logits_to_host(z[:8])
    for r in range(8):
        R._check_row(loss[r].item(), dz[r].double().cpu().numpy(), zh[r], idx[r], lq[r], tau, 0.5, dtype)

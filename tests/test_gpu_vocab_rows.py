"""GPU tests of the scoring and distillation calls as a program meets them: long calls whose rows are
masked, padded and shuffled, rows full of ties, masked vocabularies, callers on several streams and
host threads at once, graphs replayed side by side, and the LM-head form with few tokens, whose d_h is
summed in several runs. Values against the float64 oracles with the bars of the single-call tests;
everything else bit for bit."""
import threading

import numpy as np
import pytest
import torch

from rl_post_token_gb300 import _lib
from rl_post_token_gb300 import workloads as W
from tests import test_gpu_distill as D
from tests import test_gpu_lmhead_distill as L
from tests import test_gpu_score as S

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _built(grpo_lib):
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return grpo_lib


def _same(a, b):
    return torch.equal(a.view(torch.int16 if a.element_size() == 2 else torch.int32),
                       b.view(torch.int16 if b.element_size() == 2 else torch.int32))


@pytest.mark.parametrize("kind", D.KINDS)
@pytest.mark.parametrize("V, dtype, K, pad, out_pad", [(50257, "bf16", 37, 0, 0), (50257, "bf16", 256, 0, 6),
                                                       (40000, "bf16", 64, 8, 0), (151936, "bf16", 200, 0, 0),
                                                       (60001, "f32", 70, 0, 0), (60001, "f32", 70, 0, 2),
                                                       (4104, "bf16", 33, 3, 3), (200003, "f32", 12, 0, 0),
                                                       # a row takes the whole ring of slots, or all but one or two
                                                       (106400, "bf16", 32, 0, 0), (108500, "bf16", 32, 0, 0),
                                                       (110501, "bf16", 32, 0, 0)])
def test_distillation_of_many_rows_is_that_of_each(V, dtype, K, pad, out_pad, kind):
    # persistent clusters walk over hundreds of rows, masked and padding rows among them
    T = 420
    lg, idx, lq = D._inputs(30, V, K, dtype, 5, pad=pad)
    rows = torch.arange(T, device=DEV) % 30
    z = torch.zeros((T, V + pad), dtype=D.DT[dtype], device=DEV)[:, :V]
    z.copy_(lg[rows])
    idx, lq = idx[rows.cpu().numpy()], lq[rows.cpu().numpy()]
    rng = np.random.default_rng(K)
    mask = (rng.random(T) < 0.7).astype(np.uint8)
    src = rng.permutation(T)
    src[rng.choice(T, 11, replace=False)] = -2
    ti, tl = torch.from_numpy(idx).to(DEV), torch.from_numpy(lq).to(DEV)
    out = lambda n: torch.full((n, V + out_pad), 7.0, dtype=D.DT[dtype], device=DEV)[:, :V]
    want = out(30)
    wl, _, _ = D._call(z[:30], idx[:30], lq[:30], kind, 1.0, dz=want)
    D._check(z[:30], idx[:30], lq[:30], kind, dtype=dtype, rows=(0, 17))
    # row i of the call is token src[i], whose list is that of the row's logits
    put = src.copy()
    at = torch.from_numpy(put).to(DEV)
    keep = put >= 0
    ti2, tl2 = ti.clone(), tl.clone()
    ti2[at[at >= 0]] = ti[torch.from_numpy(np.nonzero(keep)[0]).to(DEV)]
    tl2[at[at >= 0]] = tl[torch.from_numpy(np.nonzero(keep)[0]).to(DEV)]
    dz = out(T)
    loss, _, acc = D._call(z, ti2, tl2, kind, 1.0, mask=mask, dz=dz, tok_src=at, rows=T)
    for i in range(T):
        if put[i] >= 0 and mask[put[i]]:
            assert _same(dz[i], want[i % 30]) and _same(loss[put[i]], wl[i % 30]), i
        else:
            assert not dz[i].any() and (put[i] < 0 or loss[put[i]] == 0), i
    only, _, _ = D._call(z, ti2, tl2, kind, 1.0, mask=mask, dz=None, tok_src=at, rows=T)
    assert _same(only, loss)
    live = int((mask[put[keep]] != 0).sum())
    res = _lib.grpo_finish_step(acc, loss, expected_N=live)
    assert res["n_tokens"] == T and res["n_valid"] == live and res["status"] == 0
    if out_pad:
        whole = torch.as_strided(dz, (T, V + out_pad), (V + out_pad, 1))
        assert torch.all(whole[:, V:] == 7)


@pytest.mark.parametrize("T", [2, 470])
@pytest.mark.parametrize("V, dtype", [(50257, "bf16"), (36001, "f32"), (9000, "bf16")])
def test_scores_of_rows_full_of_ties(V, dtype, T):
    # a few hundred equal logits around the K-th place: more candidates than K, ranked by index
    z = S._logits(T, V, dtype, 1.0, 3)
    for i, step in enumerate((0.5, 0.25, 1.0 / 16)):
        z[i::3] = (z[i::3].float() / step).round().mul(step).to(z.dtype)
    z[T - 1, :V // 2] = 4.0  # more ties than the candidate buffer
    for K in (31, 256):
        S._check(z, K, rows=(0, 1, T - 1) if T > 2 else (0, 1))


@pytest.mark.parametrize("T", [3, 470])
@pytest.mark.parametrize("V, dtype", [(50257, "bf16"), (36000, "f32")])
def test_scores_of_masked_vocabularies(V, dtype, T):
    z = S._logits(T, V, dtype, 3.0, 7)
    g = torch.Generator(device=DEV).manual_seed(1)
    cut = torch.rand((T, V), device=DEV, generator=g)
    z.masked_fill_(cut < 0.1, float("-inf"))
    z[1].masked_fill_(cut[1] > 0.5, torch.finfo(z.dtype).min)  # no mass, like -inf
    z[2, 4000:] = float("-inf")                                # tiles without any
    S._check(z, 20, rows=(0, 1, 2))
    for tau in (0.01, 50.0):
        S._check(z, 5, tau=tau, rows=(0, 1, 2))


def _work(seed):
    """Inputs of the three calls, and a function that runs them into new outputs."""
    z = S._logits(470, 50257, "bf16", 3.0, seed)
    lg, idx, lq = D._inputs(200, 50257, 40, "bf16", seed + 1)
    ti, tl = torch.from_numpy(idx).to(DEV), torch.from_numpy(lq).to(DEV)
    mask = torch.ones(200, dtype=torch.uint8, device=DEV)
    h, Wt, li, ll, lm = L._inputs(40, 20000, 256, 12, seed + 2)
    li, ll, lm = L._t(li), L._t(ll), L._t(lm)
    y = torch.arange(470, dtype=torch.int32, device=DEV)
    torch.cuda.synchronize()

    def outputs():
        return dict(logp=torch.zeros(470, device=DEV), ent=torch.zeros(470, device=DEV),
                    top=torch.zeros((470, 30), dtype=torch.int32, device=DEV), lp=torch.zeros((470, 30), device=DEV),
                    dz=torch.zeros_like(lg), loss=torch.zeros(200, device=DEV), acc=_lib.new_step_acc(DEV),
                    d_h=torch.zeros((40, 256), device=DEV), dW=torch.zeros((20000, 256), device=DEV),
                    lloss=torch.zeros(40, device=DEV), lacc=_lib.new_step_acc(DEV),
                    ws=torch.empty(_lib.grpo_lmhead_distill_workspace_size(40, 20000, 256, 12), dtype=torch.uint8,
                                   device=DEV))

    def run(o):
        _lib.grpo_token_topk_logprobs(z, 30, target=y, logp_tok=o["logp"], entropy_tok=o["ent"], top_idx=o["top"],
                                      top_logp=o["lp"])
        _lib.grpo_distill_topk_fwd_bwd(lg, ti, tl, mask, _lib.DISTILL_REVERSE_TAIL, 1.0, o["dz"], o["loss"], o["acc"])
        _lib.grpo_lmhead_distill_topk_fwd_bwd(h, Wt, li, ll, lm, 1.0, o["d_h"], o["dW"], o["lloss"], o["lacc"], o["ws"])

    return outputs, run


def _equal(a, b):
    return all(torch.equal(a[k], b[k]) for k in a if k not in ("acc", "lacc", "ws"))


def test_host_threads_on_their_own_streams():
    jobs = [_work(100 * i) for i in range(4)]
    want = []
    for outputs, run in jobs:
        o = outputs()
        run(o)
        torch.cuda.synchronize()
        want.append(o)
    outs = [outputs() for outputs, _ in jobs]
    torch.cuda.synchronize()
    errors = []

    def body(i):
        try:
            st = torch.cuda.Stream()
            with torch.cuda.stream(st):
                for _ in range(5):
                    jobs[i][1](outs[i])
            st.synchronize()
        except Exception as e:  # noqa: BLE001 (reported by the test)
            errors.append(e)

    th = [threading.Thread(target=body, args=(i,)) for i in range(4)]
    for t in th:
        t.start()
    for t in th:
        t.join()
    assert not errors, errors
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert _equal(o, w)


def test_graphs_replayed_side_by_side():
    jobs = [_work(7), _work(8)]
    graphs, outs, want = [], [], []
    for outputs, run in jobs:
        w = outputs()
        run(w)
        torch.cuda.synchronize()
        want.append(w)
        o = outputs()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            run(o)
        graphs.append(g)
        outs.append(o)
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(3):
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
        jobs[0][1](jobs[0][0]())  # and a call outside them
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert _equal(o, w)


# 9 runs of 16 K blocks; one run short of them in the last chunk; one CTA pair's tile; live tokens in
# fewer row tiles than allocated
@pytest.mark.parametrize("T, V, H, K, masked", [(70, 9000, 128, 20, 0.2), (33, 66000, 64, 8, 0.2),
                                                (1, 20000, 256, 5, 0.0), (600, 12000, 320, 16, 0.9)])
def test_lmhead_few_tokens(T, V, H, K, masked):
    a = L._inputs(T, V, H, K, T, masked=masked)
    out = L._call(*a, 0.5)
    L._check(a, 0.5, out)
    for kw in ({}, {"skip_masked": True}):
        b = L._call(*a, 0.5, **kw)
        assert all(torch.equal(x, y) for x, y in zip(out[:3], b[:3]))
    # what the workspace held before does not matter
    ws = torch.full((_lib.grpo_lmhead_distill_workspace_size(T, V, H, K),), 255, dtype=torch.uint8, device=DEV)
    b = L._call(*a, 0.5, ws=ws)
    assert all(torch.equal(x, y) for x, y in zip(out[:3], b[:3]))
    only_h = torch.full((T, H), 7.0, device=DEV)
    loss, acc = torch.zeros(T, device=DEV), _lib.new_step_acc(DEV)
    _lib.grpo_lmhead_distill_topk_fwd_bwd(a[0], a[1], L._t(a[2]), L._t(a[3]), L._t(a[4]), 0.5, only_h, None, loss, acc, ws)
    torch.cuda.synchronize()
    assert torch.equal(only_h, out[1])

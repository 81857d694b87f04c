"""GPU parity of the token scoring call against the float64 oracle.

Tolerances. With t = (z - max) log2(e)/tau the kernel forms t by one fused multiply-add (relative
error 2^-24, and 2^-24 more through the rounded log2(e)/tau), 2^t within 2^-22, and sums up to 64
exponentials of a lane in 4 chains (16 additions), 2 to join them, 5 over the lanes and at most 16
joins over the tiles: 39 roundings of 2^-24. With E the expectation over the row's distribution
  d(log S)  <= 2^-22 + 39 2^-24 + 2^-23 ln2 E|t| + 2^-24 log S    (the last: log2's own rounding)
  d(log p)  <= d(log S) + 2^-23 |z_y - max|/tau + 2^-23 |log p|
  d(H)      <= d(log S) + ln2 (E|t| (2^-22 + 39 2^-24 + 2^-23) + 2^-23 E t^2) + 2^-23 (log S + E|t|)
where every rounding counts with its full bound. Indices must be equal."""
import numpy as np
import pytest
import torch

from oracle import loss as OL
from oracle import score as OS
from rl_post_token_gb300 import _lib
from rl_post_token_gb300 import workloads as W

pytestmark = pytest.mark.gpu
DEV = "cuda"
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _built(grpo_lib):
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return grpo_lib


def _tols(z, y, tau):
    """(log S bar, E|t|, E t^2, max) of a float64 row with a distribution."""
    m = np.max(z)
    d = (z - m) / tau
    p = np.exp(d)
    S = p.sum()
    p /= S
    with np.errstate(invalid="ignore"):
        t = np.where(p > 0, d / np.log(2), 0.0)
    et, et2 = float((p * -t).sum()), float((p * t * t).sum())
    ls = 2.0 ** -22 + 39 * 2.0 ** -24 + 2.0 ** -23 * np.log(2) * et + 2.0 ** -24 * np.log(S)
    h = ls + np.log(2) * (et * (2.0 ** -22 + 39 * 2.0 ** -24 + 2.0 ** -23) + 2.0 ** -23 * et2) \
        + 2.0 ** -23 * (np.log(S) + et)
    return ls, h, m


def _call(logits, K, target=None, **kw):
    T = kw.pop("rows", logits.shape[0])
    o = dict(logp_tok=torch.full((T,), -7.0, device=DEV), entropy_tok=torch.full((T,), -7.0, device=DEV),
             top_idx=torch.full((T, max(K, 1)), -7, dtype=torch.int32, device=DEV),
             top_logp=torch.full((T, max(K, 1)), -7.0, device=DEV))
    if target is None:
        o["logp_tok"] = None
    _lib.grpo_token_topk_logprobs(logits, K, target=target, **o, **kw)
    torch.cuda.synchronize()
    return o


def _check_row(o, r, z, y, K, tau):
    logp, H, idx, top = OS.score_row(z, y, K, tau)
    got = o["top_idx"][r, :K].cpu().numpy()
    assert np.array_equal(got, idx), (r, got[:10], idx[:10])
    glp = o["logp_tok"][r].item() if o["logp_tok"] is not None else None
    gh = o["entropy_tok"][r].item()
    gt = o["top_logp"][r, :K].double().cpu().numpy()
    z = OL.as_f64(np.asarray(z))
    if np.isnan(H):
        assert np.isnan(gh) and np.isnan(gt).all() and (glp is None or np.isnan(glp))
        return
    ls, hb, m = _tols(z, y, tau)

    def bar(zz, ref):
        return ls + 2.0 ** -23 * (abs(zz - m) / tau + abs(ref))
    if glp is not None:
        if np.isnan(logp):
            assert np.isnan(glp)
        elif np.isinf(logp):
            assert glp == logp
        else:
            assert abs(glp - logp) <= bar(z[y], logp), (r, glp, logp)
    assert abs(gh - H) <= hb, (r, gh, H, hb)
    for k in range(K):
        if np.isinf(top[k]):
            assert gt[k] == top[k]
        else:
            assert abs(gt[k] - top[k]) <= bar(z[idx[k]], top[k]), (r, k, gt[k], top[k])


def _logits(T, V, dtype, std, seed, pad=0, offset=0):
    """[T, V] rows with `pad` elements between them, starting `offset` elements into a buffer."""
    rng = np.random.default_rng(seed)
    x = torch.from_numpy((rng.standard_normal((T, V)) * std).astype(np.float32)).to(DT[dtype])
    buf = torch.full((T * (V + pad) + offset + 8,), 50.0, dtype=DT[dtype], device=DEV)  # outside: larger than any logit
    v = buf[offset:offset + T * (V + pad)].view(T, V + pad)[:, :V]
    v.copy_(x)
    return v


def _check(z, K, tau=1.0, target=None, rows=None, **kw):
    T, V = z.shape
    rng = np.random.default_rng(V + K)
    y = rng.integers(0, V, T).astype(np.int32) if target is None else target
    o = _call(z, K, torch.from_numpy(y).to(DEV), temperature=tau, **kw)
    zh = W.logits_to_host(z)
    for r in range(T) if rows is None else rows:
        _check_row(o, r, zh[r], int(y[r]), K, tau)
    return o


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V, K", [(1, 1), (2, 2), (7, 3), (8, 8), (31, 20), (256, 256), (1000, 64), (2047, 256),
                                  (2048, 1), (4104, 20), (8191, 128), (20481, 37), (50257, 37)])
def test_sizes(V, K, dtype):
    _check(_logits(3, V, dtype, 3.0, V), K)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V", [151936, 163839, 163841, 400003])
def test_long_rows(V, dtype):
    _check(_logits(2, V, dtype, 3.0, V), 64)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("pad, offset", [(0, 1), (1, 0), (3, 5), (8, 0), (8, 8), (8, 3)])
def test_strides_and_alignments_give_the_same_bits(pad, offset, dtype):
    # rows that start anywhere: right, and the bits of the packed, aligned rows
    V = 5003 if offset != 8 else 5000
    z = _logits(4, V, dtype, 3.0, 9, pad, offset)
    o = _check(z, 33)
    base = torch.zeros((4, (V + 63) // 8 * 8), dtype=DT[dtype], device=DEV)[:, :V]
    base.copy_(z)
    ref = _check(base, 33)
    for k in o:
        assert torch.equal(o[k], ref[k]), k


@pytest.mark.parametrize("tau", [1e-3, 0.3, 1.0, 2.0, 100.0])
def test_temperatures(tau):
    _check(_logits(3, 3001, "bf16", 3.0, 4), 20, tau=tau)
    _check(_logits(3, 3001, "f32", 3.0, 5), 20, tau=tau)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V", [600, 30011, 151936])
def test_ties_masks_and_bad_rows(V, dtype):
    K = 40
    z = _logits(14, V, dtype, 3.0, V + 1)
    z[0] = 1.25                                       # every logit equal
    z[1] = torch.arange(V, device=DEV).float() / V    # ascending, with ties in bf16
    z[2] = -torch.arange(V, device=DEV).float() / V   # descending
    z[3] = torch.randint(0, 3, (V,), device=DEV).float()  # three values
    z[4] = float("-inf")
    z[4, 17] = 0.5
    z[4, 3] = 0.5
    z[4, V - 1] = -2.0                                # three tokens allowed, K asked
    z[5] = torch.finfo(DT[dtype]).min
    z[5, 5:90] = torch.arange(85, device=DEV).float()  # the type's lowest value as a mask
    z[6] = float("-inf")                              # nothing allowed
    z[7, V // 2] = float("nan")
    z[8, V - 1] = float("inf")
    z[9, 11] = 3e4                                    # one far outlier
    z[10] = 0.0
    z[10, ::2] = -0.0                                 # -0 and +0 tie
    z[11, : V // 2] = float("-inf")
    z[12, 0] = float("nan")
    z[12, 1:] = float("-inf")
    z[13] = -1e4 + z[13]
    _check(z, K)
    _check(z, 0)


def test_masked_rows_padding_rows_and_token_index():
    T, V, K = 12, 3000, 16
    z = _logits(T, V, "bf16", 3.0, 3)
    rng = np.random.default_rng(0)
    rows = T - 2
    src = np.concatenate([rng.permutation(rows), [-1, -4]]).astype(np.int64)
    mask = (rng.random(rows) < 0.7).astype(np.uint8)
    y = rng.integers(0, V, rows).astype(np.int32)
    t = lambda a: torch.from_numpy(a).to(DEV)
    o = _call(z, K, t(y), mask=t(mask), tok_src=t(src), rows=rows)
    zh = W.logits_to_host(z)
    for r in range(rows):
        i = int(src[r])
        if mask[i]:
            _check_row(o, i, zh[r], int(y[i]), K, 1.0)
        else:
            assert o["logp_tok"][i] == 0 and o["entropy_tok"][i] == 0
            assert torch.all(o["top_idx"][i] == -1) and torch.all(o["top_logp"][i] == float("-inf"))


def test_targets_outside_the_vocabulary_and_left_out_outputs():
    z = _logits(4, 500, "f32", 2.0, 8)
    y = np.array([-1, 500, 0, 499], np.int32)
    _check(z, 5, target=y)
    H = torch.zeros(4, device=DEV)
    _lib.grpo_token_topk_logprobs(z, 0, entropy_tok=H)
    idx = torch.zeros((4, 9), dtype=torch.int32, device=DEV)
    _lib.grpo_token_topk_logprobs(z, 5, top_idx=idx)  # a wider output: the rest is left alone
    ref = _check(z, 5, target=y)
    assert torch.equal(H, ref["entropy_tok"]) and torch.equal(idx[:, :5], ref["top_idx"])
    assert torch.all(idx[:, 5:] == 0)
    _lib.grpo_token_topk_logprobs(z[:0], 5, top_idx=idx[:0])


@pytest.mark.parametrize("V, dtype, pad", [(151936, "bf16", 0), (50257, "bf16", 0), (35001, "f32", 0),
                                           (35000, "f32", 0), (40000, "bf16", 8), (163840, "bf16", 3)])
@pytest.mark.parametrize("K", [0, 1, 20, 256])
def test_results_do_not_depend_on_how_many_rows_share_the_call(V, dtype, pad, K):
    # a few rows, or a few dozen, go to other kernels than many rows: the bits are the same, with
    # masked rows, padding rows and a shuffled order
    T = 460
    z = _logits(40, V, dtype, 3.0, 21, pad).repeat(12, 1)[:T]
    if pad:
        buf = torch.zeros((T, V + pad), dtype=DT[dtype], device=DEV)
        buf[:, :V] = z
        z = buf[:, :V]
    z[7, 3:400] = float("-inf")
    z[11, 5] = float("nan")
    y = torch.arange(T, dtype=torch.int32, device=DEV) * 70
    rng = np.random.default_rng(K)
    mask = torch.from_numpy((rng.random(T) < 0.8).astype(np.uint8)).to(DEV)
    src = rng.permutation(T)
    src[rng.choice(T, 9, replace=False)] = -3
    src = torch.from_numpy(src).to(DEV)
    same = lambda a, b: torch.equal(a.view(torch.int32), b.view(torch.int32))
    whole = _call(z, K, y)
    for a, b in [(0, 1), (1, 3), (3, 12), (12, 40), (40, 140), (140, 460)]:
        part = _call(z[a:b], K, y[a:b])
        for k in part:
            assert same(part[k], whole[k][a:b]), (k, a, b)
    zh = W.logits_to_host(z[:2])
    for r in range(2):
        _check_row(whole, r, zh[r], int(y[r]), K, 1.0)
    full = _call(z, K, y, mask=mask, tok_src=src)
    at = src.clamp(min=0)
    parts = _call(z[:1], K, y, mask=mask, tok_src=src[:1], rows=T)
    for a in range(1, T, 50):
        o = _call(z[a:a + 50], K, y, mask=mask, tok_src=src[a:a + 50], rows=T)
        for k in o:
            rows = src[a:a + 50][src[a:a + 50] >= 0]
            parts[k][rows] = o[k][rows]
    for k in full:
        assert same(full[k][at], parts[k][at]), k


def test_captured_into_a_graph_and_on_another_stream():
    z = _logits(5, 50257, "bf16", 3.0, 2)
    y = torch.arange(5, dtype=torch.int32, device=DEV)
    ref = _call(z, 20, y)
    o = {k: torch.zeros_like(v) for k, v in ref.items()}
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        _lib.grpo_token_topk_logprobs(z, 20, target=y, **o)
    z2 = _logits(5, 50257, "bf16", 2.0, 77)
    want = _call(z2, 20, y)
    for src, exp in ((z, ref), (z2, want)):
        z.copy_(src)
        g.replay()
        torch.cuda.synchronize()
        for k in o:
            assert torch.equal(o[k], exp[k]), k


def test_offsets_past_32_bits():
    # 70,000 x 50,257 bf16: the last rows start 3.5e9 elements into the buffer
    T, V = 70000, 50257
    z = torch.zeros((T, V), dtype=torch.bfloat16, device=DEV)
    z[-3:] = _logits(3, V, "bf16", 3.0, 6)
    mask = torch.zeros(T, dtype=torch.uint8, device=DEV)
    mask[-3:] = 1
    y = torch.full((T,), 7, dtype=torch.int32, device=DEV)
    o = _call(z, 4, y, mask=mask)
    zh = W.logits_to_host(z[-3:])
    for r in range(3):
        _check_row({k: v[-3:] for k, v in o.items()}, r, zh[r], 7, 4, 1.0)


def test_binding_refuses_what_the_kernel_cannot_take():
    z = torch.zeros((2, 64), device=DEV)
    i = torch.zeros((2, 8), dtype=torch.int32, device=DEV)
    for kw in (dict(K=65), dict(K=257), dict(K=-1), dict(K=4, temperature=0.0), dict(K=4, temperature=float("nan"))):
        with pytest.raises((_lib.GrpoError, ValueError)):
            _lib.grpo_token_topk_logprobs(z, kw.pop("K"), top_idx=torch.zeros((2, 300), dtype=torch.int32, device=DEV), **kw)
    with pytest.raises(ValueError):
        _lib.grpo_token_topk_logprobs(z, 8, top_idx=i.long())
    with pytest.raises(ValueError):
        _lib.grpo_token_topk_logprobs(z, 8, top_idx=i.cpu())
    with pytest.raises(ValueError):
        _lib.grpo_token_topk_logprobs(z, 8, top_idx=i[:1])
    with pytest.raises(ValueError):
        _lib.grpo_token_topk_logprobs(z.t(), 2, top_idx=i)

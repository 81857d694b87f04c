"""GPU parity of the gradient norm and the clip against float64: sizes from none to past a chunk, odd
alignments, mixed types, both tables of tensors, the ends of float32's range, non-finite gradients, the
step's status and the deferred scale.

Tolerances: a sum of squares is off by at most 20 roundings of 2^-24 (a thread's chain of 16 squares and a
tree), float64 beyond: 2^-19 of it, so 2^-20 of the norm, and its own rounding 2^-24; the factor the same
with two roundings; an output the factor's and half a step of its type (2^-8 bf16, 2^-24 float32)."""
import math

import numpy as np
import pytest
import torch

from oracle import ce as OC
from rl_post_token_gb300 import _lib

pytestmark = pytest.mark.gpu
DEV = "cuda"
F32, BF16 = torch.float32, torch.bfloat16
NORM_REL, COEF_REL = 2.0 ** -20 + 2.0 ** -24, 2.0 ** -20 + 2.0 ** -23


@pytest.fixture(scope="module", autouse=True)
def _built(grpo_lib):
    assert torch.cuda.is_available()
    return grpo_lib


def _views(sizes, dtype, gaps, seed, scale=1.0):
    """Tensors of these sizes in one buffer, gaps[i % len] elements before each: (buffer, views)."""
    at, places = 0, []
    for i, n in enumerate(sizes):
        at += gaps[i % len(gaps)]
        places.append((at, n))
        at += n
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    buf = (torch.randn(at + 9, generator=g, device=DEV) * scale).to(dtype)
    return buf, [buf[a:a + n] for a, n in places]


def _norm(grads, max_norm, acc=None, deferred=False, norms=True, fill=255):
    res = torch.full((32,), fill, dtype=torch.uint8, device=DEV)
    ws = torch.full((_lib.grpo_grad_norm_workspace_size(grads),), fill, dtype=torch.uint8, device=DEV)
    tn = torch.full((len(grads) + 1,), -7.0, device=DEV) if norms else None
    _lib.grpo_grad_norm(grads, max_norm, res, ws, tensor_norms=tn, acc=acc, deferred=deferred)
    if norms:
        assert tn[-1] == -7.0
        tn = tn[:-1]
    return res, tn


def _check(grads, max_norm, scale=1.0, **kw):
    res, tn = _norm(grads, max_norm, **kw)
    got = _lib.read_grad_norm_result(res)
    norm, coef, each = OC.clip([g.double().cpu().numpy() for g in grads], max_norm, scale)
    assert got["status"] == 0
    if norm > float(np.finfo(np.float32).max):  # (the float32 field's nearest value; sum_sq and coef hold)
        assert got["norm"] == float("inf")
    else:
        # (2^-150: half a step of the float32 field below its normal range, as for each tensor's)
        assert abs(got["norm"] - norm) <= NORM_REL * norm + 2.0 ** -150, (got, norm)
    assert abs(got["sum_sq"] - (norm / scale) ** 2) <= 2.0 ** -19 * (norm / scale) ** 2
    assert abs(got["coef"] - coef) <= COEF_REL * coef, (got, coef)
    assert np.all(np.abs(tn.double().cpu().numpy() - each) <= NORM_REL * each + 2.0 ** -150)
    return res, coef


SIZES = [[1], [0], [0, 1, 0], [7, 8, 9], [255, 256, 257, 2047], [8191, 8192, 8193], [70000, 3, 0, 81920],
         [1000] * 31 + [9], [5] * 33, [300, 0, 9000] * 171, [64] * 512, [17] * 1025]


@pytest.mark.parametrize("gaps", [[0], [8], [1, 3, 2]], ids=["packed", "aligned", "odd"])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("sizes", SIZES, ids=range(len(SIZES)))
def test_norm(sizes, dtype, gaps):
    buf, grads = _views(sizes, dtype, gaps, len(sizes))
    _check(grads, 1.0)


def test_the_order_of_the_sums_goes_by_the_sizes_alone():
    n = 100_003
    x = torch.randn(n, device=DEV)
    want = None
    for off in range(5):
        buf = torch.zeros(n + 9, device=DEV)
        buf[off:off + n] = x
        res, tn = _norm([buf[off:off + n]], 1.0)
        got = (res.clone(), tn)
        assert want is None or (torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]))
        want = got


def test_long_tensors_and_many_chunks():
    # more than 16384 chunks of 8192, so longer ones; over 8 chunks a tensor, over 256, and one
    g = [torch.randn(n, device=DEV).to(BF16) for n in (150_000_007, 8192 * 3 + 1, 12_345_678, 5)]
    res, tn = _norm(g, 1.0)
    each = [float(x.double().square().sum().sqrt()) for x in g]
    assert np.all(np.abs(tn.cpu().numpy() - np.array(each)) <= NORM_REL * np.array(each))
    norm = math.sqrt(sum(v * v for v in each))
    assert abs(_lib.read_grad_norm_result(res)["norm"] - norm) <= NORM_REL * norm


def test_a_tensor_past_2_to_the_31_elements():
    n = (1 << 31) + 70001
    g = torch.zeros(n, dtype=BF16, device=DEV)
    g[:3] = 3.0
    g[n - 70000:] = 0.5  # from 2^31 + 1 on
    res, tn = _norm([g], 2.0)
    want = math.sqrt(27 + 70000 / 4)
    assert abs(float(tn[0]) - want) <= NORM_REL * want
    out = torch.full((n,), 7.0, dtype=BF16, device=DEV)
    _lib.grpo_grad_clip([g], res, out=[out])
    assert abs(float(out[n - 1]) - 1.0 / want) <= 2.0 ** -7 / want and float(out[n - 70000]) == float(out[n - 1])
    assert abs(float(out[0]) - 6.0 / want) <= 2.0 ** -7 * 6 / want and torch.count_nonzero(out[3:n - 70000]) == 0


@pytest.mark.parametrize("value", [3e38, 1e30, 1e19, 1e-19, 1e-23, 1e-30, 1.2e-38, 1e-44])
@pytest.mark.parametrize("n", [1, 9, 20000])
def test_the_ends_of_the_range(value, n):
    g = torch.full((n,), value, device=DEV)
    norm = float(g[0].double()) * math.sqrt(n)
    res, tn = _norm([g], 1.0)
    got = _lib.read_grad_norm_result(res)
    assert abs(got["sum_sq"] - norm ** 2) <= 2.0 ** -19 * norm ** 2 and got["status"] == 0
    if norm < 3.4e38:
        assert abs(got["norm"] - norm) <= NORM_REL * norm + 2.0 ** -149
    mixed = torch.randn(n, device=DEV)
    mixed[n // 2] = value
    _check([mixed, g[:1]], float("inf") if norm > 1e38 else 1.0)


@pytest.mark.parametrize("out_dtype", [F32, BF16])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("gaps", [([0], [0]), ([8], [8]), ([1, 3, 2], [1, 3, 2]), ([8], [1, 2]), ([5], [8])])
@pytest.mark.parametrize("sizes", [[1, 0, 9], [8191, 8193, 16], [70001], [300, 0, 9000] * 171])
def test_clip(sizes, gaps, dtype, out_dtype):
    buf, grads = _views(sizes, dtype, gaps[0], 3)
    out_buf, out = _views(sizes, out_dtype, gaps[1], 4)
    before, inside = out_buf.clone(), torch.zeros(out_buf.numel(), dtype=torch.bool, device=DEV)
    for o in out:
        a = (o.data_ptr() - out_buf.data_ptr()) // o.element_size() if o.numel() else 0
        inside[a:a + o.numel()] = True
    res, coef = _check(grads, 0.75)
    keep = buf.clone()
    _lib.grpo_grad_clip(grads, res, out=out)
    rel = COEF_REL + (2.0 ** -8 if out_dtype is BF16 else 2.0 ** -24)
    for g, o in zip(grads, out):
        want = g.double() * coef
        assert torch.all((o.double() - want).abs() <= rel * want.abs() + 2.0 ** -133)
    assert torch.equal(buf, keep) and torch.equal(out_buf[~inside], before[~inside])
    if dtype is out_dtype:
        want = [torch.empty_like(g) for g in grads]  # aligned
        _lib.grpo_grad_clip(grads, res, out=want)
        _lib.grpo_grad_clip(grads, res)  # in place
        for g, o in zip(grads, want):
            assert torch.equal(g, o)


def test_below_the_limit_nothing_changes():
    buf, grads = _views([1000, 77], BF16, [1], 5)
    keep = buf.clone()
    res, _ = _norm(grads, 1e6)
    assert _lib.read_grad_norm_result(res)["coef"] == 1.0
    _lib.grpo_grad_clip(grads, res)
    assert torch.equal(buf, keep)
    out = [torch.empty_like(g) for g in grads]
    _lib.grpo_grad_clip(grads, res, out=out)
    assert all(torch.equal(a, b) for a, b in zip(out, grads))
    for limit, want in ((float("inf"), 1.0), (0.0, 0.0)):
        assert _lib.read_grad_norm_result(_norm(grads, limit)[0])["coef"] == want


def test_no_tensors_and_zero_gradients():
    res, _ = _norm([], 1.0)
    assert _lib.read_grad_norm_result(res) == dict(sum_sq=0.0, norm=0.0, coef=1.0, status=0)
    _lib.grpo_grad_clip([], res)
    zero = [torch.zeros(20000, device=DEV), -torch.zeros(3, device=DEV)]
    for limit in (0.0, 1.0):
        res, tn = _norm(zero, limit)
        assert _lib.read_grad_norm_result(res) == dict(sum_sq=0.0, norm=0.0, coef=1.0, status=0)
        assert torch.all(tn == 0)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("at", [0, 9000, 20002])
def test_a_non_finite_gradient_skips_the_step(bad, dtype, at):
    buf, grads = _views([20003, 50], dtype, [2], 6)
    grads[0][at] = bad
    res, tn = _norm(grads, 1.0)
    got = _lib.read_grad_norm_result(res)
    assert got["status"] == _lib.STEP_SKIPPED_NONFINITE and got["coef"] == 0.0 and not math.isfinite(got["norm"])
    assert not torch.isfinite(tn[0]) and torch.isfinite(tn[1])
    out = [torch.full_like(g, 7.0) for g in grads]
    _lib.grpo_grad_clip(grads, res, out=out)
    _lib.grpo_grad_clip(grads, res)
    assert all(torch.all(g == 0) for g in out + grads)


def _acc(divisor, status=0):
    acc = _lib.new_step_acc(DEV)
    acc.view(torch.int64)[5] = divisor
    acc.view(torch.int32)[16 + 14] = status
    return acc


@pytest.mark.parametrize("divisor", [0, 1, 1000, 36500])
def test_the_deferred_scale(divisor):
    _, grads = _views([5000, 300], F32, [4], 7, scale=30.0)
    s = 1.0 / max(divisor, 1)
    for limit in (0.01, 1e6):
        res, coef = _check(grads, limit, scale=s, acc=_acc(divisor), deferred=True)
    assert coef == s
    _check(grads, 1.0, acc=_acc(divisor))


@pytest.mark.parametrize("status", [1, -8, -9])
def test_a_skipped_step_stays_skipped(status):
    _, grads = _views([500], F32, [0], 8)
    res, tn = _norm(grads, 1.0, acc=_acc(10, status), deferred=True)
    got = _lib.read_grad_norm_result(res)
    assert got["status"] == status and got["coef"] == 0.0 and float(tn[0]) > 0
    _lib.grpo_grad_clip(grads, res)
    assert torch.all(grads[0] == 0)


def test_refusals():
    a, b = torch.zeros(64, device=DEV), torch.zeros(64, dtype=BF16, device=DEV)
    res = _lib.new_grad_norm_result()
    ws = torch.empty(4096, dtype=torch.uint8, device=DEV)
    for bad in (-1.0, float("nan")):
        with pytest.raises(_lib.GrpoError):
            _lib.grpo_grad_norm([a], bad, res, ws)
    with pytest.raises(_lib.GrpoError):
        _lib.grpo_grad_norm([a], 1.0, res, ws, deferred=True)
    with pytest.raises(_lib.GrpoError):
        _lib.grpo_grad_norm([a], 1.0, res, ws[:64])
    for bad in ([a.half()], [a.cpu()], [a.view(8, 8).t()]):
        with pytest.raises(ValueError):
            _lib.grpo_grad_norm(bad, 1.0, res, ws)
    with pytest.raises(ValueError):
        _lib.grpo_grad_norm([a], 1.0, res[:16], ws)
    with pytest.raises(ValueError):
        _lib.grpo_grad_norm([a, b], 1.0, res, ws, tensor_norms=torch.empty(1, device=DEV))
    _lib.grpo_grad_norm([a], 1.0, res, ws)
    with pytest.raises(ValueError):
        _lib.grpo_grad_clip([a], res, out=[a[:32]])
    for src, out in (([a[:32], a[16:48]], None), ([a, a], None), ([a], [a.view(BF16)[:64]]), ([a[:32]], [a[1:33]]),
                     ([a[:32], a[32:]], [a[32:], a[:32]])):
        with pytest.raises(_lib.GrpoError):
            _lib.grpo_grad_clip(src, res, out=out)
    _lib.grpo_grad_clip([a[:32], a[32:]], res)  # neighbours
    _lib.grpo_grad_clip([a[:32], a[:32]], res, out=[b[:32], b[32:]])  # one source twice


def test_a_captured_norm_and_clip_replay_on_new_gradients():
    buf, grads = _views([70000, 33, 900], F32, [3], 9)
    res, ws = _lib.new_grad_norm_result(), torch.empty(_lib.grpo_grad_norm_workspace_size(grads), dtype=torch.uint8, device=DEV)
    def go():
        _lib.grpo_grad_norm(grads, 1.0, res, ws)
        _lib.grpo_grad_clip(grads, res)
    first = buf.clone()
    go()
    want, tensors = buf.clone(), [x.clone() for x in grads]
    buf.copy_(first)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        go()
    for k in (1.0, 0.5, 1.0):
        buf.copy_(first * k)
        g.replay()
        torch.cuda.synchronize()
        # (the tensors: the gaps between them stay as they were, first * k)
        assert all((x - y).abs().max() <= 2.0 ** -20 * y.abs().max() for x, y in zip(grads, tensors))
        if k == 1.0:
            assert torch.equal(buf, want)


def test_a_step_from_hidden_states_to_clipped_gradients():
    # micro-batches of the policy loss and of the cross entropy into one dW, the finish, the norm with the
    # deferred scale, and the clip into bf16
    T, V, H = 256, 3000, 128
    rng = np.random.default_rng(0)
    t = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(DEV)
    h = t(rng.standard_normal((2, T, H)).astype(np.float32)).to(BF16)
    W = t((rng.standard_normal((V, H)) / math.sqrt(H)).astype(np.float32)).to(BF16)
    y, mask = rng.integers(0, V, (2, T)).astype(np.int32), (rng.random((2, T)) < 0.7).astype(np.uint8)
    dW, d_h = torch.zeros((V, H), device=DEV), torch.empty((2, T, H), device=DEV)
    loss, acc = torch.empty((2, T), device=DEV), _lib.new_step_acc(DEV)
    ws = torch.empty(_lib.grpo_lmhead_ce_workspace_size(T, V, H), dtype=torch.uint8, device=DEV)
    for i in range(2):
        _lib.grpo_lmhead_ce_fwd_bwd(h[i], W, t(y[i]), t(mask[i]), 1.0, d_h[i], dW, loss[i], acc, ws,
                                    label_smoothing=0.1, dw_accumulate=True)
    N = int(mask.sum())
    step = _lib.grpo_finish_step(acc, loss.view(-1), expected_N=N)
    assert step["status"] == 0
    bias = torch.randn(V, device=DEV).to(BF16)  # another parameter's gradient sum
    grads, out = [dW, bias], [torch.empty((V, H), dtype=BF16, device=DEV), torch.empty(V, dtype=BF16, device=DEV)]
    res, tn = _norm(grads, 0.01, acc=acc, deferred=True)
    _lib.grpo_grad_clip(grads, res, out=out)
    ref = OC.lmhead(h.view(-1, H).double().cpu().numpy(), W.double().cpu().numpy(), y.ravel(), mask.ravel(), 1.0, eps=0.1)
    assert abs(step["loss"] - ref["loss"].sum() / N) <= 1e-5 * ref["loss"].sum() / N
    norm, coef, _ = OC.clip([ref["dW"], bias.double().cpu().numpy()], 0.01, 1.0 / N)
    got = _lib.read_grad_norm_result(res)
    # dlogits as bf16: 2^-8 of each entry, so of the norm of dW too, at most by |dx|^T |h| over |dx^T h|
    slack = np.linalg.norm(np.abs(ref["dx"]).T @ np.abs(h.view(-1, H).double().cpu().numpy())) / np.linalg.norm(ref["dW"])
    rel = (2.0 ** -8 + 2.0 ** -10) * slack
    assert abs(got["norm"] - norm) <= rel * norm and abs(got["coef"] - coef) <= 2 * rel * coef
    want = dW.double() * got["coef"]
    assert torch.all((out[0].double() - want).abs() <= (2.0 ** -8 + 2.0 ** -22) * want.abs())
    norm2, coef2, _ = OC.clip([g.double().cpu().numpy() for g in grads], 0.01, 1.0 / N)
    assert abs(got["norm"] - norm2) <= NORM_REL * norm2 and abs(got["coef"] - coef2) <= COEF_REL * coef2

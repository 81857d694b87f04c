"""GPU gradient norm and clip of lists long enough for every loop of their kernels: shares of more than 14336
elements, where a thread folds its sums (13 million elements and more), and the clip's groups of vectors, in both
types, aligned and not. Tolerances of test_gpu_clip.py for the norms; a clip multiplies in float32 by the
factor that the result holds and rounds to the output's type, so its bits are those of the same two roundings."""
import math

import pytest
import torch

from rl_post_token_gb300 import _lib
from tests.test_gpu_clip import BF16, DEV, F32, NORM_REL, _built, _norm, _views  # noqa: F401

pytestmark = pytest.mark.gpu
# one tensor past one, two and six waves of shares of 32768 elements, the last at its most shares; and a list whose
# shares hold parts of several tensors
LONG = [[13_200_001], [70_000_003], [190_000_007], [20_000_001, 5, 0, 33_333, 9_999_999, 1, 12_345_678] + [70_001] * 40]


def _sums(grads):
    step = 1 << 26
    return [math.fsum(float(g[a:a + step].double().square().sum()) for a in range(0, g.numel(), step)) for g in grads]


@pytest.mark.parametrize("gaps", [[0], [8], [1, 3, 2]], ids=["packed", "aligned", "odd"])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("sizes", LONG, ids=range(len(LONG)))
def test_norm_of_long_lists(sizes, dtype, gaps):
    buf, grads = _views(sizes, dtype, gaps, len(sizes))
    res, tn = _norm(grads, 1.0)
    got, sums = _lib.read_grad_norm_result(res), _sums(grads)
    total = math.fsum(sums)
    assert abs(got["sum_sq"] - total) <= 2.0 ** -19 * total and got["status"] == 0
    assert abs(got["norm"] - math.sqrt(total)) <= NORM_REL * math.sqrt(total)
    for have, s in zip(tn.tolist(), sums):
        assert abs(have - math.sqrt(s)) <= NORM_REL * math.sqrt(s)


@pytest.mark.parametrize("dtype, n", [(F32, 60_000_011), (BF16, 60_000_011)])
def test_the_order_of_long_sums_goes_by_the_sizes_alone(dtype, n):
    g = torch.Generator(device=DEV)
    g.manual_seed(n)
    x = torch.randn(n, generator=g, device=DEV).to(dtype)
    buf, want = torch.zeros(n + 9, dtype=dtype, device=DEV), None
    for off in (0, 1, 3, 8):
        buf[off:off + n] = x
        res, tn = _norm([buf[off:off + n]], 1.0)
        assert want is None or (torch.equal(res, want[0]) and torch.equal(tn, want[1]))
        want = res, tn


@pytest.mark.parametrize("at", [0, 13_000_000, 59_999_999])
@pytest.mark.parametrize("off", [0, 1])
@pytest.mark.parametrize("bad", [float("nan"), float("-inf"), 3e38])
def test_a_large_or_non_finite_element_of_a_long_tensor(bad, off, at):
    n = 60_000_000
    buf = torch.full((n + 1,), 0.5, device=DEV)
    buf[off + at] = bad
    res, tn = _norm([buf[off:off + n]], 1.0)
    got = _lib.read_grad_norm_result(res)
    if math.isfinite(bad):  # (3e38: the share's sum is formed again in float64)
        big = float(buf[off + at].double()) ** 2
        assert got["status"] == 0 and abs(got["sum_sq"] - big) <= 2.0 ** -19 * big
    else:
        assert got["status"] == _lib.STEP_SKIPPED_NONFINITE and got["coef"] == 0.0 and not torch.isfinite(tn).any()


@pytest.mark.parametrize("out_dtype", [F32, BF16])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("gaps", [([0], [0]), ([1, 3, 2], [1, 3, 2]), ([8], [1, 2])], ids=["packed", "odd", "apart"])
@pytest.mark.parametrize("sizes", LONG[:1] + LONG[3:], ids=["one", "list"])
def test_clip_of_long_lists(sizes, gaps, dtype, out_dtype):
    buf, grads = _views(sizes, dtype, gaps[0], 3)
    out_buf, out = _views(sizes, out_dtype, gaps[1], 4)
    places = [(o.storage_offset(), o.numel()) for o in out]
    want, keep = out_buf.clone(), buf.clone()
    res, _ = _norm(grads, 0.75)
    coef = res.view(F32)[3]
    assert 0 < float(coef) < 1
    for (a, n), g in zip(places, grads):
        want[a:a + n] = (g.float() * coef).to(out_dtype)
    _lib.grpo_grad_clip(grads, res, out=out)
    assert torch.equal(out_buf, want) and torch.equal(buf, keep)
    if dtype is out_dtype:
        for g in grads:
            a = g.storage_offset()
            keep[a:a + g.numel()] = (g.float() * coef).to(dtype)
        _lib.grpo_grad_clip(grads, res)  # in place
        assert torch.equal(buf, keep)

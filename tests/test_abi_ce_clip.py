"""Argument checks of the cross entropy, gradient norm and clip entry points, on the CPU: answered before any
device memory or CUDA call is touched (placeholder pointers, never dereferenced)."""
import ctypes as C

import pytest

from rl_post_token_gb300 import _lib

P = 1 << 20  # a placeholder address
Q = 1 << 16  # the matrices' distance


@pytest.fixture(scope="module", autouse=True)
def _no_gpu(grpo_lib):
    import torch
    if torch.cuda.is_available():
        pytest.skip("host-side argument checks are exercised without a GPU")
    return grpo_lib


def _ce(T=4, V=10, H=64, h=P, W=P, target=P, mask=P, eps=0.0, lam=0.0, cap=0.0, scale=1.0, d_h=P, dh=0, dW=P, dw=0,
        flags=0, loss=P, acc=P, ws=P, size=None):
    need = _lib.lib().grpo_lmhead_ce_workspace_size(max(T, 1), max(V, 1), max(H, 8))
    tm = _lib.grpo_ce_terms(eps, lam, cap, None)
    h, W, d_h, dW = (x + k * Q if x == P else x for k, x in enumerate((h, W, d_h, dW)))
    return _lib.lib().grpo_lmhead_ce_fwd_bwd(h, W, T, V, H, target, mask, C.byref(tm), scale, d_h, dh, dW, dw, flags, loss,
                                             None, None, acc, ws, need if size is None else size, None)


INV = dict(T=[-1, 1 << 31], V=[0, -3, 1 << 31], H=[0, 4, 60, 66, -8, (1 << 24) + 8], h=[None, P + 2, P + 8], W=[None, P + 8],
           target=[None], eps=[-0.1, 1.01, float("nan")], lam=[-1.0, float("nan"), float("inf")],
           cap=[-1.0, 1e-7, 1e7, float("nan"), float("inf")], scale=[float("nan"), float("inf")], d_h=[P + 4], dW=[P + 8],
           flags=[2, 4, 1 << 31], loss=[None], acc=[None, P + 4], ws=[None, P + 128])


@pytest.mark.parametrize("key, value", [(k, v) for k, vs in INV.items() for v in vs])
def test_cross_entropy_refuses(key, value):
    assert _ce(**{key: value}) == _lib.ERR_INVALID


def test_cross_entropy_types_sizes_and_capacity():
    for bad in (2, -1):
        assert _ce(dh=bad) == _lib.ERR_UNSUPPORTED and _ce(dw=bad) == _lib.ERR_UNSUPPORTED
    assert _ce(dw=1, flags=1) == _lib.ERR_INVALID  # bf16 sums
    need = _lib.grpo_lmhead_ce_workspace_size(4, 10, 64)
    assert need > 0 and _ce(size=need - 1) == _lib.ERR_CAPACITY
    for bad in ((0, 10, 64), (4, 0, 64), (4, 10, 0), (-1, 10, 64), (1 << 31, 10, 64), (4, 1 << 31, 64),
                (4, 10, (1 << 24) + 8)):
        assert _lib.grpo_lmhead_ce_workspace_size(*bad) == 0
    assert _ce(T=0, dW=None) == _lib.OK  # nothing to launch


@pytest.mark.parametrize("kw", [dict(d_h=P + 16), dict(d_h=P + Q + 16), dict(dW=P + 4 * 64 * 2 - 16), dict(dW=P + Q + 16),
                                dict(dW=P + 2 * Q + 4 * 64 * 4 - 16), dict(d_h=P + Q - 16, dh=1)])
def test_cross_entropy_refuses_overlaps(kw):
    assert _ce(**kw) == _lib.ERR_INVALID


def _list(n, ptr=P, numel=8, dtype=0, gap=1 << 12):
    return ((C.c_uint64 * n)(*[ptr + i * gap for i in range(n)]), (C.c_int64 * n)(*[numel] * n), (C.c_int32 * n)(*[dtype] * n))


def _norm(n=2, ptr=P, numel=8, dtype=0, max_norm=1.0, acc=None, deferred=0, result=P, ws=P, size=1 << 16):
    p, m, d = _list(max(n, 0), ptr, numel, dtype)
    return _lib.lib().grpo_grad_norm(p, m, d, n, max_norm, acc, deferred, None, result, ws, size, None)


@pytest.mark.parametrize("kw", [dict(n=-1), dict(ptr=P + 2), dict(ptr=0, n=1), dict(dtype=1, ptr=P + 1), dict(numel=-1),
                                dict(numel=1 << 49), dict(max_norm=-1.0), dict(max_norm=float("nan")), dict(deferred=1),
                                dict(acc=P + 4), dict(result=None), dict(result=P + 4), dict(ws=None), dict(ws=P + 4)])
def test_norm_refuses(kw):
    assert _norm(**kw) == _lib.ERR_INVALID


def test_norm_types_and_capacity():
    assert _norm(dtype=2) == _lib.ERR_UNSUPPORTED
    size = _lib.lib().grpo_grad_norm_workspace_size(16, 2)
    assert 0 < size <= 512 and _norm(size=size - 1) == _lib.ERR_CAPACITY
    assert _lib.lib().grpo_grad_norm_workspace_size(-1, 2) == 0 == _lib.lib().grpo_grad_norm_workspace_size(1, -2)
    assert _lib.lib().grpo_grad_norm_workspace_size((1 << 32) + 5, 32768) <= 400 << 10
    assert _lib.lib().grpo_grad_norm(None, None, None, 1, 1.0, None, 0, None, P, P, 4096, None) == _lib.ERR_INVALID


def _clip(src, dst, numels, sd=None, dd=None, result=P):
    n = len(src)
    return _lib.lib().grpo_grad_clip((C.c_uint64 * n)(*src), (C.c_int32 * n)(*(sd or [0] * n)), (C.c_uint64 * n)(*dst),
                                     (C.c_int32 * n)(*(dd or [0] * n)), (C.c_int64 * n)(*numels), n, result, None)


@pytest.mark.parametrize("src, dst, numels, sd, dd", [
    ([P], [P + 4], [8], [0], [0]),               # shifted by one
    ([P], [P], [8], [0], [1]),                   # in place with another type
    ([P, P], [P, P], [8, 8], None, None),        # one tensor twice
    ([P, P + 16], [P, P + 16], [8, 8], None, None),
    ([P, P + 4096], [P + 4096, P + 8192], [8, 8], None, None),  # written and read
    ([P, P + 64], [P + 4096, P + 4096], [8, 8], None, None),    # written twice
    ([P] * 40, [P + 4096 + 16 * i for i in range(40)], [8] * 40, None, None),
])
def test_clip_refuses_overlaps(src, dst, numels, sd, dd):
    assert _clip(src, dst, numels, sd, dd) == _lib.ERR_INVALID


def test_clip_refuses_the_rest():
    assert _clip([P], [P], [8], result=None) == _lib.ERR_INVALID and _clip([P], [P], [8], result=P + 4) == _lib.ERR_INVALID
    assert _clip([P], [P], [8], [0], [3]) == _lib.ERR_UNSUPPORTED and _clip([P], [P + 2], [1]) == _lib.ERR_INVALID
    assert _clip([P], [0], [8]) == _lib.ERR_INVALID
    assert _clip([0, P], [0, P], [0, 0]) == _lib.OK  # nothing to do


def test_struct_sizes():
    assert C.sizeof(_lib.grpo_grad_norm_result) == _lib.GRAD_NORM_BYTES == 32
    assert C.sizeof(_lib.grpo_ce_terms) == 24

"""Argument checks of the distillation entry points, on the CPU: answered before any device memory or CUDA
call is touched (placeholder pointers, never dereferenced)."""
import pytest

from rl_post_token_gb300 import _lib
from tests import test_abi_validation as A


@pytest.fixture(scope="module", autouse=True)
def _no_gpu(grpo_lib):
    import torch
    if torch.cuda.is_available():
        pytest.skip("host-side argument checks are exercised without a GPU")
    return grpo_lib


@pytest.mark.parametrize("off", [1, 2, 4])
def test_the_step_accumulator_must_be_aligned(off):
    # its counters take 64-bit atomics; a slice of a byte buffer may start anywhere
    assert A._distill(acc=A.P + off) == _lib.ERR_INVALID
    assert A._lm_distill(acc=A.P + off) == _lib.ERR_INVALID


@pytest.mark.parametrize("tau, code", [(1e-38, _lib.ERR_INVALID), (1.69e-38, _lib.ERR_INVALID), (1.75e-38, _lib.OK),
                                       (1e-30, _lib.OK), (1.2e38, _lib.OK), (1.3e38, _lib.ERR_INVALID)])
def test_temperatures_whose_scale_is_no_ordinary_float(tau, code):
    # log2(e)/tau from 2^-126 to below 2^126; with no rows there is nothing to launch
    assert A._score(T=0, temperature=tau) == code
    assert A._distill(T=0, temperature=tau) == code

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

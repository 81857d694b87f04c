"""GPU scoring and distillation of rows whose logits leave the float32 range after the scaling by
log2(e)/tau, against the oracles: above it a row has no distribution, and is counted."""
import numpy as np
import pytest
import torch

from oracle import score as OS
from rl_post_token_gb300 import _lib
from rl_post_token_gb300 import workloads as W
from tests import test_gpu_distill as D
from tests import test_gpu_score as S

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _built(grpo_lib):
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return grpo_lib


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T, V", [(6, 700), (6, 40000), (470, 40001)])
def test_the_types_largest_value(T, V, dtype):
    big = torch.finfo(D.DT[dtype]).max
    z, idx, lq = D._inputs(T, V, 9, dtype, 5, unused=0.0)
    z[1, V - 7] = big          # outside the list
    z[2, int(idx[2, 3])] = big  # a listed token
    z[3, 5:] = big             # whole tiles
    bad = [1, 2, 3]
    o = S._check(z, 9, rows=range(6))
    assert all(np.isnan(o["entropy_tok"][r].item()) for r in bad) and torch.isfinite(o["entropy_tok"][4:]).all()
    for kind in D.KINDS:
        loss, dz, acc = D._check(z, idx, lq, kind, dtype=dtype, rows=range(6))
        assert torch.isnan(loss[bad]).all() and torch.isnan(dz[bad]).all()
        assert _lib.grpo_finish_step(acc, loss)["n_nonfinite"] == 3
    # at a temperature of 2 its scaled value is a float32 number: a distribution of one token
    one = S._call(z, 9, torch.full((T,), V - 7, dtype=torch.int32, device=DEV), temperature=2.0)
    assert one["logp_tok"][1].item() == 0 and one["entropy_tok"][1].item() == 0
    assert one["top_idx"][1, 0].item() == V - 7 and one["top_logp"][1, 0].item() == 0
    zh = W.logits_to_host(z[:6])
    for r in range(6):
        logp, H, top, _ = OS.score_row(zh[r], V - 7, 9, 2.0)
        assert np.array_equal(one["top_idx"][r].cpu().numpy(), top)

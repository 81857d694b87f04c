"""The LM-head distillation of a list scored at another temperature: h / tau in the place of h, d_h / tau of
the result. At a power of two nothing is rounded by it, so that the logits are those of the row call at that
temperature. Bars: the other LM-head tests' (loss: the log-prob bar of both calls; d_h and dW: bf16 dlogits,
half a step 2^-8 of each product)."""
import pytest
import torch

from rl_post_token_gb300 import _lib
from tests import test_gpu_lmhead_distill as L

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("tau", [0.5, 2.0])
def test_a_list_scored_at_another_temperature(grpo_lib, tau):
    h, Wt, idx, lq, mask = L._inputs(96, 5000, 128, 24, 9, std=0.2)
    loss, d_h, dW, _ = L._call((h / tau).contiguous(), Wt, idx, lq, mask, 1.0)
    z = (h.double() @ Wt.double().T).float()
    want, dz = torch.empty(96, device=DEV), torch.empty_like(z)
    _lib.grpo_distill_topk_fwd_bwd(z, L._t(idx), L._t(lq), L._t(mask), _lib.DISTILL_FORWARD_TOPK, 1.0, dz, want,
                                   _lib.new_step_acc(DEV), temperature=tau)
    assert torch.all((loss - want).abs() <= 2e-5 * torch.clamp(want.abs(), min=1.0) + 2e-5)
    dz, w, hd = dz.double(), Wt.double(), h.double()  # dz holds its 1 / tau
    bar = 2.0 ** -8 + 2.0 ** -10 + 1e-4
    assert torch.all((d_h.double() / tau - dz @ w).abs() <= bar * (dz.abs() @ w.abs()) + 1e-9)
    assert torch.all((dW.double() - dz.T @ hd).abs() <= bar * (dz.abs().T @ hd.abs()) + 1e-9)

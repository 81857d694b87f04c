"""Refusals of the scoring and distillation bindings: per-token tensors that are not contiguous. The
kernels walk them by element, so a slice of a [B, S] tensor would be read and written in the wrong places,
and an expanded one past its storage. Without a GPU the check is called on stand-ins for device tensors."""
import pytest
import torch

from rl_post_token_gb300 import _lib


class OnDevice:
    """A host tensor that says it is on device 0."""
    is_cuda = True

    def __init__(self, t):
        self.t = t

    def get_device(self):
        return 0

    def __getattr__(self, name):
        return getattr(self.t, name)


@pytest.fixture
def device0(monkeypatch):
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)


def _slices(dtype):
    """Tensors of at least 12 elements that are not 12 elements in a row."""
    z = torch.zeros((3, 6), dtype=dtype)
    return [z[:, 1:], torch.zeros((3, 8), dtype=dtype)[:, ::2], torch.zeros((6, 3), dtype=dtype).t(), z[:1, :1].expand(3, 4),
            z[:1, :1].expand(12, 1), torch.zeros(24, dtype=dtype)[::2], torch.zeros(1, dtype=dtype).expand(12),
            torch.zeros((2, 3, 4), dtype=dtype).transpose(0, 1)]


@pytest.mark.parametrize("n", [12, 0])  # (0: the count is not known, the rows are indexed through tok_src)
@pytest.mark.parametrize("case", range(8))
def test_per_token_tensors_must_be_contiguous(device0, case, n):
    logits = OnDevice(torch.zeros((12, 8)))
    t = _slices(torch.uint8)[case]
    with pytest.raises(ValueError, match="mask must be contiguous"):
        _lib._device_args(logits, ("mask", OnDevice(t), torch.uint8, n))


@pytest.mark.parametrize("t", [torch.zeros(12), torch.zeros((3, 4)), torch.zeros((12, 1)), torch.zeros(40)[5:17],
                               torch.zeros((9, 4))[2:6], torch.zeros((1, 12)), torch.zeros((5, 30))[:1, 2:20]])
def test_contiguous_ones_of_any_shape_are_taken(device0, t):
    _lib._device_args(OnDevice(torch.zeros((12, 8))), ("w_tok", OnDevice(t), torch.float32, 12), ("none", None, None, 0))
    with pytest.raises(ValueError, match="at least 41"):
        _lib._device_args(OnDevice(torch.zeros((12, 8))), ("w_tok", OnDevice(t), torch.float32, 41))


@pytest.mark.gpu
def test_the_calls_refuse_slices(grpo_lib):
    dev = "cuda"
    B, S, V, K = 2, 6, 500, 4
    T = B * (S - 1)
    z = torch.randn((T, V), device=dev)
    idx = torch.empty((T, K), dtype=torch.int32, device=dev)
    lq = torch.empty((T, K), device=dev)
    full = lambda dt: torch.ones((B, S), dtype=dt, device=dev)
    mask, loss, acc = torch.ones((B, S - 1), dtype=torch.uint8, device=dev), torch.zeros((B, S - 1), device=dev), _lib.new_step_acc(dev)
    src = torch.arange(T, device=dev)
    _lib.grpo_token_topk_logprobs(z, K, top_idx=idx, top_logp=lq, mask=mask, entropy_tok=loss)  # any shape in a row
    h, Wt = torch.zeros((T, 64), dtype=torch.bfloat16, device=dev), torch.zeros((V, 64), dtype=torch.bfloat16, device=dev)
    ws = torch.empty(_lib.grpo_lmhead_distill_workspace_size(T, V, 64, K), dtype=torch.uint8, device=dev)
    bad_mask = [full(torch.uint8)[:, 1:], torch.ones((1, 1), dtype=torch.uint8, device=dev).expand(B, S - 1)]
    for tok_src in (None, src):
        for m in bad_mask:
            with pytest.raises(ValueError, match="contiguous"):
                _lib.grpo_token_topk_logprobs(z, K, top_idx=idx, top_logp=lq, mask=m, tok_src=tok_src)
            with pytest.raises(ValueError, match="contiguous"):
                _lib.grpo_distill_topk_fwd_bwd(z, idx, lq, m, 0, 1.0, None, loss, acc, tok_src=tok_src)
        for kw in (dict(logp_tok=full(torch.float32)[:, 1:], target=full(torch.int32)[:, :5].contiguous()),
                   dict(logp_tok=loss, target=full(torch.int32)[:, 1:]), dict(entropy_tok=full(torch.float32)[:, :5])):
            with pytest.raises(ValueError, match="contiguous"):
                _lib.grpo_token_topk_logprobs(z, 0, tok_src=tok_src, **kw)
        with pytest.raises(ValueError, match="contiguous"):
            _lib.grpo_distill_topk_fwd_bwd(z, idx, lq, mask, 0, 1.0, None, full(torch.float32)[:, 1:], acc, tok_src=tok_src)
        with pytest.raises(ValueError, match="contiguous"):
            _lib.grpo_distill_topk_fwd_bwd(z, idx, lq, mask, 0, 1.0, None, loss, acc, w_tok=full(torch.float32)[:, 1:],
                                           tok_src=tok_src)
    for m, l, w in ((bad_mask[0], loss, None), (bad_mask[1], loss, None), (mask, full(torch.float32)[:, 1:], None),
                    (mask, loss, full(torch.float32)[:, :5])):
        with pytest.raises(ValueError, match="contiguous"):
            _lib.grpo_lmhead_distill_topk_fwd_bwd(h, Wt, idx, lq, m, 1.0, None, None, l, acc, ws, w_tok=w)
    with pytest.raises(ValueError):
        _lib.grpo_token_topk_logprobs(z, K, top_idx=idx[:, :3], top_logp=lq[:, :3])
    with pytest.raises(ValueError):
        _lib.grpo_token_topk_logprobs(z, K, top_idx=idx.view(-1), top_logp=lq.view(-1))
    _lib.grpo_distill_topk_fwd_bwd(z, idx, lq, mask, 0, 1.0, None, loss, acc, tok_src=src)
    assert _lib.grpo_finish_step(acc, loss, expected_N=T)["status"] == 0

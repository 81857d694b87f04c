"""Cross entropy, gradient norm and clip from several host threads at once, each on a stream of its own with
its own workspaces: the bits of the same calls made alone."""
import math
import threading

import pytest
import torch

from rl_post_token_gb300 import _lib

pytestmark = pytest.mark.gpu
DEV, BF16 = "cuda", torch.bfloat16
SIZES = [(4200, 35000, 64), (300, 9000, 264), (64, 5000, 128), (4300, 33000, 72)]  # two pieces, kept, joint, two pieces


def _job(i):
    T, V, H = SIZES[i]
    g = torch.Generator(device=DEV)
    g.manual_seed(i)
    r = lambda *s: torch.randn(s, generator=g, device=DEV)
    h, W = r(T, H).to(BF16), (r(V, H) / math.sqrt(H)).to(BF16)
    y = torch.randint(V, (T,), generator=g, device=DEV).int()
    mask = (torch.rand(T, generator=g, device=DEV) < 0.7).to(torch.uint8)
    return dict(h=h, W=W, y=y, mask=mask, d_h=torch.empty_like(h), dW=torch.empty((V, H), device=DEV), out=torch.empty_like(W),
                loss=torch.empty(T, device=DEV), acc=_lib.new_step_acc(DEV), res=_lib.new_grad_norm_result(DEV),
                ws=torch.empty(_lib.grpo_lmhead_ce_workspace_size(T, V, H), dtype=torch.uint8, device=DEV),
                ws2=torch.empty(1 << 17, dtype=torch.uint8, device=DEV), norms=torch.empty(2, device=DEV))


def _run(j, stream):
    _lib.grpo_lmhead_ce_fwd_bwd(j["h"], j["W"], j["y"], j["mask"], 0.01, j["d_h"], j["dW"], j["loss"], j["acc"], j["ws"],
                                label_smoothing=0.1, z_loss=1e-3, stream=stream)
    _lib.grpo_finish_step(j["acc"], j["loss"], sync=False, stream=stream)
    _lib.grpo_grad_norm([j["dW"], j["d_h"]], 0.5, j["res"], j["ws2"], tensor_norms=j["norms"], acc=j["acc"], deferred=True,
                        stream=stream)
    _lib.grpo_grad_clip([j["dW"]], j["res"], out=[j["out"]], stream=stream)


def test_threads_give_the_bits_of_calls_made_alone(grpo_lib):
    jobs = [_job(i) for i in range(4)]
    names = ("loss", "d_h", "dW", "out", "res", "norms")
    want = []
    for j in jobs:
        _run(j, torch.cuda.current_stream())
        torch.cuda.synchronize()
        want.append({k: j[k].clone() for k in names})
    errors = []

    def work(i):
        try:
            torch.cuda.set_device(0)
            stream = torch.cuda.Stream()
            for _ in range(6):
                _run(jobs[i], stream)
            stream.synchronize()
        except Exception as e:  # (reported by the test's own thread)
            errors.append(e)

    for _ in range(3):
        for j in jobs:
            for k in names:
                j[k].zero_()
        torch.cuda.synchronize()
        threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
        for t in threads:
            t.start()
        for t in threads:
            t.join()
        torch.cuda.synchronize()
        assert not errors, errors
        for j, w in zip(jobs, want):
            for k in names:
                assert torch.equal(j[k], w[k]), k

"""Register and spill budget of the cross entropy's and the clip's kernels, from the ptxas report the build
records (no GPU needed): 320 threads of a product share an SM's 65,536 registers, and six blocks of 256 of the
norm; a spill or a local array in their loops would cost bandwidth."""
import re

import pytest

from rl_post_token_gb300 import build as B
from tests.test_kernel_resources import _report


@pytest.mark.parametrize("src, name, n, regs", [("grpo_lmhead_ce.cu", "11gemm_kernel", 8, 200), ("grpo_lmhead_ce.cu", "10bwd_kernel", 2, 200),
                                                ("grpo_lmhead_ce.cu", "ce_", 8, 64), ("grpo_clip.cu", "11norm_kernel", 2, 40),
                                                ("grpo_clip.cu", "11clip_kernel", 2, 40), ("grpo_clip.cu", "12final_kernel", 2, 64)])
def test_no_instance_spills(grpo_lib, src, name, n, regs):
    k = {e: v for e, v in _report(src).items() if name in e and ("gemm" in e) == ("gemm" in name)}
    assert len(k) == n, sorted(k)
    for e, v in k.items():
        assert v["spill"] == 0 and v["regs"] <= regs, (e, v)
    stack = re.findall(r"Compiling entry function '(\S+)'.*?\n\s+(\d+) bytes stack frame", open(B.ptxas_report(src)).read(), flags=re.S)
    assert all(int(b) == 0 for e, b in stack if e in k), stack

"""Register and spill budget of the scoring and distillation kernels, from the ptxas report the build
records (no GPU needed): their warps share an SM's registers by launch bounds, and a spill in a loop
over a row's tiles would cost them bandwidth."""
import pytest

from tests.test_kernel_resources import _report


@pytest.mark.parametrize("src, name, n, regs", [("grpo_score.cu", "13stream_kernel", 4, 96),
                                                ("grpo_score.cu", "10row_kernel", 8, 128),
                                                ("grpo_distill.cu", "14cluster_kernel", 12, 104)])
def test_no_instance_spills(grpo_lib, src, name, n, regs):
    k = {e: v for e, v in _report(src).items() if name in e}
    assert len(k) == n, sorted(k)
    for e, v in k.items():
        assert v["spill"] == 0 and v["regs"] <= regs, (e, v)

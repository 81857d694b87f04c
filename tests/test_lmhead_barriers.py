"""The orderings that the LM-head kernels' barriers carry, read from their sources (no GPU needed): a missing
release may go unnoticed in every run."""
import glob
import os
import re

from rl_post_token_gb300 import build as B


def test_an_accumulator_is_given_back_with_a_releasing_arrive():
    files = sorted(glob.glob(os.path.join(B.CSRC, "grpo_lmhead*.cu*")))
    text = {f: open(f).read() for f in files}
    assert len(files) >= 5
    for f, s in text.items():
        assert not re.search(r"\bmbar_arrive\w*_relaxed\s*\(", s), f
    release = re.search(r"struct AccRelease \{.*?\n\};", "\n".join(text.values()), flags=re.S).group(0)
    assert "mbar_arrive_remote(" in release and "mbar_arrive(" in release
    common = open(os.path.join(B.CSRC, "grpo_common.cuh")).read()
    assert "mbarrier.arrive.release.cluster" in re.search(r"void mbar_arrive_remote\(.*?\n\}", common, flags=re.S).group(0)

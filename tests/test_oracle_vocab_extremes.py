"""The scoring and distillation oracles on rows whose logits leave the float32 range after the scaling."""
import numpy as np
import pytest

from oracle import distill as OD
from oracle import score as OS


@pytest.mark.parametrize("big", [np.finfo(np.float32).max, 3.3895e38])
def test_a_logit_above_the_range_counts_as_infinite(big):
    z = np.array([0.0, float(big), 1.0])
    logp, H, idx, top = OS.score_row(z, 1, 2)
    assert np.isnan(logp) and np.isnan(H) and idx.tolist() == [-1, -1] and np.isnan(top).all()
    for kind in range(3):
        loss, g, _ = OD.row_loss(z, [1, -1], [-0.5, 0.0], kind)
        assert np.isnan(loss) and np.isnan(g).all()
    # at a temperature of 2 it is within the range
    logp, H, idx, top = OS.score_row(z, 1, 2, tau=2.0)
    assert logp == 0 and H == 0 and idx.tolist() == [1, 2]

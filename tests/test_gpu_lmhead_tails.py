"""GPU policy loss from hidden states where a vocabulary's last tile ends on an odd group of 32 columns and the same
CTAs go on to further tiles: the dlogits' staging buffers are then taken out of their turn. Checks and tolerances
of test_gpu_lmhead.py."""
import pytest

from tests.test_gpu_lmhead import _built, _check, cta_group  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("V", [20, 256 + 70, 256 + 140])
def test_an_odd_tail_followed_by_other_tiles(cta_group, V):
    # 40000 tokens: 157 pairs' tiles (313 of one CTA) to a column of tiles, two and more to each pair (CTA)
    _check(40000, V, 64, seed=V, valid_lo=0.1, old=False)

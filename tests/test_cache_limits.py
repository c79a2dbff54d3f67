"""Limits of the paged cache's calls that the host refuses, in both directions:
the last size that is taken and the first that is not."""
import numpy as np
import pytest

import gated_deltanet_prefill_varlen_amd as gdn
from test_cache_boundary import HIP, SHAPE, append, no_gpu


@no_gpu
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_frequencies_whose_angles_are_not_held(sign):
    top = float(np.float32(65536.0))
    over = float(np.nextafter(np.float32(65536.0), np.float32(np.inf)))
    assert append(rope=gdn.make_rope([1.0] * 31 + [sign * top])) == HIP       # no device to launch on
    for f in (over, 1e30, float("inf"), float("nan")):
        assert append(rope=gdn.make_rope([1.0] * 31 + [sign * f])) == SHAPE

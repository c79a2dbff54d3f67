"""Limits of the paged cache's calls that the host refuses, in both directions:
the last size that is taken and the first that is not."""
import numpy as np
import pytest

import gated_deltanet_prefill_varlen_amd as gdn
from test_cache_boundary import HIP, SHAPE, append, cache, no_gpu, packed


@no_gpu
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_frequencies_whose_angles_are_not_held(sign):
    top = float(np.float32(65536.0))
    over = float(np.nextafter(np.float32(65536.0), np.float32(np.inf)))
    assert append(rope=gdn.make_rope([1.0] * 31 + [sign * top])) == HIP       # no device to launch on
    for f in (over, 1e30, float("inf"), float("nan")):
        assert append(rope=gdn.make_rope([1.0] * 31 + [sign * f])) == SHAPE


@no_gpu
def test_prompts_of_few_rows_that_no_launch_holds():
    """128 rows of each of 2^22 kv heads are four workgroups of 256 a head, 2^32
    threads; 96 rows are three."""
    wide = dict(c=cache(num_kv_heads=1 << 22), hq=1 << 22, out=1 << 50)
    assert packed(cu=(0, 96), **wide) == HIP and packed(cu=(0, 128), **wide) == SHAPE

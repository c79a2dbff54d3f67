"""What the state space layers' calls accept and refuse at the limits of their
launches, and which of their buffers may lie over one another; without a GPU."""
import numpy as np

import gated_deltanet_prefill_varlen_amd as gdn
from tests.test_ssm_boundary import HIP, SHAPE, need, no_gpu, prefill, ssm, step


@no_gpu
def test_many_groups():
    """A launch's second axis holds 65,535: a group each, and eight heads each."""
    wide = dict(head_dim=32, state_dim=32)
    most = 58253                                   # 58,253 + 7,282 = 65,535
    s = ssm(num_heads=most, num_groups=most, **wide)
    assert need((0, 4), s)[0] == 0 and prefill(s=s, xs=0, dts=0, pos=None, size=1 << 40) == HIP and step(s=s, snap=None) == HIP
    s = ssm(num_heads=most + 1, num_groups=most + 1, **wide)
    assert need((0, 4), s)[0] == SHAPE


@no_gpu
def test_many_prompts_and_tokens():
    """A launch's first axis holds fewer than 2^32 threads, 256 a workgroup."""
    s = gdn.make_ssm(1, 1, 32, 32)
    args = dict(s=s, pos=None, ci=None, co=None, cc=None, w=None, b=None, init=None, final=None, x=1 << 50, out=1 << 60, ws=1 << 52, dt=1 << 58,
                size=1 << 56)
    assert prefill(cu=(0, 500_000_000), **args) == HIP
    assert prefill(cu=(0, 540_000_000), **args) == SHAPE
    assert prefill(cu=np.zeros((1 << 23) + 1, np.int32), **args) == HIP

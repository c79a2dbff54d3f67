"""The packed scan at the lengths where its launches change: the chunk of 32
tokens, and the longest prompt that is not cut into segments."""
import pytest
import torch

from tests.ssm_util import Layer

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n", [31, 32, 33, 95, 96, 97, 1023, 1024, 1025, 1279, 1280, 1281, 1312, 1313, 2047, 2049])
@pytest.mark.parametrize("conv", [False, True])
def test_lengths(n, conv):
    """A prompt of n tokens between two others, and alone: the same bits."""
    y = Layer(2, 1, 64, 64, [n, 40, n], seed=n, conv=conv, init=True, window=conv)
    ck = sorted({n - 30, n, n + 40 + min(32, n), 2 * n + 40 - 1, 2 * n + 40})   # (increasing, as the call wants them)
    r = y.run(ck)
    y.check(r, y.oracle(ck), ck)
    alone = y.run(ck, only=2)
    assert torch.equal(alone["out"][:n], r["out"][n + 40:2 * n + 40]) and torch.equal(alone["final"][0], r["final"][2])
    assert torch.equal(alone["kept"], r["kept"][2:])        # (the first two are in the first prompt)

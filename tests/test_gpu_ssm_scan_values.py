"""The packed scan of state space layers on values that lie far apart, vanish,
or come near the ends of fp32's range, against the fp64 oracle."""
import pytest

from tests.ssm_util import Layer

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("what", ["x", "B", "dt", "rows"])
@pytest.mark.parametrize("conv", [False, True])
@pytest.mark.parametrize("init", [False, True])
def test_zeros(what, conv, init):
    """Zeros at a prompt's start and across its chunks and segments: one channel of x (one more in all
    prompts), B, the steps, or whole rows, on states that hardly decay.  Finite inputs, so finite results."""
    y = Layer(2, 1, 64, 64, [50, 1300, 33], seed=50, conv=conv, bias=False, init=init, a_scale=1e-3)
    parts = [(0, 40), (50, 90), (50 + 500, 50 + 560), (50 + 1023, 50 + 1100), (1350, 1383)]
    if what == "x":
        y.x[:, 7] = 0
    for a, b in parts:
        if what == "x":
            y.x[a:b, 70] = 0
        elif what == "B":
            y.x[a:b, 128:192] = 0
        elif what == "dt":
            y.dt[a:b] = -200.0           # softplus: 0 in fp32
        else:
            y.x[a:b] = 0
    ck = [20, 50, 90, 50 + 1024, 1383]
    y.check(y.run(ck), y.oracle(ck), ck)

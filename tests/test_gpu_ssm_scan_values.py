"""The packed scan of state space layers on values that lie far apart, vanish,
or come near the ends of fp32's range, against the fp64 oracle."""
import numpy as np
import pytest
import torch

from oracle import ssm_oracle as O
from tests.ssm_util import DEV, Layer, close, f64, out_tol, state_tol

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


def check(y, ck=()):
    """Against the oracle, with what fp16's smallest step adds to an output.  x is an operand times a power of
    two: half the smallest step, 2^-25, is 2^-28 of the largest |x| of its channel in the chunk of 32 tokens,
    or less (the power is 2^11 where that largest is 2^-8 or more, else it is brought to 2^14).  Outputs are
    sums of weights times x: 2^-28 of the same sum of absolute values with each |x| at its chunk's largest."""
    r, want = y.run(ck), y.oracle(ck)
    H, G, P, N = y.dims
    u = []
    for s, n in enumerate(y.lens):
        rows = f64(y.x[y.cu[s]:y.cu[s + 1]])
        if y.w is not None:
            rows = O.conv(rows, f64(y.w), f64(y.b), np.zeros((3, y.C)) if y.window is None else f64(y.window)[s])[0]
        rows = np.abs(rows)
        for c in range(0, n, 32):
            rows[c:c + 32, :H * P] = rows[c:c + 32, :H * P].max(0)
        u.append(rows)
    top = O.prefill(H, G, P, N, y.cu, np.concatenate(u), y.steps(), f64(y.A), None if y.D is None else np.abs(f64(y.D)))["out"]
    T, longest = int(y.cu[-1]), max(y.lens)
    close(r["out"][:T], want["out"], out_tol(want["out"], want["out_mass"]) + 2.0 ** -28 * top, "out")
    close(r["final"], want["final"], state_tol(want["final_mass"], longest), "final")
    if len(ck):
        close(r["kept"], want["kept"], state_tol(want["kept_mass"], longest), "kept")


def spread(shape, low, seed):
    """Powers of two between 2^low and 1."""
    return torch.exp2(torch.randint(low, 1, shape, generator=torch.Generator().manual_seed(seed)).float()).to(DEV)


@pytest.mark.parametrize("low", [-12, -25])
@pytest.mark.parametrize("conv", [False, True])
@pytest.mark.parametrize("init", [False, True])
def test_channels_apart(low, conv, init):
    """Channels of one head that differ by up to 2^25: each is held to its own size."""
    y = Layer(4, 2, 64, 64, [70, 1200, 33], seed=51, conv=conv, bias=False, init=init)
    f = spread((4 * 64,), low, 1)
    y.x[:, :256] = (y.x[:, :256].float() * f).bfloat16()
    if init:
        y.init *= f.view(4, 64, 1)
    ck = [20, 70, 70 + 1024, 1303]
    check(y, ck)


@pytest.mark.parametrize("low", [-12, -25])
def test_states_apart(low):
    """The same of the states that enter, beside rows of one size."""
    y = Layer(4, 2, 64, 64, [70, 33], seed=52, conv=False, init=True, a_scale=1e-3)
    y.init *= spread((2, 4, 64, 1), low, 2) * 2.0 ** 12
    y.x[:, :256] *= 2.0 ** -16
    check(y, [20])


@pytest.mark.parametrize("D", [False, True])
@pytest.mark.parametrize("a_scale", [1.0, 50.0])
def test_x_of_tokens_apart(D, a_scale):
    """x of a prompt's first tokens, and of others, 2^-20 to 2^-25 of its channel's largest in a chunk; with
    decays that leave nothing of a token, the next stands alone in the state too."""
    y = Layer(4, 2, 64, 64, [70, 1200, 33], seed=53, conv=False, D=D, a_scale=a_scale, dt_shift=4.0 if a_scale > 1 else 0.0)
    f = spread((1303, 1), -25, 3)
    f[[0, 70, 1270]] = 2.0 ** -25
    f[[69, 1269, 1302]] = 2.0 ** -20
    y.x[:, :256] = (y.x[:, :256].float() * f).bfloat16()
    ck = [20, 70, 70 + 1024, 1303]
    check(y, ck)

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


def floors(y):
    """What fp16's smallest step, whose half is 2^-25, may add to each output.
    - x is an operand times a power of two: 2^11 where the channel's largest |x| in the chunk of 32 tokens is
      2^-8 or more, else the power that brings that largest to 2^14 or more.  2^-25 is 2^-28 of that largest,
      or less: 2^-28 of the sum of absolute terms with each |x| at its chunk's largest.
    - A token's weights are products of C, brought to 2^13 or more by its largest, of B, by the chunk's largest, of
      steps, by the largest that is left of any up to the token, and of 2^-20.  The products round at 2^-25, in units of
      the three largest 2^-25 / 2^(13 + 13 - 20) = 2^-31; the weights at twice that (a step is brought to 1/2 or
      more); C and B at 2^-25 in each of N products with values below 2^14, N 2^-31 / 2^6, 2^-30 each for N = 128.
      Together less than 2^-28, times the sum of the chunk's |x| up to the token.
      Where D is larger it is brought to 2^13 or more instead, 2^-38 of it, times 32 tokens' |x|: 2^-5 of the first."""
    H, G, P, N = y.dims
    A, dt = f64(y.A), y.steps()
    rows, weights = [], np.zeros((int(y.cu[-1]), H, P))
    for s, n in enumerate(y.lens):
        u = f64(y.x[y.cu[s]:y.cu[s + 1]])
        if y.w is not None:
            u = O.conv(u, f64(y.w), f64(y.b), np.zeros((3, y.C)) if y.window is None else f64(y.window)[s])[0]
        u = np.abs(u)
        for c in range(0, n, 32):
            part, at = u[c:c + 32], slice(y.cu[s] + c, min(y.cu[s] + c + 32, y.cu[s + 1]))
            x, b, k = part[:, :H * P].reshape(-1, H, P), part[:, H * P:H * P + G * N].reshape(-1, G, N), part[:, H * P + G * N:].reshape(-1, G, N)
            left = np.abs(dt[at])
            for i in range(1, len(left)):
                left[i] = np.maximum(left[i], left[i - 1] * np.exp(A * dt[y.cu[s] + c + i]))
            weights[at] = np.cumsum(x, 0) * (np.repeat(b.max((0, 2)) * k.max(2), H // G, 1) * left)[:, :, None]
            part[:, :H * P] = part[:, :H * P].max(0)
        rows.append(u)
    D = None if y.D is None else np.abs(f64(y.D))
    return 2.0 ** -28 * (1 + 2.0 ** -5) * O.prefill(H, G, P, N, y.cu, np.concatenate(rows), dt, A, D)["out"] + 2.0 ** -28 * weights


def state_floors(y, ck):
    """The same for states, of final and kept ones: [.., H, P, 1].  Of a chunk's products x w (w: the steps, decayed to
    its end) a channel's largest, each with its token's largest |B|, is brought to 2^4 or more, and each is off by
    2^-25: 2^-28 of that largest with its |B| (2^-29, and a power of two's slack in the |B|), 32 times at most.  B itself, brought
    to 2^13 or more in each token, is off by 2^-38 of that, far less.  Kept states inside a chunk come from the one at its start."""
    H, G, P, N = y.dims
    A, dt, final, kept = f64(y.A), y.steps(), [], []
    for s, n in enumerate(y.lens):
        u = f64(y.x[y.cu[s]:y.cu[s + 1]])
        if y.w is not None:
            u = O.conv(u, f64(y.w), f64(y.b), np.zeros((3, y.C)) if y.window is None else f64(y.window)[s])[0]
        u, F = np.abs(u), np.zeros((H, P, 1))
        for c in range(0, n, 32):
            L = min(32, n - c)
            kept += [F] * sum(int(y.cu[s]) + c < k < int(y.cu[s]) + c + L for k in ck)
            part, d = u[c:c + L], dt[y.cu[s] + c:y.cu[s] + c + L]
            cum = np.cumsum(A * d, 0)
            w = np.abs(d) * np.exp(cum[-1] - cum)
            b = np.repeat(part[:, H * P:H * P + G * N].reshape(L, G, N).max(2), H // G, 1)
            F = np.exp(cum[-1])[:, None, None] * F + 2.0 ** -23 * (part[:, :H * P].reshape(L, H, P) * (w * b)[..., None]).max(0)[..., None]
            kept += [F] * (int(y.cu[s]) + c + L in ck)
        final.append(F)
    return np.array(final), np.array(kept)


def check(y, ck=(), decays=0.0):
    r, want = y.run(ck), y.oracle(ck)
    T, longest = int(y.cu[-1]), max(y.lens)
    final, kept = state_floors(y, ck)
    close(r["out"][:T], want["out"], out_tol(want["out"], want["out_mass"]) + floors(y), "out")
    close(r["final"], want["final"], state_tol(want["final_mass"], longest) + decays * want["final_mass"] + final, "final")
    if len(ck):
        close(r["kept"], want["kept"], state_tol(want["kept_mass"], longest) + decays * want["kept_mass"] + kept, "kept")


def spread(shape, low, seed):
    """Powers of two between 2^low and 1."""
    return torch.exp2(torch.randint(low, 1, shape, generator=torch.Generator().manual_seed(seed)).float()).to(DEV)


@pytest.mark.parametrize("low", [-12, -25])
@pytest.mark.parametrize("conv", [False, True])
@pytest.mark.parametrize("init", [False, True])
def test_channels_apart(low, conv, init):
    """Channels of one head that differ by up to 2^25: each is held to its own size."""
    y = Layer(4, 2, 64, 64, [70, 1400, 33], seed=51, conv=conv, bias=False, init=init)
    f = spread((4 * 64,), low, 1)
    y.x[:, :256] = (y.x[:, :256].float() * f).bfloat16()
    if init:
        y.init *= f.view(4, 64, 1)
    ck = [20, 70, 70 + 1024, 1503]
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
    y = Layer(4, 2, 64, 64, [70, 1400, 33], seed=53, conv=False, D=D, a_scale=a_scale, dt_shift=4.0 if a_scale > 1 else 0.0)
    f = spread((1503, 1), -25, 3)
    f[[0, 70, 1470]] = 2.0 ** -25
    f[[69, 1469, 1502]] = 2.0 ** -20
    y.x[:, :256] = (y.x[:, :256].float() * f).bfloat16()
    ck = [20, 70, 70 + 1024, 1503]
    check(y, ck)


@pytest.mark.parametrize("low", [-17, -20, -40])
@pytest.mark.parametrize("a_scale", [1.0, 50.0])
@pytest.mark.parametrize("what", ["B and C", "C"])
def test_b_and_c_of_tokens_apart(low, a_scale, what):
    """Tokens whose B and C, or C alone, are far below those of others in the chunk: a prompt's first, whose
    output is nothing but their product, and, with decays that leave nothing, any."""
    y = Layer(4, 2, 64, 64, [70, 1400, 33], seed=54, conv=False, D=False, a_scale=a_scale, dt_shift=4.0 if a_scale > 1 else 0.0)
    f = spread((1503, 1), low, 4)
    f[[0, 70, 1470, 69, 1502]] = 2.0 ** low
    at = 384 if what == "C" else 256
    y.x[:, at:] = (y.x[:, at:].float() * f).bfloat16()
    ck = [20, 70, 70 + 1024, 1503]
    check(y, ck)


@pytest.mark.parametrize("lens", [[32], [20, 39, 32]], ids=str)
@pytest.mark.parametrize("D", [False, True])
def test_growth(lens, D):
    """States that grow by 2^100 in a chunk.  The running sums of the exponents, below 128, round at 2^-18 in each of five
    additions, and each exponent at 2^-22 in two products: 2^-15 of a decay, ln 2 counted."""
    y = Layer(2, 1, 64, 64, lens, seed=55, conv=False, D=D, softplus=False, dt_bias=False, x_scale=2.0 ** -8)
    y.dt[:] = 0.75
    y.A[:] = 2.9
    check(y, [10, sum(lens)], decays=2.0 ** -15)


@pytest.mark.parametrize("low", [-20, -40])
def test_steps_apart(low):
    """Steps of a prompt's first tokens far below those of the others: their outputs are products with them alone."""
    y = Layer(4, 2, 64, 64, [70, 1400, 33], seed=56, conv=False, D=False, softplus=False, dt_bias=False, dt_f32=True)
    f = spread((1503, 1), low, 5)
    f[[0, 1, 2, 70, 71, 1470]] = 2.0 ** low
    y.dt = y.dt * f
    ck = [20, 70, 70 + 1024, 1503]
    check(y, ck)


@pytest.mark.parametrize("power", [110, 100, -100])
@pytest.mark.parametrize("conv", [False, True])
@pytest.mark.parametrize("what", ["x", "B", "C"])
def test_ends_of_the_range(power, conv, what):
    """x, B or C of about 2^110, beside others that keep products and outputs in fp32; and of 2^-100."""
    y = Layer(2, 1, 64, 64, [70, 33], seed=57, conv=conv, bias=False, D=False)
    parts = dict(x=slice(0, 128), B=slice(128, 192), C=slice(192, 256))
    f = 2.0 ** (power - 2)
    y.x[:, parts[what]] = (y.x[:, parts[what]].float() * f).bfloat16()
    if what == "C" and power > 0:
        y.x[:, parts["B"]] = (y.x[:, parts["B"]].float() * 2.0 ** -20).bfloat16()
    check(y, [20, 103])


@pytest.mark.parametrize("power", [110, -100])
def test_large_and_small_states(power):
    """States that enter at 2^110 and 2^-100."""
    y = Layer(2, 1, 64, 64, [70, 33], seed=58, conv=False, init=True, D=False)
    y.init *= 2.0 ** power
    y.x[:, :128] = (y.x[:, :128].float() * 2.0 ** (power if power < 0 else 0)).bfloat16()
    check(y, [20, 103])


@pytest.mark.parametrize("n", [5, 31, 33, 60, 1100])
def test_rows_that_do_not_exist(n):
    """Inputs that cancel in every token's convolution, but would not in tokens behind the last: those play no part."""
    y = Layer(2, 1, 64, 64, [n, 40], seed=59, bias=False, D=False)
    sign = 1.0 - 2.0 * (torch.arange(n + 40, device=DEV)[:, None] % 2).float()
    y.x[:, 3:100:7] = (sign * 2.0 ** 115).bfloat16()
    y.w[3:100:7] = 1.0
    r, want = y.run(), y.oracle()
    # the sums are exact, so what an output holds is its own largest products
    close(r["out"][:n + 40], want["out"], out_tol(want["out"], want["out_mass"]), "out")
    close(r["final"], want["final"], state_tol(want["final_mass"], n), "final")

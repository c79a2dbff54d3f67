"""The packed scan of state space layers against the fp64 oracle."""
import numpy as np
import pytest
import torch

import gated_deltanet_prefill_varlen_amd as gdn
from tests.ssm_util import DEV, Layer, close, f64, out_tol, state_tol

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("P", [32, 64, 128])
@pytest.mark.parametrize("N", [32, 64, 128])
@pytest.mark.parametrize("H,G", [(1, 1), (4, 2), (3, 1)])
def test_geometry(H, G, P, N):
    y = Layer(H, G, P, N, [70, 0, 1, 129], seed=P + N + H, init=True, window=True)
    ck = [64, 70, 71, 99, 199]
    y.check(y.run(ck), y.oracle(ck), ck)


@pytest.mark.parametrize("lens", [[1], [2], [3], [4], [16], [63], [64], [65], [127, 128, 129], [0], [0, 5, 0, 0, 64, 0], [300, 17, 1, 700]])
def test_lengths(lens):
    y = Layer(4, 1, 64, 64, lens, seed=len(lens) + lens[0], init=True, window=True)
    y.check(y.run(), y.oracle())


@pytest.mark.parametrize("H,P,N,n", [(1, 32, 32, 2100), (2, 64, 64, 1500), (1, 128, 64, 1025), (4, 32, 128, 3000)])
def test_long(H, P, N, n):
    """Prompts that several workgroups share, beside short ones."""
    y = Layer(H, 1, P, N, [40, n, 1023, 0, n - 7], seed=n, init=True, window=True)
    ck = [40, 41, 40 + 512, 40 + n - 1, 40 + n, 40 + n + 1000]
    y.check(y.run(ck), y.oracle(ck), ck)


@pytest.mark.parametrize("kw", [dict(conv=False), dict(bias=False), dict(D=False), dict(dt_bias=False), dict(softplus=False, dt_bias=False),
                                dict(dt_f32=True), dict(init=True), dict(window=True), dict(pad=24), dict(init=True, conv=False, D=False)],
                         ids=str)
def test_options(kw):
    y = Layer(6, 3, 64, 32, [130, 33], seed=5, **kw)
    ck = [7, 64, 130, 131]
    y.check(y.run(ck), y.oracle(ck), ck)


@pytest.mark.parametrize("kw", [dict(a_scale=0.0), dict(a_scale=-0.01), dict(a_scale=50.0, dt_shift=4.0), dict(a_scale=1e-4),
                                dict(x_scale=2.0 ** 40, conv=False, D=False), dict(x_scale=2.0 ** -40, conv=False, init=True),
                                dict(x_scale=2.0 ** 20), dict(x_scale=2.0 ** -20), dict(dt_shift=-12.0)], ids=str)
def test_ranges(kw):
    """No decay, growth, decays that leave nothing, large and tiny values and steps."""
    y = Layer(3, 1, 64, 128, [200, 30], seed=9, **kw)
    ck = [50, 128]
    y.check(y.run(ck), y.oracle(ck), ck)


def test_step_clamp():
    y = Layer(2, 1, 32, 32, [100], seed=3)
    y.shape = gdn.make_ssm(2, 1, 32, 32, dt_min=0.01, dt_max=0.05)
    keep = y.steps
    y.steps = lambda: np.clip(keep(), np.float32(0.01), np.float32(0.05)).astype(np.float64)
    y.check(y.run(), y.oracle())


def test_alone_as_packed():
    """A prompt's bits do not depend on the pack."""
    y = Layer(4, 2, 64, 128, [90, 1300, 64, 2, 300], seed=21, init=True, window=True)
    ck = [70, 90 + 640, 90 + 1300]
    r = y.run(ck)
    at = 0
    for s, n in enumerate(y.lens):
        one = y.run(ck, only=s)
        a = int(y.cu[s])
        k = one["kept"].shape[0]
        assert torch.equal(one["out"][:n], r["out"][a:a + n]) and torch.equal(one["final"][0], r["final"][s])
        assert torch.equal(one["kept"], r["kept"][at:at + k]) and torch.equal(one["window"][0], r["window"][s])
        at += k


def test_checkpoints_change_nothing():
    y = Layer(4, 1, 64, 64, [500, 1500], seed=22)
    a, b = y.run(), y.run([3, 64, 65, 499, 501, 1999, 2000])
    assert torch.equal(a["out"], b["out"]) and torch.equal(a["final"], b["final"])


def test_resumed():
    """A prompt continued from a checkpoint and its window."""
    y = Layer(2, 1, 64, 64, [300], seed=23)
    r, want = y.run([133]), y.oracle()
    z = Layer(2, 1, 64, 64, [300], seed=23)
    z.lens, z.cu, z.x, z.dt = [167], np.array([0, 167], np.int32), y.x[133:], y.dt[133:]
    z.init, z.window = r["kept"], r["window_kept"]
    q = z.run()
    close(q["out"][:167], want["out"][133:], out_tol(want["out"][133:], want["out_mass"][133:]), "out")
    close(q["final"], want["final"], 2 * state_tol(want["final_mass"], 300), "final")
    assert torch.equal(q["window"], r["window"])


def test_window_in_place():
    y = Layer(2, 2, 32, 32, [5, 1, 0, 2, 200], seed=24, window=True)
    a, b = y.run(), y.run(window_out="in place")
    for k in a:
        assert a[k] is None or torch.equal(a[k], b[k]), k


@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
def test_not_finite(value):
    """A value that is not finite, in x, leaves earlier tokens, other channels and other prompts as they were."""
    y = Layer(2, 1, 64, 64, [100, 150, 80], seed=25, conv=False)
    ck = [100 + 70, 100 + 100]
    a = y.run(ck)
    t, p = 100 + 75, 37
    y.x = y.x.clone()
    y.x[t, p] = value
    b = y.run(ck)
    same = torch.ones_like(a["out"], dtype=torch.bool)
    same[t:250, 0, p] = False
    assert torch.equal(a["out"][same], b["out"][same])
    assert not bool(b["out"][t:250, 0, p].isfinite().any())
    keep = torch.ones_like(a["final"], dtype=torch.bool)
    keep[1, 0, p] = False
    assert torch.equal(a["final"][keep], b["final"][keep]) and not bool(b["final"][1, 0, p].isfinite().any())
    assert torch.equal(a["kept"][0], b["kept"][0])
    assert not bool(b["kept"][1, 0, p].isfinite().any()) and torch.equal(a["kept"][1, 1], b["kept"][1, 1])


@pytest.mark.parametrize("what", ["B", "C", "dt"])
def test_not_finite_columns(what):
    y = Layer(2, 1, 64, 64, [100, 150, 80], seed=26, conv=False)
    ck = [100 + 70]
    a = y.run(ck)
    t = 100 + 75
    y.x, y.dt = y.x.clone(), y.dt.clone()
    if what == "dt":
        y.dt[t, 0] = float("nan")
    else:
        y.x[t, 128 + (64 if what == "C" else 0) + 5] = float("nan")
    b = y.run(ck)
    assert torch.equal(a["out"][:t], b["out"][:t]) and torch.equal(a["out"][250:330], b["out"][250:330])
    assert torch.equal(a["kept"], b["kept"])
    assert bool(b["out"][t, 0].isnan().all())
    if what == "C":
        assert torch.equal(a["out"][t + 1:], b["out"][t + 1:]) and torch.equal(a["final"], b["final"])
    elif what == "dt":
        assert torch.equal(a["out"][:, 1], b["out"][:, 1]) and bool(b["out"][t:250, 0].isnan().all())


def test_many_prompts():
    rng = np.random.default_rng(4)
    y = Layer(2, 1, 32, 64, rng.integers(0, 90, 150).tolist(), seed=27, init=True, window=True)
    ck = [int(c) for c in sorted(rng.choice(np.arange(1, y.cu[-1] + 1), 40, replace=False))]
    y.check(y.run(ck), y.oracle(ck), ck)


def test_only_outputs_asked_for():
    """No final state, no windows."""
    y = Layer(2, 1, 64, 64, [77], seed=28)
    r = y.run()
    out = torch.zeros_like(r["out"])
    gdn.gdn_ssm_prefill_packed(y.shape, torch.from_numpy(y.cu).to(DEV), y.cu, y.x, y.dt, y.A, out, dt_bias=y.dt_bias, D=y.D,
                               conv_weight=y.w, conv_bias=y.b, workspace=y.workspace)
    assert torch.equal(out[:77], r["out"][:77])


def test_streams_and_graph():
    """Two packs on two streams at once; a captured call replayed on new rows."""
    a = Layer(4, 1, 64, 128, [1200, 50], seed=29, init=True, window=True)
    b = Layer(4, 1, 64, 128, [60, 1100], seed=30, init=True, window=True)
    ra, rb = a.run([100]), b.run([100])
    torch.cuda.synchronize()
    s = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for _ in range(3):
        for y, st in zip((a, b), s):
            with torch.cuda.stream(st):
                got.append(y.run([100]))
    torch.cuda.synchronize()
    for i, r in enumerate(got):
        for k in r:
            assert torch.equal(r[k], (ra, rb)[i % 2][k]), k
    out, final = torch.zeros_like(ra["out"]), torch.zeros_like(ra["final"])
    x, dt, cu = a.x.clone(), a.dt.clone(), torch.from_numpy(a.cu).to(DEV)
    ws = torch.empty_like(a.workspace)
    call = lambda: gdn.gdn_ssm_prefill_packed(a.shape, cu, a.cu, x, dt, a.A, out, dt_bias=a.dt_bias, D=a.D, init_state=a.init,
                                              final_state=final, conv_weight=a.w, conv_bias=a.b, conv_state_in=a.window, workspace=ws)
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for k in range(4):
        x.copy_(a.x.float() * (1 + 0.25 * k))
        g.replay()
        torch.cuda.synchronize()
        o, f = out.clone(), final.clone()
        out.zero_(), final.zero_()
        call()
        torch.cuda.synchronize()
        assert torch.equal(o, out) and torch.equal(f, final)


@pytest.mark.parametrize("lens", [[5000, 60, 0, 3000], [40, 7]], ids=str)
def test_states_in_place(lens):
    """final_state may be init_state, where a prompt is cut into segments too."""
    y = Layer(4, 2, 64, 64, lens, seed=31, init=True, window=True)
    want = y.run()
    for _ in range(3):
        state = y.init.clone()
        out = torch.empty_like(want["out"])
        i32 = torch.from_numpy(y.cu).to(DEV)
        gdn.gdn_ssm_prefill_packed(y.shape, i32, y.cu, y.x, y.dt, y.A, out, dt_bias=y.dt_bias, D=y.D, init_state=state, final_state=state,
                                   conv_weight=y.w, conv_bias=y.b, conv_state_in=y.window, workspace=y.workspace)
        T = int(y.cu[-1])
        assert torch.equal(out[:T], want["out"][:T]) and torch.equal(state, want["final"])


def test_windows_and_states_in_place_with_checkpoints():
    """Checkpoints one and two tokens into a prompt, between chunks' ends and on
    them, with the windows and states written over the ones read."""
    lens = [70, 1, 2, 300, 33]
    y = Layer(4, 1, 32, 64, lens, seed=32, init=True, window=True)
    ck = [1, 2, 32, 35, 70, 71, 72, 73, 74, 75, 105, 373, 374, 406]
    want, whole = y.oracle(ck), y.run(ck)
    y.check(whole, want, ck)
    again = y.run(ck, window_out="in place")
    assert all(torch.equal(whole[k], again[k]) for k in ("out", "final", "kept", "window", "window_kept"))
    assert torch.equal(y.run()["window"], y.run(window_out="in place")["window"])

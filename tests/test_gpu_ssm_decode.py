"""The decode step of state space layers against the fp64 oracle."""
import numpy as np
import pytest
import torch

import gated_deltanet_prefill_varlen_amd as gdn
from oracle import ssm_oracle as O
from tests.ssm_util import DEV, Layer, close, f64, out_tol, state_tol

pytestmark = pytest.mark.gpu


def step(y, n_tok, slots, pool, state, window, snap=True, stream=None):
    H, G, P, N = y.dims
    B = len(slots)
    out = torch.full((B * n_tok, H, P), 7.0, dtype=torch.bfloat16, device=DEV)
    snaps = torch.full((B, n_tok, H, P, N), float("nan"), device=DEV) if snap else None
    sl = np.asarray(slots, np.int32)
    gdn.gdn_ssm_decode(y.shape, n_tok, y.x, y.dt, y.A, state, out, dt_bias=y.dt_bias, D=y.D, conv_weight=y.w, conv_bias=y.b,
                       conv_state=window, slot=torch.from_numpy(sl).to(DEV), slot_host=sl, snapshots=snaps, stream=stream)
    return out, snaps


def pools(y, pool, seed):
    H, G, P, N = y.dims
    g = torch.Generator().manual_seed(seed)
    state = (0.5 * torch.randn(pool, H, P, N, generator=g)).to(DEV)
    window = torch.randn(pool, 3, y.C, generator=g).bfloat16().to(DEV) if y.w is not None else None
    return state, window


def check(y, n_tok, slots, pool, seed, snap=True):
    H, G, P, N = y.dims
    state, window = pools(y, pool, seed)
    s0, w0 = state.clone(), None if window is None else window.clone()
    out, snaps = step(y, n_tok, slots, pool, state, window, snap)
    B = len(slots)
    cu = np.arange(B + 1) * n_tok
    want = O.prefill(H, G, P, N, cu, f64(y.x), y.steps(), f64(y.A), f64(y.D), f64(y.w), f64(y.b),
                     None if w0 is None else f64(w0)[slots], f64(s0)[slots], set(range(1, B * n_tok + 1)))
    close(out, want["out"], out_tol(want["out"], want["out_mass"]), "out")
    close(state[slots], want["final"], state_tol(want["final_mass"], n_tok), "state")
    if snap:
        close(snaps.reshape(-1, H, P, N), want["kept"], state_tol(want["kept_mass"], n_tok), "snapshots")
    rest = [i for i in range(pool) if i not in slots]
    assert torch.equal(state[rest], s0[rest])
    if window is not None:
        assert np.array_equal(f64(window)[slots], want["window"]) and torch.equal(window[rest], w0[rest])


@pytest.mark.parametrize("P", [32, 64, 128])
@pytest.mark.parametrize("N", [32, 64, 128])
@pytest.mark.parametrize("H,G", [(1, 1), (6, 2), (3, 1), (8, 1)])
def test_geometry(H, G, P, N):
    check(Layer(H, G, P, N, [4], seed=P + N), 1, [5, 0, 3, 1], 7, 1)


@pytest.mark.parametrize("n_tok", [1, 2, 3, 4, 7])
@pytest.mark.parametrize("conv", [True, False])
@pytest.mark.parametrize("snap", [True, False])
def test_tokens(n_tok, conv, snap):
    check(Layer(4, 2, 64, 64, [3 * n_tok], seed=n_tok, conv=conv), n_tok, [2, 4, 0], 5, 2, snap)


@pytest.mark.parametrize("kw", [dict(bias=False), dict(D=False), dict(dt_bias=False), dict(softplus=False, dt_bias=False), dict(dt_f32=True),
                                dict(pad=16), dict(a_scale=0.0), dict(a_scale=50.0, dt_shift=4.0), dict(x_scale=2.0 ** 30, conv=False)], ids=str)
def test_options(kw):
    check(Layer(2, 1, 64, 128, [6], seed=8, **kw), 2, [0, 2, 1], 3, 3)


@pytest.mark.parametrize("B", [1, 33, 200])
def test_batches(B):
    slots = np.random.default_rng(B).permutation(B + 5)[:B].tolist()
    check(Layer(2, 1, 32, 32, [B], seed=B), 1, slots, B + 5, 4)


def test_without_slots():
    y = Layer(4, 1, 64, 64, [3], seed=1)
    s1, w1 = pools(y, 4, 5)
    s2, w2 = s1.clone(), w1.clone()
    a, _ = step(y, 1, [0, 1, 2], 4, s1, w1, False)
    b = torch.empty_like(a)
    gdn.gdn_ssm_decode(y.shape, 1, y.x, y.dt, y.A, s2, b, dt_bias=y.dt_bias, D=y.D, conv_weight=y.w, conv_bias=y.b, conv_state=w2)
    assert torch.equal(a, b) and torch.equal(s1, s2) and torch.equal(w1, w2)


def test_tokens_at_once_as_one_by_one():
    y = Layer(4, 1, 64, 128, [8], seed=11)
    s1, w1 = pools(y, 3, 6)
    s2, w2 = s1.clone(), w1.clone()
    a, snaps = step(y, 4, [2, 0], 3, s1, w1)
    x, dt = y.x.clone(), y.dt.clone()
    for i in range(4):
        y.x, y.dt = x[i::4], dt[i::4]
        b, _ = step(y, 1, [2, 0], 3, s2, w2, False)
        assert torch.equal(b, a[i::4]) and torch.equal(s2[[2, 0]], snaps[:, i])
    assert torch.equal(s1, s2) and torch.equal(w1, w2)


def test_not_finite_stays():
    """A sequence's values that are not finite reach no other sequence, head or channel."""
    y = Layer(2, 1, 64, 64, [3], seed=12, conv=False)
    s1, _ = pools(y, 3, 7)
    s2 = s1.clone()
    a, _ = step(y, 1, [0, 1, 2], 3, s1, None, False)
    s2[1, 0, 9, 3] = float("nan")
    b, _ = step(y, 1, [0, 1, 2], 3, s2, None, False)
    bad = torch.zeros_like(a, dtype=torch.bool)
    bad[1, 0, 9] = True
    assert torch.equal(a[~bad], b[~bad]) and bool(b[bad].isnan().all())
    keep = torch.ones_like(s1, dtype=torch.bool)
    keep[1, 0, 9, 3] = False
    assert torch.equal(s1[keep], s2[keep])


def test_prefill_then_decode_then_norm():
    """A layer as a program runs it: the norm, the scan of the prompts into the pool, decode steps captured in a graph, the
    gated norm with codes; against one scan over all tokens."""
    H, G, P, N = 8, 1, 64, 128
    lens, more = [37, 130], 5
    full = Layer(H, G, P, N, [n + more for n in lens], seed=13)
    want = full.oracle()
    pool = 4
    state = torch.full((pool, H, P, N), float("nan"), device=DEV)
    window = torch.zeros(pool, 3, full.C, dtype=torch.bfloat16, device=DEV)
    y = Layer(H, G, P, N, lens, seed=13)
    rows = lambda t: torch.cat([t[int(full.cu[s]):int(full.cu[s]) + lens[s]] for s in range(2)])
    y.x, y.dt = rows(full.x), rows(full.dt)
    for k in ("A", "dt_bias", "D", "w", "b"):
        setattr(y, k, getattr(full, k))
    r = y.run()
    slots = [3, 1]
    state[slots], window[slots] = r["final"], r["window"]
    sl = np.array(slots, np.int32)
    dsl = torch.from_numpy(sl).to(DEV)
    pick = lambda t, i: torch.stack([t[int(full.cu[s]) + lens[s] + i] for s in range(2)])
    x, dt = pick(full.x, 0), pick(full.dt, 0)
    out = torch.zeros(2, H, P, dtype=torch.bfloat16, device=DEV)
    z = torch.randn(2, H * P, device=DEV).bfloat16()
    w = torch.rand(H * P, device=DEV)
    norm = gdn.make_norm(H * P, groups=H, gate_first=True)
    codes, scales = torch.zeros(2, H * P, dtype=torch.float8_e4m3fn, device=DEV), torch.zeros(2, 1, device=DEV)

    def one():
        gdn.gdn_ssm_decode(y.shape, 1, x, dt, full.A, state, out, dt_bias=full.dt_bias, D=full.D, conv_weight=full.w, conv_bias=full.b,
                           conv_state=window, slot=dsl, slot_host=sl)
        gdn.gdn_rms_norm(norm, out.view(2, H * P), w, gate=z, codes=codes, scales=scales)

    keep = state.clone(), window.clone()
    one()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        one()
    state.copy_(keep[0]), window.copy_(keep[1])
    for i in range(more):
        x.copy_(pick(full.x, i)), dt.copy_(pick(full.dt, i))
        g.replay()
        torch.cuda.synchronize()
        at = [int(full.cu[s]) + lens[s] + i for s in range(2)]
        close(out, want["out"][at], out_tol(want["out"][at], want["out_mass"][at]), "out")
        normed, _ = O.rms_norm(f64(out).reshape(2, -1), f64(w), gate=f64(z), gate_first=True, groups=H)
        got = f64(codes) * f64(scales)
        assert np.all(np.abs(got - normed) <= (2.0 ** -4 + 2.0 ** -18) * np.abs(normed) + 2.0 ** -10 * f64(scales))
    close(state[slots], want["final"], 2 * state_tol(want["final_mass"], 200), "state")
    assert np.array_equal(f64(window)[slots], want["window"])


def test_states_past_the_last_cache_as_within_it():
    """More states than the last cache holds: the same bits as in parts."""
    H, G, P, N, B = 64, 4, 64, 128, 130
    y = Layer(H, G, P, N, [B], seed=21)
    state, window = pools(y, B + 2, 9)
    slots = np.random.default_rng(3).permutation(B + 2)[:B].tolist()
    s2, w2 = state.clone(), window.clone()
    a, _ = step(y, 1, slots, B + 2, state, window, False)
    x, dt = y.x, y.dt
    for i in range(0, B, 50):
        y.x, y.dt = x[i:i + 50], dt[i:i + 50]
        b, _ = step(y, 1, slots[i:i + 50], B + 2, s2, w2, False)
        assert torch.equal(b, a[i:i + 50])
    assert torch.equal(state, s2) and torch.equal(window, w2)

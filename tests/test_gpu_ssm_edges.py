"""State space layers and the norm at the edges of what their calls allow: rows,
slots and strides past 32 bits, growing states, packs of nothing, captured
calls, and a layer's step as a model would run it."""
import numpy as np
import pytest
import torch

import gated_deltanet_prefill_varlen_amd as gdn
from tests.ssm_util import DEV, Layer

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("conv", [True, False])
def test_growing_states(conv):
    """A above 0: states that grow by up to e^2 in a chunk of 32 tokens.  Bounds as elsewhere."""
    y = Layer(4, 2, 64, 64, [300, 33, 64], seed=41, conv=conv, init=True, a_scale=-0.04)
    assert bool((y.A > 0).all())
    ck = [40, 64, 300, 333]
    y.check(y.run(ck), y.oracle(ck), ck)


def test_packs_of_nothing():
    y = Layer(2, 1, 32, 64, [0, 0], seed=42, init=True, window=True)
    r = y.run()
    assert torch.equal(r["final"], y.init) and torch.equal(r["window"], y.window) and bool((r["out"] == 7.0).all())
    z = Layer(2, 1, 32, 64, [0], seed=42)
    r = z.run()
    assert not r["final"].any() and not r["window"].any()


def test_rows_past_32_bits():
    """Rows 2 MB apart: the last lie past 4 GB."""
    T, stride = 2200, 1 << 20
    y = Layer(2, 1, 32, 32, [T - 40, 40], seed=43, window=True)
    want = y.run([5, 2048, 2190])
    wide = torch.empty(T, stride, dtype=torch.bfloat16, device=DEV)
    wide[:, 64:64 + y.C] = y.x
    wide[:, 512:512 + 2] = y.dt
    y.x, y.dt = wide[:, 64:64 + y.C], wide[:, 512:512 + 2]
    got = y.run([5, 2048, 2190])
    assert all(torch.equal(want[k], got[k]) for k in ("out", "final", "kept", "window", "window_kept"))


def test_slots_past_32_bits():
    H, G, P, N, pool, B = 64, 1, 64, 128, 2100, 3
    y = Layer(H, G, P, N, [B], seed=44)
    s0, w0 = torch.randn(B, H, P, N, device=DEV), torch.randn(B, 3, y.C, device=DEV).bfloat16()
    state = torch.empty(pool, H, P, N, device=DEV)
    window = torch.zeros(pool, 3, y.C, dtype=torch.bfloat16, device=DEV)
    slots = np.array([2099, 0, 2060], np.int32)
    at = torch.from_numpy(slots).to(DEV)
    state[at.long()], window[at.long()] = s0, w0
    outs = []
    for st, wi, sl in ((state, window, slots), (s0, w0, None)):
        o = torch.empty(B, H, P, dtype=torch.bfloat16, device=DEV)
        gdn.gdn_ssm_decode(y.shape, 1, y.x, y.dt, y.A, st, o, dt_bias=y.dt_bias, D=y.D, conv_weight=y.w, conv_bias=y.b, conv_state=wi,
                           slot=None if sl is None else at, slot_host=sl)
        outs.append(o)
    assert torch.equal(outs[0], outs[1]) and torch.equal(state[at.long()], s0) and torch.equal(window[at.long()], w0)


def test_norm_rows_past_32_bits():
    rows, dim, stride = 2200, 1000, 1 << 20
    x, r, z = (torch.randn(rows, dim, device=DEV).bfloat16() for _ in range(3))
    w = torch.randn(dim, device=DEV)
    shape = gdn.make_norm(dim)

    def run(x, r, ro, z):
        out = torch.empty(rows, dim, dtype=torch.bfloat16, device=DEV)
        codes, scales = torch.empty(rows, dim, dtype=torch.int8, device=DEV), torch.empty(rows, 1, device=DEV)
        gdn.gdn_rms_norm(shape, x, w, out=out, residual=r, residual_out=ro, gate=z, codes=codes, scales=scales)
        return out, ro, codes, scales

    want = run(x, r, torch.empty_like(r), z)
    wide, stream = (torch.empty(rows, stride, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    cols = [wide[:, 3:3 + dim], stream[:, 2049:2049 + dim], wide[:, 4096:4096 + dim]]
    for c, v in zip(cols, (x, r, z)):
        c.copy_(v)
    got = run(cols[0], cols[1], cols[1], cols[2])
    assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_step_as_captured():
    """A layer's step between its norms, captured once and replayed on new rows,
    with eager calls in between; every replay against the eager result."""
    H, G, P, N, B, hidden = 8, 2, 64, 64, 5, 640
    y = Layer(H, G, P, N, [B], seed=45)
    g = torch.Generator().manual_seed(46)
    rnd = lambda *s: torch.randn(*s, generator=g).to(DEV)
    proj_in, proj_out = (rnd(hidden, y.C + H * P + 8) / 25).bfloat16(), (rnd(H * P, hidden) / 23).bfloat16()
    w1, w2 = 1 + 0.1 * rnd(hidden), 1 + 0.1 * rnd(H * P)
    first, last = gdn.make_norm(hidden), gdn.make_norm(H * P, groups=G, gate_first=True)
    slots = np.array([4, 1, 6, 0, 2], np.int32)
    slot = torch.from_numpy(slots).to(DEV)
    x, res = torch.empty(B, hidden, dtype=torch.bfloat16, device=DEV), torch.empty(B, hidden, device=DEV)
    state, window = torch.empty(7, H, P, N, device=DEV), torch.empty(7, 3, y.C, dtype=torch.bfloat16, device=DEV)
    codes, scales = torch.empty(B, H * P, dtype=torch.float8_e4m3fn, device=DEV), torch.empty(B, 1, device=DEV)

    def layer():
        h = torch.empty_like(x)
        gdn.gdn_rms_norm(first, x, w1, out=h, residual=res, residual_out=res)
        row = h @ proj_in
        z, xbc, dt = row[:, :H * P], row[:, H * P:H * P + y.C], row[:, H * P + y.C:]
        o = torch.empty(B, H, P, dtype=torch.bfloat16, device=DEV)
        gdn.gdn_ssm_decode(y.shape, 1, xbc, dt, y.A, state, o, dt_bias=y.dt_bias, D=y.D, conv_weight=y.w, conv_bias=y.b, conv_state=window,
                           slot=slot, slot_host=slots)
        n = torch.empty(B, H * P, dtype=torch.bfloat16, device=DEV)
        gdn.gdn_rms_norm(last, o.view(B, H * P), w2, out=n, gate=z, codes=codes, scales=scales)
        return n @ proj_out

    def fill(i):
        q = torch.Generator().manual_seed(100 + i)
        for t in (x, res, state, window):
            t.copy_(torch.randn(t.shape, generator=q))

    def result(y0):
        return [t.clone() for t in (y0, res, state, window, codes.view(torch.uint8), scales)]

    side = torch.cuda.Stream()
    fill(0)
    with torch.cuda.stream(side):
        layer()
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            y0 = layer()
    for i in range(4):
        fill(i)
        want = result(layer())
        fill(i)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, result(y0))), i

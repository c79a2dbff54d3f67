"""Rotary positions at the edges of their inputs: channels that are infinite,
and angles of every size that the call takes."""
import numpy as np
import pytest
import torch

import gated_deltanet_prefill_varlen_amd as gdn
from cache_util import DEV, DevCache, bf, f64, i32, i64, slots_of
from oracle import cache_oracle as C

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("adjacent", [False, True])
@pytest.mark.parametrize("code", ["e4m3", "int8"])
@pytest.mark.parametrize("d,rot", [(64, 64), (128, 32), (256, 128)])
def test_infinite_channels_turn_as_the_formula_says(d, rot, code, adjacent):
    """(a c - b s, a s + b c) with one of a, b infinite is infinite, not NaN: a
    key is stored as its largest code.  At position 0 the formula has 0 x
    infinity, and NaN comes out."""
    rng = np.random.default_rng(d + rot)
    T, hkv, page = 40, 2, 16
    freq = [float(np.float32(10000.0 ** (-2 * i / rot))) for i in range(rot // 2)]
    rope = gdn.make_rope(freq, adjacent=adjacent)
    q, k = rng.standard_normal((2, T, hkv, d))
    for x in (q, k):
        x[3, 0, 1], x[4, 1, rot - 1], x[5, 0, rot // 2] = np.inf, -np.inf, np.inf
        x[6, 0, 2], x[6, 0, 3], x[6, 0, rot // 2 + 2] = np.inf, -np.inf, -np.inf
        x[0, 0, 0], x[7, 1, d - 1], x[8, 0, 4] = np.inf, -np.inf, np.nan
    q, k = bf(q).to(DEV), bf(k).to(DEV)
    v = torch.zeros_like(k)
    pos, table = np.arange(T, dtype=np.int32), np.array([[2, 0, 1]])
    dev, out = DevCache(3, hkv, page, d, code), torch.empty_like(q)
    slots = slots_of(table, page, 0, 0, T)
    gdn.gdn_rope_append(rope, dev.handle, i32([0, T]), [0, T], q, k, v, i32(pos), i64(slots), out)
    with np.errstate(invalid="ignore"):
        want = C.rotate(f64(q), pos[None], freq, [0] * len(freq), adjacent)
        k_rot = C.round_bf16(C.rotate(f64(k), pos[None], freq, [0] * len(freq), adjacent))
    got, num = f64(out), np.isfinite(want)
    np.testing.assert_array_equal(np.isnan(got), np.isnan(want))
    np.testing.assert_array_equal(got[np.isinf(want)], want[np.isinf(want)])
    assert np.isinf(want).sum() > 10 and np.isnan(want).sum() >= 4
    # fp32: two products and a sum of cos and sin off by 2^-22, then bf16
    assert np.all(np.abs(got[num] - want[num]) <= 2.0 ** -8 * np.abs(want[num]) + 2.0 ** -20 * 2 * np.abs(f64(q))[np.isfinite(f64(q))].max())
    kc, _, ks, _ = dev.codes()
    for t, s in enumerate(slots):
        x, y = kc[s // page, :, s % page], k_rot[t]
        np.testing.assert_array_equal(np.isnan(x), np.isnan(y) if code == "e4m3" else np.zeros_like(x, bool))
        inf = np.isinf(y)
        np.testing.assert_array_equal(x[inf], np.copysign(C.TOP[code], y[inf]))
        assert np.all(x[np.isnan(y)] == 0) or code == "e4m3"


@pytest.mark.parametrize("top", [1.0, 300.0, 65536.0])
def test_angles_of_every_size(top):
    """Frequencies up to the largest that the call takes at positions up to
    2^31, negative ones too: the rotation by the angle itself, in 80 bits (the
    products of 24 and 31 bits are exact there).  Error: the bf16
    result by 2^-8 of itself; 2^-20 of the pair covers cos and sin (2^-24) and the
    fp32 work."""
    if np.finfo(np.longdouble).nmant < 63:
        pytest.skip("no 80-bit numbers here")
    rng = np.random.default_rng(int(top))
    d, T = 128, 64
    freq = [float(np.float32(top * x)) for x in np.concatenate([[1.0, -1.0], rng.uniform(0.3, 1.0, 62)])]
    pos = np.concatenate([[0, 1, -1, 2 ** 31 - 1, -2 ** 31], rng.integers(-2 ** 31, 2 ** 31, T - 5)]).astype(np.int32)
    x = bf(rng.standard_normal((T, 4, d))).to(DEV)
    kv, out = torch.zeros(T, 1, d, dtype=torch.bfloat16, device=DEV), torch.empty_like(x)
    dev = DevCache(1, 1, 16, d, "int8")
    gdn.gdn_rope_append(gdn.make_rope(freq), dev.handle, i32([0, T]), [0, T], x, kv, kv, i32(pos), i64([-1] * T), out)
    angle = pos.astype(np.longdouble)[:, None, None] * np.array(freq, np.longdouble)
    c, s = np.cos(angle).astype(np.float64), np.sin(angle).astype(np.float64)
    a, b = f64(x)[..., :64], f64(x)[..., 64:]
    want = np.concatenate([a * c - b * s, a * s + b * c], -1)
    assert np.all(np.abs(f64(out) - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -20 * 2 * np.abs(f64(x)).max())

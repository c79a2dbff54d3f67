"""Pins of the paged cache's fp64 oracle: codes against torch's casts and by
hand, scales, rotations, the planner's bookkeeping, attention's closed forms."""
import math

import numpy as np
import pytest
import torch

from oracle import cache_oracle as C


def test_codes_equal_torch_casts_and_hand_values():
    x = np.concatenate([np.linspace(-448, 448, 20011), np.linspace(-0.02, 0.02, 4001),
                        C._E4M3[:-1] + np.diff(C._E4M3) / 2])          # the midpoints: ties
    t = torch.from_numpy(x).float()
    np.testing.assert_array_equal(C.code_round(t.double().numpy(), "e4m3"), t.to(torch.float8_e4m3fn).double().numpy())
    np.testing.assert_array_equal(C.code_round([0.5, 1.5, -2.5, 300, -np.inf, np.nan], "int8"), [0, 2, -2, 127, -127, 0])
    assert [C.e4m3_value(c) for c in (0x01, 0x08, 0x7E, 0xFE)] == [2.0 ** -9, 2.0 ** -6, 448.0, -448.0]
    assert math.isnan(C.code_round([np.nan], "e4m3")[0]) and C.code_round([np.inf], "e4m3")[0] == 448


@pytest.mark.parametrize("code", ["e4m3", "int8"])
def test_scale_is_the_smallest_power_of_two_that_covers(code):
    assert C.scale_for(0.0, code) == C.MIN_SCALE
    for a in (1e-40, 3e-29, 0.3, 1.0, C.TOP[code], C.TOP[code] * (1 + 2.0 ** -7), 3e38):
        s = C.scale_for(a, code)
        assert math.log2(s) == int(math.log2(s)) and a <= s * C.TOP[code]
        assert s == C.MIN_SCALE or a > s / 2 * C.TOP[code]


def test_append_grows_a_scale_and_rounds_the_older_codes_again():
    c = C.PagedCache(2, 1, 16, 64, "int8")
    one = np.full((1, 1, 64), 1.0)
    c.append([0, 1], [16], one, one)
    assert c.ks[1, 0] == 2.0 ** -6 and c.k[1, 0, 0, 0] == 64
    c.append([0, 1], [17], 100 * one, one)
    assert c.ks[1, 0] == 1.0 and c.k[1, 0, 0, 0] == 1 and c.k[1, 0, 1, 0] == 100
    assert c.vs[1, 0] == 2.0 ** -6
    c.append([0, 1], [16], one / 4, one)                       # token 0 again: the page starts anew
    assert c.ks[1, 0] == 2.0 ** -8 and c.k[1, 0, 0, 0] == 64
    assert c.ks[0, 0] == C.MIN_SCALE


def test_rotation_keeps_lengths_and_relative_positions():
    rng = np.random.default_rng(0)
    freq, axis = [1.0, 0.3, 0.01, 2.0], [0, 1, 2, 0]
    for adjacent in (False, True):
        x, y = rng.standard_normal((2, 1, 1, 16))
        p = lambda a: np.array([[a], [2 * a], [5]])
        u, w = C.rotate(x, p(7), freq, axis, adjacent), C.rotate(y, p(3), freq, axis, adjacent)
        np.testing.assert_allclose(np.linalg.norm(u), np.linalg.norm(x))
        np.testing.assert_array_equal(u[..., 8:], x[..., 8:])
        u2, w2 = C.rotate(x, p(107), freq, axis, adjacent), C.rotate(y, p(103), freq, axis, adjacent)
        np.testing.assert_allclose(np.sum(u * w), np.sum(u2 * w2))
        np.testing.assert_array_equal(C.rotate(x, 0 * p(7), freq, axis, adjacent), x)


def test_planner_never_holds_a_page_twice_or_loses_one():
    rng = np.random.default_rng(1)
    for trial in range(200):
        page, n, m, n_pages = 16, int(rng.integers(1, 9)), 6, 24
        kv = [int(x) for x in rng.integers(0, 50, n)]
        ids = [int(x) for x in rng.permutation(n_pages)]
        table = [[-1] * m for _ in range(n)]
        for i in range(n):
            for j in range(-(-kv[i] // page)):
                if not ids:
                    kv[i] = j * page
                    break
                table[i][j] = ids.pop()
        want = [int(x) for x in rng.integers(0, 110, n)]
        kv2, t2, free, cu, slots, pos, st = C.plan_pages(page, want, kv, table, ids, n_pages, 200)
        held = [t2[i][j] for i in range(n) for j in range(-(-kv2[i] // page))]
        assert sorted(held + free) == list(range(n_pages))
        for i in range(n):
            assert kv2[i] == (want[i] if st[i] == 0 else kv[i])
            assert (st[i] == 2) == (want[i] > m * page)
        granted = [s for s in slots if s >= 0]
        assert len(set(granted)) == len(granted) == sum(max(0, want[i] - kv[i]) for i in range(n) if st[i] == 0)


def test_attention_closed_forms():
    rng = np.random.default_rng(2)
    k, v = rng.standard_normal((2, 5, 2, 8))
    o, mass, _ = C.attention(np.zeros((2, 4, 8)), k, v, 1, 0.3)     # equal scores: means
    np.testing.assert_allclose(o[0, 1], v[:2, 0].mean(0))
    np.testing.assert_allclose(o[1, 3], v[:3, 1].mean(0))
    np.testing.assert_allclose(mass[1, 3], np.abs(v[:3, 1]).mean(0))
    o, _, _ = C.attention(rng.standard_normal((3, 2, 8)), k, v, -2, 1.0)
    assert np.all(o[:1] == 0)
    np.testing.assert_allclose(o[2], v[0])

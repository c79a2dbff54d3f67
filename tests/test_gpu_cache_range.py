"""Attention over values of every size that bf16 holds: pages whose scales lie
far apart, sums that would pass fp32, and keys whose scale times the call's
passes it."""
import numpy as np
import pytest
import torch

import gated_deltanet_prefill_varlen_amd as gdn
from cache_util import DEV, DevCache, bf, f64, filled, i32, i64
from oracle import cache_oracle as C
from packed_util import few_rows, many_rows_call, packed_call
from test_gpu_cache import check_rows, decode_call, oracle_rows

pytestmark = pytest.mark.gpu

# sizes of the values in turn, each over a few pages
RISING, FALLING = [0.0, 1e-30, 1.0, 1e12, 1e30], [1e30, 1e12, 1.0, 1e-30, 0.0]
ORDERS = {"rising": RISING, "falling": FALLING, "mixed": [1.0, 0.0, 1e30, 1e-30, 1e12], "zeros first": [0.0, 1e37, 0.0, 1e37, 1e-20],
          "far below the first": [1e11, 0.0, 0.0, 0.0, 0.0], "at the border": [1e21, 1e-12, 1e23, 1e-10, 1e19],
          "near the largest": [3e37] * 5}


def sized(sizes, L, run):
    """[L, 1, 1]: the size of each token's values, `run` tokens each in turn."""
    return np.array([sizes[t // run % len(sizes)] for t in range(L)])[:, None, None]


@pytest.mark.parametrize("code", ["e4m3", "int8"])
@pytest.mark.parametrize("d,page,g", [(64, 16, 2), (128, 32, 2), (256, 16, 1)])
@pytest.mark.parametrize("order", list(ORDERS))
def test_packed_pages_of_values_far_apart(order, d, page, g, code):
    """Every row of a whole prompt, so that its first ones see the first sizes
    alone; heads whose queries are zero weigh all keys alike, so a page that
    dropped out of the sum shows."""
    rng = np.random.default_rng(d)
    L = max(170, 2 * few_rows(d))
    ref, dev, table, rows = filled(rng, [L], 1, page, d, code, 1.0, sized(ORDERS[order], L, 32))
    q = rng.standard_normal((L, g, d))
    q[::3] = 0.0
    q = bf(q).to(DEV)
    check_rows(many_rows_call(dev, [L], [L], table, q), oracle_rows(f64(q), rows, [L], [L], d ** -0.5), d, order)


@pytest.mark.parametrize("code", ["e4m3", "int8"])
@pytest.mark.parametrize("size", [1e-30, 1e-27, 1e20, 1e30])
def test_packed_small_probabilities_of_tiny_and_huge_values(size, code):
    """Scores spread over a hundred: channels whose likeliest keys hold codes of
    0 consist of probabilities far below 2^-26."""
    rng = np.random.default_rng(3)
    d, L = 128, 3 * few_rows(128)
    ref, dev, table, rows = filled(rng, [L], 1, 32, d, code, 1.0, size)
    q = bf(rng.standard_normal((L, 1, d))).to(DEV)
    check_rows(many_rows_call(dev, [L], [L], table, q, 1.0), oracle_rows(f64(q), rows, [L], [L], 1.0), d, size)


@pytest.mark.parametrize("code", ["e4m3", "int8"])
@pytest.mark.parametrize("low", [0, 2, 4])
def test_packed_sizes_apart_and_scores_apart(low, code):
    """One size's keys score hundreds below the others: huge values that no row
    weighs leave the tiny ones as they are."""
    rng = np.random.default_rng(low)
    d, page, run, L = 128, 16, 48, 240
    ref, dev, table, rows = filled(rng, [L], 1, page, d, code, 1.0, sized(RISING, L, run))
    k, v = ref.read([int(table[0, p // page]) * page + p % page for p in range(L)])
    k[:, :, 0] = np.where(np.arange(L) // run % 5 == low, 20.0, -20.0)[:, None]
    ref.append([0, L], [int(table[0, p // page]) * page + p % page for p in range(L)], C.round_bf16(k), C.round_bf16(v))
    dev.load(ref, [(int(table[0, p // page]), p % page) for p in range(L)])
    rows = [ref.read([int(table[0, p // page]) * page + p % page for p in range(L)])]
    q = 0.1 * rng.standard_normal((L, 2, d))
    q[:, 0, 0], q[:, 1, 0] = 20.0, -20.0
    q = bf(q).to(DEV)
    check_rows(many_rows_call(dev, [L], [L], table, q, 1.0), oracle_rows(f64(q), rows, [L], [L], 1.0), d, low)


@pytest.mark.parametrize("code", ["e4m3", "int8"])
@pytest.mark.parametrize("d,page,g,n_tok", [(64, 32, 2, 1), (128, 64, 4, 3), (128, 16, 20, 1), (256, 32, 2, 1), (256, 64, 6, 4)])
def test_decode_sums_of_values_near_the_largest(d, page, g, n_tok, code):
    """Thousands of values of one sign near bf16's largest: their mean is a
    number, their sum is none in fp32.  Alone, after pages of zeros and of ones,
    and as prompts of few rows."""
    rng = np.random.default_rng(d + g)
    lens = [4200, 3500, 700]
    assert n_tok * g <= few_rows(d)
    ref, dev, table, rows = filled(rng, lens, 1, page, d, code, 0.1, 1.0)
    # in place of the codes' scales: huge ones on all pages of the first request, and on some of the others'
    for i, every in enumerate((1, 3, 5)):
        ids = table[i, :-(-lens[i] // page)]
        ref.v[ids] = np.abs(ref.v[ids])
        ref.vs[ids[::every]] = 2.0 ** (119 if code == "e4m3" else 120)
        if every == 5:
            ref.vs[ids[1::5]] = 2.0 ** -100
    top = {"e4m3": 224.0, "int8": 100.0}[code]
    ref.v[:] = np.minimum(ref.v, top)
    dev.load(ref, [(int(table[i, p // page]), p % page) for i, n in enumerate(lens) for p in range(n)])
    rows = [ref.read([int(table[i, p // page]) * page + p % page for p in range(n)]) for i, n in enumerate(lens)]
    q = bf(rng.standard_normal((3 * n_tok, g, d))).to(DEV)
    want = oracle_rows(f64(q), rows, lens, [n_tok] * 3, d ** -0.5)
    check_rows(decode_call(dev, n_tok, lens, table, q), want, d, "decode")
    check_rows(packed_call(dev, [n_tok] * 3, lens, table, q), want, d, "few rows")


@pytest.mark.parametrize("code", ["e4m3", "int8"])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_keys_whose_scale_times_the_calls_passes_fp32(d, code):
    """Scores of 0 stay 0 however large the factor: the mean of the values."""
    rng = np.random.default_rng(d)
    L = 2 * few_rows(d) + 5
    ref, dev, table, rows = filled(rng, [L], 1, 32, d, code, 2e37, 1.0)
    q = torch.zeros(L, 1, d, dtype=torch.bfloat16, device=DEV)
    for scale in (5000.0, -5000.0):
        want = oracle_rows(f64(q), rows, [L], [L], scale)
        check_rows(many_rows_call(dev, [L], [L], table, q, scale), want, d, "packed")
        check_rows(decode_call(dev, 1, [L], table, q[:1], scale=scale), want[-1:], d, "decode")


@pytest.mark.parametrize("code", ["e4m3", "int8"])
def test_the_largest_values_read_back_as_rounded(code):
    """bf16's last values round up to 2^128, which it holds as infinity; those
    below 1.9375 * 2^127 read back as numbers."""
    top = np.array([255.0, 254.0, 252.0, 249.0, 248.0, 247.0, 240.0, 130.0, 1.0] + [0.0] * 7) * 2.0 ** 120
    for x in (top, top[4:], top[5:]):                  # the largest sets the page's scale
        rows = np.zeros((16, 1, 64))
        rows[:, 0, :len(x)] = x
        ref, dev = C.PagedCache(1, 1, 16, 64, code), DevCache(1, 1, 16, 64, code)
        t, slots = bf(rows).to(DEV), list(range(16))
        gdn.gdn_rope_append(gdn.make_rope([]), dev.handle, i32([0, 16]), [0, 16], None, t, -t, None, i64(slots), None)
        ref.append([0, 16], slots, f64(t), f64(-t))
        k, v = torch.empty_like(t), torch.empty_like(t)
        gdn.gdn_cache_gather(dev.handle, i64(slots), k, v)
        for got, want in zip((k, v), ref.read(slots)):
            np.testing.assert_array_equal(f64(got), np.where(np.abs(want) >= 2.0 ** 128, np.copysign(np.inf, want), want))
            assert np.all(np.isfinite(f64(got)[np.abs(f64(t)) < 1.9375 * 2.0 ** 127]))

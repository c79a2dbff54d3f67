"""The packed kernel of many rows on what a cache may hold besides numbers:
codes that are none, pages that are not held, pages behind the last token."""
import numpy as np
import pytest
import torch

from cache_util import DEV, bf, f64, filled
from oracle import cache_oracle as C
from packed_util import few_rows, many_rows_call
from test_gpu_cache import check_rows, oracle_rows

pytestmark = pytest.mark.gpu


def filled_apart_from_page_0(seed, lens, hkv, page, d, code):
    """Page 0, which is read where none is held, is nobody's: codes that are no
    numbers and NaN scales."""
    while True:
        rng = np.random.default_rng(seed)
        ref, dev, table, rows = filled(rng, lens, hkv, page, d, code)
        if all(0 not in table[i, :-(-n // page)] for i, n in enumerate(lens)):
            return rng, ref, dev, table, rows
        seed += 1000


@pytest.mark.parametrize("what", ["key", "value"])
@pytest.mark.parametrize("d,page,g,extra", [(64, 16, 1, 22), (64, 128, 3, 171), (128, 64, 2, 101), (128, 16, 1, 172), (256, 32, 2, 40), (256, 16, 1, 236)])
def test_codes_that_are_no_numbers_stay_with_the_rows_that_see_them(what, d, page, g, extra):
    """e4m3's NaN at the last key, at both ends and inside of the new tokens, in
    tiles that some rows see and in tiles that all see."""
    n = few_rows(d) // g + extra
    L, hkv = n + 75, 2
    rng, ref, dev, table, rows = filled_apart_from_page_0(d + n, [L, L], hkv, page, d, "e4m3")
    q = bf(rng.standard_normal((2 * n, hkv * g, d))).to(DEV)
    want = oracle_rows(f64(q), rows, [L, L], [n, n], d ** -0.5)
    for p in (L - 1, L - 2, L - n // 2, L - n + 1, L - n, L - n - 1, 64, 3):
        page_id, off = int(table[0, p // page]), p % page
        if what == "key":
            at = dev.k.view(torch.uint8)[page_id, 1, off, 5:6]
        else:
            at = dev.v.view(torch.uint8)[page_id, 1, off // 16, 5, off % 16:off % 16 + 1]
        old = at.clone()
        at.fill_(0xFF)
        got = f64(many_rows_call(dev, [n, n], [L, L], table, q))
        at.copy_(old)
        first = max(0, p - (L - n))                       # the first row that sees it
        nan = np.isnan(got[first:n, g:])
        assert np.all(nan if what == "key" else nan[..., 5]), p
        got[first:n, g:] = 0
        clean = list(want)
        for r in range(first, n):
            o = want[r][0].copy()
            o[g:] = 0
            clean[r] = (o,) + want[r][1:]
        check_rows(torch.from_numpy(got), clean, d, (what, p))


@pytest.mark.parametrize("code", ["e4m3", "int8"])
@pytest.mark.parametrize("d,page,g", [(64, 16, 2), (64, 64, 1), (128, 16, 1), (128, 128, 2), (256, 16, 1), (256, 32, 2)])
def test_pages_not_held_are_not_seen(d, page, g, code):
    """Holes at the first page, inside of a step's keys, over several steps and
    at the last page; a prompt whose pages are all gone, and one with none gone."""
    n = few_rows(d) // g + 30
    ctx = [0, 90, 33, 0, 200]
    lens = [n + x for x in ctx]
    new = [n] * len(lens)
    rng, ref, dev, table, rows = filled_apart_from_page_0(d + page, lens, 1, page, d, code)
    last = [(x - 1) // page for x in lens]
    holes = [{0}, {1, last[1]}, set(range(1, last[2])), set(range(last[3] + 1)), set()]
    outside = [-1, 1 << 30, dev.k.shape[0], -(1 << 31)]
    for i, cols in enumerate(holes):
        for c in cols:
            table[i, c] = outside[c % 4]
    q = bf(rng.standard_normal((sum(new), g, d))).to(DEV)
    out = many_rows_call(dev, new, lens, table, q)
    want, at = [], 0
    for i, x in enumerate(lens):
        keep = np.array([p for p in range(x) if p // page not in holes[i]], int)
        for r in range(n):
            sees = keep[keep <= x - n + r]
            o, mass, dot = C.attention(f64(q[at:at + 1]), rows[i][0][sees], rows[i][1][sees], len(sees) - 1, d ** -0.5)
            want.append((o[0], mass[0], dot[0], max(1, len(sees))))
            at += 1
    check_rows(out, want, d)
    assert torch.all(out[3 * n:4 * n] == 0)


@pytest.mark.parametrize("code", ["e4m3", "int8"])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_lengths_out_of_bounds_and_prompts_longer_than_their_keys(d, code):
    """NaN rows for lengths below 0 or over the table; prompts with more rows
    than keys: zeros ahead of the first key; the prompts beside them as alone."""
    n = few_rows(d) + 19
    lens = [n + 40, n - 25, 3, n]
    rng, ref, dev, table, rows = filled_apart_from_page_0(d, lens, 1, 32, d, code)
    q = bf(rng.standard_normal((4 * n, 1, d))).to(DEV)
    out = many_rows_call(dev, [n] * 4, lens, table, q)
    check_rows(out, oracle_rows(f64(q), rows, lens, [n] * 4, d ** -0.5), d)
    assert torch.all(out[n:n + 25] == 0) and torch.all(out[2 * n:3 * n - 3] == 0)
    bad = many_rows_call(dev, [n] * 4, [-1, lens[1], table.shape[1] * 32 + 1, n], table, q)
    assert torch.all(bad[:n].isnan()) and torch.all(bad[2 * n:3 * n].isnan())
    for i in (1, 3):
        assert torch.equal(bad[i * n:(i + 1) * n].view(torch.int16), out[i * n:(i + 1) * n].view(torch.int16))

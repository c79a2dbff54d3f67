"""The page planner over 1,024 requests, whose sums carry from one block of
requests to the next: refusals of every kind, in every block."""
import numpy as np
import pytest

from test_gpu_cache import check_plan, held

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("n", [1025, 2048, 2500])
def test_refusals_carry_over_blocks(n, in_place):
    rng = np.random.default_rng(n)
    m, page = 5, 16
    seen = set()
    for spare, kind in ((0, "any"), (n // 3, "any"), (n, "few"), (4 * n, "few"), (4 * n, "any"), (9, "grow"), (n // 2, "grow"), (n, "grow")):
        kv = [int(x) for x in rng.integers(0, m * page + 1, n)]
        table, free, n_pages = held(rng, kv, page, m, spare)
        want = [int(x) for x in rng.integers(0, m * page + 1, n)]
        if kind != "any":                            # a few tokens more (the slot map needs no launch of its own), or pages more
            want = [min(x + int(y), m * page) for x, y in zip(kv, rng.integers(0, 3 if kind == "few" else 40, n))]
        for i in rng.integers(0, n, 12):             # 3: negative or more than a row holds; 2: more wanted than a row holds
            want[i] = -1 - int(i)
        for i in rng.integers(0, n, 12):
            want[i] = m * page + 1 + int(i)
        for i in rng.integers(0, n, 6):
            kv[i] = -3 if i % 2 else m * page + 1
        new = [0 if w < 0 or x < 0 or x > m * page else max(0, w - x) for w, x in zip(want, kv)]
        for cap in (1, sum(new[:1024]) + 1, sum(new) // 2, sum(new[:-1]), sum(new), sum(new) + 7):
            got = check_plan(page, want, kv, table, free, n_pages, max(1, cap), in_place)
            seen |= {(int(s), i // 1024) for i, s in enumerate(got["st"])}
    blocks = n // 1024                               # (one request alone, the 1,025th, has one of them)
    assert seen >= {(s, b) for s in range(5) for b in range(blocks)} and max(b for _, b in seen) == (n - 1) // 1024


@pytest.mark.parametrize("cap", [4095, 4096, 4097])
def test_slot_maps_on_both_sides_of_a_launch_of_their_own(cap):
    rng = np.random.default_rng(cap)
    n, m, page = 1500, 6, 32
    for total in (cap - 40, cap, cap + 40):
        kv = [int(x) for x in rng.integers(0, m * page - 8, n)]
        want = list(kv)
        while sum(want) - sum(kv) < total:
            i = int(rng.integers(0, n))
            want[i] = min(want[i] + 5, m * page, want[i] + total - (sum(want) - sum(kv)))
        for i in range(0, n, 7):
            if want[i] == kv[i]:
                want[i] = kv[i] // 2
        total_new = sum(max(0, w - x) for w, x in zip(want, kv))
        assert total_new == total
        table, free, n_pages = held(rng, kv, page, m, n)
        check_plan(page, want, kv, table, free, n_pages, cap)

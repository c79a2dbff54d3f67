"""The paged cache's calls at the edges: codes that are no numbers seen by some
rows only, requests over several splits, packs of many row blocks and key steps
of every remainder, tables that share pages, the planner at its block's size."""
import numpy as np
import pytest
import torch

import gated_deltanet_prefill_varlen_amd as gdn
from cache_util import DEV, bf, f64, filled, i32, i64, slots_of
from oracle import cache_oracle as C
from test_gpu_cache import check_plan, check_rows, decode_call, held, oracle_rows

pytestmark = pytest.mark.gpu


def packed_call(dev, new, lens, table, q, **kw):
    cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    out = torch.full_like(q, 5.0)
    gdn.gdn_attn_packed(dev.handle, i32(cu), cu, i32(lens), i32(table), q, out, **kw)
    return out


@pytest.mark.parametrize("what", ["key", "value"])
@pytest.mark.parametrize("d,page,n_tok,L", [(64, 16, 4, 67), (128, 64, 4, 131), (128, 16, 2, 1025), (256, 32, 3, 66), (256, 16, 12, 300)])
def test_a_code_that_is_no_number_stays_with_the_rows_that_see_it(what, d, page, n_tok, L):
    """The j-th last key holds e4m3's NaN: the rows before it must come out as
    if it were not there, the rows from it on hold NaN."""
    rng = np.random.default_rng(d + L)
    hkv, g = 2, 3
    ref, dev, table, rows = filled(rng, [L, L], hkv, page, d, "e4m3")
    for back in (1, 2, n_tok):
        p = L - back
        page_id, off = int(table[0, p // page]), p % page
        if what == "key":
            at = dev.k.view(torch.uint8)[page_id, 1, off, 5:6]
        else:
            at = dev.v.view(torch.uint8)[page_id, 1, off // 16, 5, off % 16:off % 16 + 1]
        old = at.clone()
        at.fill_(0x7F)
        q = bf(rng.standard_normal((2 * n_tok, hkv * g, d))).to(DEV)
        want = oracle_rows(f64(q), rows, [L, L], [n_tok, n_tok], d ** -0.5)
        for out in (decode_call(dev, n_tok, [L, L], table, q), packed_call(dev, [n_tok, n_tok], [L, L], table, q)):
            got = f64(out)
            sees = slice(n_tok - back, n_tok)
            nan = np.isnan(got[sees, g:])
            assert np.all(nan if what == "key" else nan[..., 5])
            got[sees, g:] = 0
            clean = [(o.copy(), m, dt, k) for o, m, dt, k in want]
            for r in range(n_tok - back, n_tok):
                clean[r][0][g:] = 0
            check_rows(torch.from_numpy(got), clean, d, (what, back))
        at.copy_(old)


@pytest.mark.parametrize("code", ["e4m3", "int8"])
@pytest.mark.parametrize("d,page,hkv,g,n_tok", [(64, 128, 1, 4, 1), (128, 16, 1, 8, 1), (128, 32, 2, 9, 2), (256, 64, 1, 4, 1), (256, 128, 1, 12, 2)])
def test_decode_over_several_splits(code, d, page, hkv, g, n_tok):
    rng = np.random.default_rng(d + n_tok)
    lens = [5001, 0, 1024, 1536, 1537, 2049, 4607, 4609, n_tok, 9000]
    ref, dev, table, rows = filled(rng, lens, hkv, page, d, code)
    q = bf(rng.standard_normal((len(lens) * n_tok, hkv * g, d))).to(DEV)
    out = decode_call(dev, n_tok, lens, table, q)
    check_rows(out, oracle_rows(f64(q), rows, lens, [n_tok] * len(lens), d ** -0.5), d)
    # a bound far over the lengths (more splits than any request has) leaves the bits as they are
    wide = np.full((len(lens), table.shape[1] + 200), -1, np.int32)
    wide[:, :table.shape[1]] = table
    assert torch.equal(decode_call(dev, n_tok, lens, wide, q).view(torch.int16), out.view(torch.int16))
    # and so does a bound that just holds them
    assert torch.equal(decode_call(dev, n_tok, lens, wide, q, max_kv=9000).view(torch.int16), out.view(torch.int16))


@pytest.mark.parametrize("code", ["e4m3", "int8"])
@pytest.mark.parametrize("d,page,g", [(64, 32, 3), (128, 64, 4), (128, 16, 5), (256, 128, 2)])
def test_packed_many_row_blocks_and_key_steps_of_every_remainder(code, d, page, g):
    rng = np.random.default_rng(d + g)
    new = [90, 64, 130, 1, 256, 3]
    lens = [90 + 64 * 5, 64 + 64 * 3, 130 + 63, 1 + 64 * 4, 256, 3 + 64 * 8 - 2]
    ref, dev, table, rows = filled(rng, lens, 1, page, d, code)
    q = bf(rng.standard_normal((sum(new), g, d))).to(DEV)
    check_rows(packed_call(dev, new, lens, table, q), oracle_rows(f64(q), rows, lens, new, d ** -0.5), d)


@pytest.mark.parametrize("n", [1, 2, 63, 64, 65, 130])
def test_packed_every_row_of_any_number_of_prompts(n):
    """Long, short, empty and out-of-bounds prompts: whatever the order in which
    tiles are taken, each row is written once and rows behind the last stay."""
    rng = np.random.default_rng(n)
    d, page, g = 64, 64, 8
    new = [int(x) for x in rng.choice([0, 1, 3, 31, 33, 70, 100], n)]
    new[0] = 90
    ctx = [int(x) for x in rng.choice([0, 0, 5, 250, 600, 1300, -40], n)]
    lens = [max(0, a + b) for a, b in zip(new, ctx)]
    ref, dev, table, rows = filled(rng, lens, 1, page, d, "int8")
    q = bf(rng.standard_normal((sum(new), g, d))).to(DEV)
    want = oracle_rows(f64(q), rows, lens, new, d ** -0.5)
    out = packed_call(dev, new, lens, table, q)
    check_rows(out, want, d)
    bad = list(lens)
    bad[n // 2], bad[0] = -3, table.shape[1] * page + 1
    got, at = packed_call(dev, new, bad, table, q), 0
    for i, x in enumerate(new):
        if bad[i] != lens[i]:
            assert torch.all(torch.isnan(got[at:at + x]))
        else:
            assert torch.equal(got[at:at + x].view(torch.int16), out[at:at + x].view(torch.int16))
        at += x


@pytest.mark.parametrize("code", ["e4m3", "int8"])
def test_requests_that_share_the_pages_of_a_prefix(code):
    rng = np.random.default_rng(21)
    d, page, hkv, g = 128, 16, 2, 2
    ref, dev, table, rows = filled(rng, [200], hkv, page, d, code)
    lens = [200, 131, 131, 16, 1]
    both = np.repeat(table, len(lens), 0)
    cut = [(rows[0][0][:n], rows[0][1][:n]) for n in lens]
    q = bf(rng.standard_normal((len(lens), hkv * g, d))).to(DEV)
    q[2] = q[1]
    want = oracle_rows(f64(q), cut, lens, [1] * len(lens), d ** -0.5)
    for out in (decode_call(dev, 1, lens, both, q), packed_call(dev, [1] * len(lens), lens, both, q)):
        check_rows(out, want, d)
        assert torch.equal(out[1].view(torch.int16), out[2].view(torch.int16))
    s = slots_of(table, page, 0, 60, 90) * 2       # the same rows twice in one read
    k_out = torch.empty(60, hkv, d, dtype=torch.bfloat16, device=DEV)
    gdn.gdn_cache_gather(dev.handle, i64(s), k_out, None)
    np.testing.assert_array_equal(f64(k_out), np.concatenate([rows[0][0][60:90]] * 2))


@pytest.mark.parametrize("code", ["e4m3", "int8"])
@pytest.mark.parametrize("d,g", [(64, 4), (128, 4), (128, 1), (256, 4), (256, 16)])
def test_packed_bits_do_not_depend_on_the_pack(code, d, g):
    """Prompts of few and of many rows, on both sides of every limit: alone, two
    together and all in one pack."""
    rng = np.random.default_rng(d + g)
    new = [1, 4, 5, 16, 17, 32, 33, 2, 64, 65, 129, 0]
    lens = [int(x) + int(y) for x, y in zip(new, rng.choice([0, 7, 300, 700], len(new)))]
    ref, dev, table, rows = filled(rng, lens, 1, 32, d, code)
    q = bf(rng.standard_normal((sum(new), g, d))).to(DEV)
    whole = packed_call(dev, new, lens, table, q)
    check_rows(whole, oracle_rows(f64(q), rows, lens, new, d ** -0.5), d)
    cu = np.concatenate([[0], np.cumsum(new)])
    for a, b in [(i, i + 1) for i in range(len(new))] + [(i, i + 2) for i in range(0, len(new) - 1, 2)]:
        part = packed_call(dev, new[a:b], lens[a:b], table[a:b], q[cu[a]:cu[b]].contiguous())
        assert torch.equal(part.view(torch.int16), whole[cu[a]:cu[b]].view(torch.int16)), (a, b)


def test_rows_that_overlap_are_refused():
    """A broadcast token has a stride of 0, which the C call takes for dense
    rows: the binding must not pass it on."""
    rng = np.random.default_rng(2)
    ref, dev, table, rows = filled(rng, [20, 20], 1, 16, 64, "int8")
    one = bf(rng.standard_normal((1, 2, 64))).to(DEV)
    wide, out = one.expand(2, 2, 64), torch.empty(2, 2, 64, dtype=torch.bfloat16, device=DEV)
    with pytest.raises(ValueError, match="overlap"):
        gdn.gdn_attn_decode(dev.handle, 1, i32([20, 20]), i32(table), wide, out)
    with pytest.raises(ValueError, match="overlap"):
        gdn.gdn_attn_packed(dev.handle, i32([0, 1, 2]), [0, 1, 2], i32([20, 20]), i32(table), wide, out)
    kv = out[:, :1].contiguous()
    slots, cu = i64([0, 1]), i32([0, 2])
    for args in ((wide, kv, kv, out), (out, one[:, :1].expand(2, 1, 64), kv, out), (out, kv, kv, wide)):
        with pytest.raises(ValueError, match="overlap"):
            gdn.gdn_rope_append(gdn.make_rope([]), dev.handle, cu, [0, 2], args[0], args[1], args[2], None, slots, args[3])
    got = torch.empty_like(out[:1])                                    # a single row may have any stride
    gdn.gdn_attn_decode(dev.handle, 1, i32([20]), i32(table[:1]), one.expand(2, 2, 64)[:1], got)
    check_rows(got, oracle_rows(f64(one), rows[:1], [20], [1], 64 ** -0.5), 64)


@pytest.mark.parametrize("n", [63, 64, 65, 1000, 1023, 1024])
def test_plan_at_the_block_size(n):
    """Growing, shrinking and ending requests with a stack too short for all:
    the last ones are refused, pages given back serve the others."""
    rng = np.random.default_rng(n)
    m, page = 5, 16
    kv = [int(x) for x in rng.integers(0, m * page + 1, n)]
    for spare in (0, n // 3, 3 * n):
        table, free, n_pages = held(rng, kv, page, m, spare)
        want = [int(x) for x in rng.integers(0, m * page + 1, n)]
        want[0] = -1
        if n > 2:
            want[n // 2], want[n - 1] = m * page + 1, kv[n - 1] + 1
        new = sum(max(0, w - x) for w, x in zip(want, kv))
        for cap in (max(1, new // 2), new + 7):
            check_plan(page, want, kv, table, free, n_pages, cap, in_place=spare == 0)


def test_planner_append_and_read_in_a_graph_with_requests_that_end():
    """Two tokens a request and replay, captured once; between replays some
    requests end and begin again.  Each replay equals the eager calls on a copy."""
    page, n, m, d, hkv = 16, 5, 8, 64, 1
    kv, want = i32([0] * n), i32([0] * n)
    table, free, count = i32(np.full((n, m), -1)), i32(range(n * m)), i32([n * m])
    cu, slots, st, pos = i32([0] * (n + 1)), i64([0] * (2 * n)), i32([0] * n), i32([0] * (2 * n))
    host = [2 * i for i in range(n + 1)]
    k = bf(np.random.default_rng(4).standard_normal((2 * n, hkv, d))).to(DEV)
    cache = [torch.zeros(n * m, hkv, page, d, dtype=torch.int8, device=DEV), torch.zeros(n * m, hkv, 1, d, 16, dtype=torch.int8, device=DEV),
             torch.zeros(n * m, hkv, device=DEV), torch.zeros(n * m, hkv, device=DEV)]
    state = (kv, table, free, count, cache, torch.empty_like(k), want, cu, slots, st, pos)
    copy = lambda s: tuple([x.clone() for x in t] if isinstance(t, list) else t.clone() for t in s)
    flat = lambda s: [x for t in s for x in (t if isinstance(t, list) else [t])]

    def step(kv, table, free, count, cache, out, want, cu, slots, st, pos):
        gdn.gdn_plan_pages(page, want, kv, kv, table, free, count, count, cu, slots, pos, st)
        h = gdn.make_cache(*cache)
        gdn.gdn_rope_append(gdn.make_rope([1.0] * 8), h, cu, host, None, k, k, pos, slots, None)
        gdn.gdn_cache_gather(h, slots, out, None)

    def end(s, which):
        lens = s[0].clone()
        lens[which] = 0
        gdn.gdn_plan_pages(page, lens, s[0], s[0], s[1], s[2], s[3], s[3], i32([0] * (n + 1)), i64([0]), None, i32([0] * n))

    eager = copy(state)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(*state)
    for rep in range(12):
        for s in (state, eager):
            if rep % 4 == 3:
                end(s, [rep % n, (rep + 2) % n])
            s[6].copy_(s[0] + 2)
            k.mul_(1.0 + rep % 2)          # scales grow now and then
        graph.replay()
        step(*eager)
        torch.cuda.synchronize()
        assert torch.all(state[9] == 0) and int(state[0].max()) > 0
        for a, b in zip(flat(state), flat(eager)):
            assert torch.equal(a, b)

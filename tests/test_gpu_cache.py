"""The paged 8-bit cache on the GPU against its fp64 oracle: page planner,
rotary positions with the cache's write, read back, and attention for packs
and decode batches; then all of them together, eager and captured."""
import numpy as np
import pytest
import torch

import gated_deltanet_prefill_varlen_amd as gdn
from cache_util import DEV, DevCache, attn_bound, bf, f64, filled, i32, i64, slots_of, tables
from oracle import cache_oracle as C

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ planner --

def run_plan(page, want, kv, table, free, n_pages, cap, in_place=False):
    n = len(want)
    stack = np.full(n_pages, -7, np.int32)
    stack[:len(free)] = free
    d = dict(want=i32(want), kv=i32(kv), table=i32(np.asarray(table).reshape(n, len(table[0]) if n else 2)), free=i32(stack), count=i32([len(free)]),
             cu=i32([-9] * (n + 1)), slots=i64([-9] * cap), pos=i32([-9] * cap), st=i32([-9] * n))
    d["kv2"] = d["kv"] if in_place else i32([-9] * n)
    d["count2"] = d["count"] if in_place else i32([-9])
    gdn.gdn_plan_pages(page, d["want"], d["kv"], d["kv2"], d["table"], d["free"], d["count"], d["count2"], d["cu"], d["slots"],
                       d["pos"], d["st"])
    torch.cuda.synchronize()
    return {k: v.cpu().numpy() for k, v in d.items()}


def check_plan(page, want, kv, table, free, n_pages, cap, in_place=False):
    got = run_plan(page, want, kv, table, free, n_pages, cap, in_place)
    kv2, t2, f2, cu, slots, pos, st = C.plan_pages(page, want, kv, table, free, n_pages, cap)
    for name, ref in (("kv2", kv2), ("cu", cu), ("slots", slots), ("pos", pos), ("st", st)):
        np.testing.assert_array_equal(got[name], ref, err_msg=name)
    np.testing.assert_array_equal(got["table"].reshape(-1), np.reshape(t2, -1))
    assert got["count2"][0] == len(f2)
    np.testing.assert_array_equal(got["free"][:len(f2)], f2)
    return got


def held(rng, lens, page, m, spare):
    need = [-(-x // page) for x in lens]
    n_pages = sum(need) + spare
    ids = [int(x) for x in rng.permutation(n_pages)]
    table = [[-1 - j for j in range(m)] for _ in lens]
    for i, x in enumerate(need):
        for j in range(x):
            table[i][j] = ids.pop()
    return table, ids, n_pages


@pytest.mark.parametrize("page", [16, 32, 64, 128])
def test_plan_random_lengths_refusals_and_aliases(page):
    rng = np.random.default_rng(page)
    for trial in range(12):
        n, m = int(rng.integers(1, 40)), 9
        kv = [int(x) for x in rng.integers(0, m * page + 1, n)]
        table, free, n_pages = held(rng, kv, page, m, int(rng.integers(0, 60)))
        want = [int(x) for x in rng.integers(-3, (m + 1) * page, n)]
        for i in rng.integers(0, n, 3):
            want[i] = kv[i] + 1
        if trial % 3 == 0:
            kv[int(rng.integers(0, n))] = -5 if trial % 2 else m * page + 1
        new = sum(max(0, w - x) for w, x in zip(want, kv))
        check_plan(page, want, kv, table, free, n_pages, max(1, int(new * rng.choice([0.6, 1.0, 1.3]))), in_place=trial % 2 == 0)


def test_plan_none_one_and_many_requests():
    rng = np.random.default_rng(3)
    got = run_plan(16, [], [], np.zeros((0, 2)), [4, 5], 6, 3)
    assert got["count2"][0] == 2 and got["cu"][0] == 0 and list(got["slots"]) == [-1] * 3
    check_plan(16, [1], [0], [[-1]], [0], 1, 1)
    check_plan(16, [0], [16], [[0]], [], 1, 1)
    check_plan(16, [16], [16], [[0]], [], 1, 1)
    # over 1,024 requests: the prefix sums carry on; long rows; a slot map of its own launch
    for n, hi, m in [(1025, 40, 4), (2500, 40, 4), (9, 4000, 300)]:
        kv = [int(x) for x in rng.integers(0, hi, n)]
        table, free, n_pages = held(rng, kv, 16, m, n)
        want = [x + int(y) for x, y in zip(kv, rng.integers(0, 30 if m == 4 else 800, n))]
        for i in range(0, n, 5):
            want[i] = 0
        new = sum(max(0, w - x) for w, x in zip(want, kv))
        for cap in (new, new + 5000):
            check_plan(16, want, kv, table, free, n_pages, cap)


# --------------------------------------------------------- rotation, write --

def half_step(value, scale, code):
    """Half a step of the code that holds `value`."""
    if code == "int8":
        return 0.5 * scale
    return np.maximum(2.0 ** -4 * np.abs(value), 2.0 ** -10 * scale)


def check_cache(dev, ref, rotated):
    """Device codes and scales against the oracle's: equal where nothing is
    rotated.  A rotated key in fp32 is off by a few 2^-24 of its pair, so its
    bf16 rounding may go the other way (a step of 2^-7) and its code with it."""
    k, v, ks, vs = dev.codes()
    live = ~np.isnan(vs)
    np.testing.assert_array_equal(np.where(live, vs, 0), np.where(live, ref.vs, 0))
    np.testing.assert_array_equal(np.where(live, ks, 0), np.where(live, ref.ks, 0))
    return k, v


@pytest.mark.parametrize("code", ["e4m3", "int8"])
@pytest.mark.parametrize("d,page,hkv,hq,rot,axes,adjacent", [
    (64, 16, 1, 3, 16, 1, True), (64, 128, 2, 2, 64, 3, False), (128, 16, 8, 32, 64, 3, False), (128, 64, 2, 4, 128, 4, True),
    (256, 32, 3, 3, 64, 1, False), (256, 128, 1, 5, 256, 2, True), (128, 32, 2, 2, 0, 1, False), (256, 64, 2, 2, 48, 2, False)])
def test_append_and_gather_vs_oracle(code, d, page, hkv, hq, rot, axes, adjacent):
    """Prompts from the middle of pages, then single tokens, on columns of one
    row; scales grow; the pages held poison before."""
    rng = np.random.default_rng(d + page + rot)
    first = [0, 5, page - 1, 3 * page + 7, page, 0]
    steps = [[1, page, 2, 2 * page + 3, 0, 3 * page], [1, 1, 1, 1, 2, 1], [1, 0, 1, 3, 1, 1]]
    total = [a + sum(s[i] for s in steps) for i, a in enumerate(first)]
    table, n_pages = tables(rng, total, page)
    ref, dev = C.PagedCache(n_pages, hkv, page, d, code), DevCache(n_pages, hkv, page, d, code)
    freq = [float(np.float32(10000.0 ** (-i / max(1, rot // 2)))) for i in range(rot // 2)]
    axis = [i % axes for i in range(rot // 2)]
    rope = gdn.make_rope(freq, axis, axes, adjacent, 1.25)
    written = []
    lens = [0] * len(first)
    for step, new in enumerate([first] + steps):
        cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        T = int(cu[-1])
        row = rng.standard_normal((T, (hq + 2 * hkv) * d + 8)) * (1.0 + 3.0 * step)
        row = bf(row).to(DEV)
        q = row[:, :hq * d].view(T, hq, d)
        k = row[:, hq * d:(hq + hkv) * d].view(T, hkv, d)
        v = row[:, (hq + hkv) * d:(hq + 2 * hkv) * d].view(T, hkv, d)
        pos = rng.integers(0, 1 << 20, (axes, T)).astype(np.int32)
        slots = [s for i, x in enumerate(new) for s in slots_of(table, page, i, lens[i], lens[i] + x)]
        out = torch.full((T + 1, hq, d), 7.0, dtype=torch.bfloat16, device=DEV)
        gdn.gdn_rope_append(rope, dev.handle, i32(cu), cu, q, k, v, i32(pos), i64(slots), out)
        q64, k64 = f64(q), f64(k)
        q_ref = C.rotate(q64, pos, freq, axis, adjacent, 1.25)
        # fp32: two products and a sum (3 roundings) of cos and sin off by 2^-22
        pair = 1.25 * (np.abs(q64).max() * 2)
        assert np.all(np.abs(f64(out[:T]) - q_ref) <= 2.0 ** -8 * np.abs(q_ref) + 2.0 ** -20 * pair)
        assert torch.all(out[T:] == 7.0)
        k_rot = C.round_bf16(C.rotate(k64, pos, freq, axis, adjacent, 1.25)) if rot else k64
        ref.append(list(cu), slots, k_rot, f64(v))
        lens = [a + b for a, b in zip(lens, new)]
        written += slots
        check_cache(dev, ref, rot > 0)
        kr, vr = ref.read(written)
        k_out = torch.empty(len(written), hkv, d, dtype=torch.bfloat16, device=DEV)
        v_out = torch.empty_like(k_out)
        gdn.gdn_cache_gather(dev.handle, i64(written), k_out, v_out)
        np.testing.assert_array_equal(f64(v_out), vr)
        if rot == 0:
            np.testing.assert_array_equal(f64(k_out), kr)
        else:
            got = f64(k_out)
            ksc = np.stack([ref.ks[s // page] for s in written])[:, :, None]
            # two code roundings (older codes were rounded once per growth before: under a step more), two bf16 ones
            lim = 2 * (half_step(got, ksc, code) + half_step(kr, ksc, code)) + 2.0 ** -6 * np.abs(kr) + 2.0 ** -20 * np.abs(k64).max()
            assert np.all(np.abs(got - kr) <= lim)
            assert np.mean(got != kr) < 1e-3
        # read back: exactly code * scale
        kc, _, ks, _ = dev.codes()
        pg, off = np.array(written) // page, np.array(written) % page
        np.testing.assert_array_equal(f64(k_out), kc[pg, :, off] * ks[pg][:, :, None])


@pytest.mark.parametrize("code", ["e4m3", "int8"])
def test_append_far_positions_skipped_slots_and_values_that_are_no_numbers(code):
    rng = np.random.default_rng(5)
    d, page, hkv, T = 128, 32, 2, 70
    k, v = rng.standard_normal((2, T, hkv, d))
    v[3, 0, 5], v[4, 1, 6], v[5, 0, 7] = np.inf, -np.inf, np.nan
    v[6] = 0.0
    v[40, 0, 9] = np.nan
    dev, ref = DevCache(9, hkv, page, d, code), C.PagedCache(9, hkv, page, d, code)
    slots = slots_of(np.array([[4, 2, 7]]), page, 0, 6, 6 + T)
    slots[10] = -1                    # refused
    slots[30] = slots[30] + 1         # breaks its page's run
    slots[60:] = [page * 9 + 5] * 10  # outside the cache
    kt, vt = bf(k).to(DEV), bf(v).to(DEV)
    gdn.gdn_rope_append(gdn.make_rope([]), dev.handle, i32([0, T]), [0, T], None, kt, vt, None, i64(slots), None)
    ref.append([0, T], slots, f64(kt), f64(vt))
    kc, vc, ks, vs = dev.codes()
    for t, s in enumerate(slots):
        if t in (10, 30) or t >= 60:
            continue
        np.testing.assert_array_equal(kc[s // page, :, s % page], ref.k[s // page, :, s % page])
        np.testing.assert_array_equal(vc[s // page, :, s % page], ref.v[s // page, :, s % page])
    np.testing.assert_array_equal(vs[[4, 2, 7]], ref.vs[[4, 2, 7]])
    raw = dev.k.view(torch.uint8).cpu().numpy()
    for p in (0, 1, 3, 5, 6, 8):      # nobody's pages, and the offset not written
        assert np.all(raw[p] == 0x7F)
    assert np.all(raw[4, :, 6 + 10] == 0x7F)   # (offsets 0 to 5 count as held: rounded again to the new scale)
    # gather: any order, repeated, outside
    odd = [slots[5], -1, slots[5], 9 * page, slots[0], -(1 << 40), 1 << 40]
    ko = torch.full((len(odd), hkv, d), 3.0, dtype=torch.bfloat16, device=DEV)
    gdn.gdn_cache_gather(dev.handle, i64(odd), None, ko)
    got = f64(ko)
    np.testing.assert_array_equal(got[0], got[2])
    assert np.all(got[[1, 3, 5, 6]] == 0)
    np.testing.assert_array_equal(got[4], ref.read([slots[0]])[1][0])
    # positions near 2^31: the angle is formed in 64 bits
    T, freq = 5, [float(np.float32(1.0 / (i + 1))) for i in range(64)]
    pos = np.array([[0, 1, 1 << 24, (1 << 31) - 1, 123456789]], np.int32)
    x = bf(rng.standard_normal((T, 4, d))).to(DEV)
    y = x.clone()
    none = i64([-1] * T)
    gdn.gdn_rope_append(gdn.make_rope(freq), dev.handle, i32([0, T]), [0, T], y, kt[:T], vt[:T], i32(pos[0]), none, y)   # in place
    want = C.rotate(f64(x), pos, freq, [0] * 64)
    assert np.all(np.abs(f64(y) - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -20 * 2 * np.abs(f64(x)).max())
    assert np.all(dev.k.view(torch.uint8).cpu().numpy() == raw)


# -------------------------------------------------------------- attention --

def check_rows(out, ref_rows, d, what=""):
    got = f64(out)
    for r, (o, mass, dot, keys) in enumerate(ref_rows):
        err = np.abs(got[r] - o) - attn_bound(o, mass, dot, d, keys)
        assert np.all(err <= 0), (what, r, float(err.max()))


def oracle_rows(q64, rows, lens, new, scale):
    out, at = [], 0
    for i, n in enumerate(new):
        k, v = rows[i]
        o, mass, dot = C.attention(q64[at:at + n], k, v, lens[i] - n, scale)
        out += [(o[j], mass[j], dot[j], max(1, lens[i])) for j in range(n)]
        at += n
    return out


def decode_call(dev, n_tok, lens, table, q, out=None, max_kv=None, scale=None, **kw):
    out = torch.full_like(q, 5.0) if out is None else out
    m = table.shape[1] * dev.page if max_kv is None else max_kv
    size = gdn.gdn_attn_decode_workspace(dev.handle, q.shape[1], len(lens), n_tok, m)
    ws = torch.full((size,), 0xFF, dtype=torch.uint8, device=DEV)      # what memory may hold: NaN
    gdn.gdn_attn_decode(dev.handle, n_tok, i32(lens), i32(table), q, out, max_kv, scale, ws, **kw)
    return out


LENS = [0, 1, 15, 16, 17, 63, 64, 65, 127, 128, 129, 200, 255, 256, 257, 511, 513, 700, 1023, 1024, 1025]


@pytest.mark.parametrize("code", ["e4m3", "int8"])
@pytest.mark.parametrize("d,page,hkv,g,n_tok", [(64, 16, 2, 1, 1), (64, 64, 1, 8, 4), (128, 16, 2, 4, 1), (128, 64, 1, 16, 1), (128, 128, 1, 5, 3),
                                                (128, 32, 1, 17, 1), (256, 16, 1, 8, 1), (256, 128, 1, 3, 2), (256, 32, 1, 12, 5),
                                                (64, 32, 1, 64, 2), (128, 64, 1, 1, 70)])
def test_decode_vs_oracle(code, d, page, hkv, g, n_tok):
    rng = np.random.default_rng(d + page + g + n_tok)
    lens = LENS if n_tok < 10 else [0, 30, 69, 70, 71, 333]
    ref, dev, table, rows = filled(rng, lens, hkv, page, d, code)
    q = bf(rng.standard_normal((len(lens) * n_tok, hkv * g, d))).to(DEV)
    out = decode_call(dev, n_tok, lens, table, q)
    check_rows(out, oracle_rows(f64(q), rows, lens, [n_tok] * len(lens), d ** -0.5), d)


@pytest.mark.parametrize("code", ["e4m3", "int8"])
@pytest.mark.parametrize("d,page,hkv,g", [(64, 16, 2, 1), (64, 64, 1, 7), (128, 16, 1, 4), (128, 64, 2, 2), (128, 128, 1, 16), (128, 32, 1, 33), (256, 16, 1, 8),
                                          (256, 64, 1, 3)])
def test_packed_vs_oracle(code, d, page, hkv, g):
    """Prompts with and without a cached prefix, empty ones, more rows than
    keys (their first rows see nothing), rows of a wider row, untouched tail."""
    rng = np.random.default_rng(d + page + g)
    new = [1, 0, 17, 64, 65, 130, 7, 33, 200]
    ctx = [0, 9, 0, 0, 100, 3, -4, 257, 63]
    lens = [max(0, a + b) for a, b in zip(new, ctx)]
    ref, dev, table, rows = filled(rng, lens, hkv, page, d, code)
    T, hq = sum(new), hkv * g
    wide = bf(rng.standard_normal((T, hq * d + 16))).to(DEV)
    q = wide[:, :hq * d].view(T, hq, d)
    cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    out = torch.full((T + 3, hq, d), 5.0, dtype=torch.bfloat16, device=DEV)
    gdn.gdn_attn_packed(dev.handle, i32(cu), cu, i32(lens), i32(table), q, out, scale=0.11)
    check_rows(out[:T], oracle_rows(f64(q), rows, lens, new, 0.11), d)
    assert torch.all(out[T:] == 5.0)


@pytest.mark.parametrize("code", ["e4m3", "int8"])
def test_attention_wide_scores_tiny_and_huge_values(code):
    """Scores spread over hundreds (one key takes all), a steady rise (the
    running maximum moves with every key), values of 1e-30 and 1e30."""
    rng = np.random.default_rng(8)
    d, page, hkv, g = 128, 16, 1, 4
    for k_scale, v_scale in [(30.0, 1.0), (1.0, 1e-30), (1.0, 1e30), (1e-20, 1.0)]:
        lens = [300, 77]
        ref, dev, table, rows = filled(rng, lens, hkv, page, d, code, k_scale, v_scale)
        q = bf(rng.standard_normal((2, hkv * g, d))).to(DEV)
        check_rows(decode_call(dev, 1, lens, table, q), oracle_rows(f64(q), rows, lens, [1, 1], d ** -0.5), d, (k_scale, v_scale))
        new = [40, 77]
        q = bf(rng.standard_normal((117, hkv * g, d))).to(DEV)
        out, cu = torch.empty_like(q), np.array([0, 40, 117], np.int32)
        gdn.gdn_attn_packed(dev.handle, i32(cu), cu, i32(lens), i32(table), q, out)
        check_rows(out, oracle_rows(f64(q), rows, lens, new, d ** -0.5), d, (k_scale, v_scale))
    ramp = np.linspace(-40, 40, 300)[:, None, None] * np.ones((1, 1, d)) / d
    ref, dev, table, rows = filled(rng, [300], hkv, page, d, code)
    ref.append([0, 300], slots_of(table, page, 0, 0, 300), ramp, f64(bf(rng.standard_normal((300, 1, d)))))
    dev.load(ref)
    rows = [ref.read(slots_of(table, page, 0, 0, 300))]
    for sign in (1.0, -1.0):
        q = torch.full((1, g, d), sign, dtype=torch.bfloat16, device=DEV)
        check_rows(decode_call(dev, 1, [300], table, q, scale=1.0), oracle_rows(f64(q), rows, [300], [1], 1.0), d, sign)


def test_pages_not_held_and_lengths_out_of_bounds():
    """Entries outside the cache are pages not seen; all of them gone: zeros.
    Lengths below 0 or over the bound: NaN rows, nothing else touched."""
    rng = np.random.default_rng(9)
    d, page, hkv, g = 128, 16, 2, 4
    lens = [300, 300, 40, 100]
    ref, dev, table, rows = filled(rng, lens, hkv, page, d, "e4m3")
    holes = {0: [0, 3, 4, 18], 1: list(range(19)), 3: list(range(1, 6))}
    for i, cols in holes.items():
        for c in cols:
            table[i, c] = [-1, 1 << 30, dev.k.shape[0], -(1 << 31)][c % 4]
    q = bf(rng.standard_normal((4, hkv * g, d))).to(DEV)
    out = decode_call(dev, 1, lens, table, q)
    want = []
    for i, x in enumerate(lens):
        keep = [p for p in range(x) if p // page not in holes.get(i, [])]
        o, mass, dot = C.attention(f64(q)[i:i + 1], rows[i][0][keep], rows[i][1][keep], len(keep) - 1, d ** -0.5)
        want.append((o[0], mass[0], dot[0], x))
    check_rows(out, want, d)
    assert torch.all(out[1] == 0)
    out2, cu = torch.empty_like(out), np.arange(5, dtype=np.int32)
    gdn.gdn_attn_packed(dev.handle, i32(cu), cu, i32(lens), i32(table), q, out2)
    check_rows(out2, want, d)
    ref, dev, table, rows = filled(rng, lens, hkv, page, d, "int8")
    bad = [-1, 300, 41, 1 << 30]
    out = decode_call(dev, 1, bad, table, q, max_kv=300)
    assert torch.all(out[[0, 3]].isnan())
    check_rows(out[1:2], oracle_rows(f64(q)[1:2], rows[1:2], [300], [1], d ** -0.5), d)
    gdn.gdn_attn_packed(dev.handle, i32(cu), cu, i32([-7, 300, 40, table.shape[1] * page + 1]), i32(table), q, out2)
    assert torch.all(out2[[0, 3]].isnan()) and not torch.any(out2[1:3].isnan())


def test_a_request_gives_the_same_bits_alone_and_in_any_batch():
    rng = np.random.default_rng(10)
    d, page, hkv, g = 128, 64, 2, 4
    lens = [2000, 70, 4100, 513, 1]
    ref, dev, table, rows = filled(rng, lens, hkv, page, d, "e4m3")
    q = bf(rng.standard_normal((len(lens), hkv * g, d))).to(DEV)
    out = decode_call(dev, 1, lens, table, q)
    for i, x in enumerate(lens):
        one = decode_call(dev, 1, [x], table[i:i + 1], q[i:i + 1].clone(), max_kv=x)
        assert torch.equal(one[0], out[i])
    order = [3, 1, 4, 0, 2]
    again = decode_call(dev, 1, [lens[i] for i in order], table[order], q[order].contiguous(), stream=torch.cuda.current_stream())
    assert torch.equal(again, out[order])
    new = [150, 70, 300, 13, 1]
    cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    q = bf(rng.standard_normal((sum(new), hkv * g, d))).to(DEV)
    whole = torch.empty_like(q)
    gdn.gdn_attn_packed(dev.handle, i32(cu), cu, i32(lens), i32(table), q, whole)
    for i in range(len(new)):
        part = q[cu[i]:cu[i + 1]].contiguous()
        one = torch.empty_like(part)
        gdn.gdn_attn_packed(dev.handle, i32([0, new[i]]), [0, new[i]], i32(lens[i:i + 1]), i32(table[i:i + 1]), part, one)
        assert torch.equal(one, whole[cu[i]:cu[i + 1]])


def test_addresses_past_32_bits():
    """A cache of more than 4 GiB of codes: pages at its far end."""
    rng = np.random.default_rng(11)
    d, page, hkv = 256, 128, 16
    n_pages = (1 << 32) // (hkv * page * d) + 40
    dt = torch.int8
    k = torch.empty(n_pages, hkv, page, d, dtype=dt, device=DEV)
    v = torch.empty(n_pages, hkv, page // 16, d, 16, dtype=dt, device=DEV)
    ks, vs = (torch.empty(n_pages, hkv, device=DEV) for _ in range(2))
    h = gdn.make_cache(k, v, ks, vs)
    table = np.array([[n_pages - 1, 3, n_pages - 17]], np.int32)
    T = 300
    x = bf(rng.standard_normal((T, 3 * hkv, d))).to(DEV)
    kk, vv, q = x[:, :hkv], x[:, hkv:2 * hkv], x[:, 2 * hkv:]
    slots = i64(slots_of(table, page, 0, 0, T))
    gdn.gdn_rope_append(gdn.make_rope([]), h, i32([0, T]), [0, T], None, kk, vv, None, slots, None)
    ko, vo = (torch.empty(T, hkv, d, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    gdn.gdn_cache_gather(h, slots, ko, vo)
    ref = C.PagedCache(3, hkv, page, d, "int8")
    local = slots_of(np.array([[0, 1, 2]]), page, 0, 0, T)
    ref.append([0, T], local, f64(kk), f64(vv))
    kr, vr = ref.read(local)
    np.testing.assert_array_equal(f64(ko), kr)
    np.testing.assert_array_equal(f64(vo), vr)
    pick = [0, 140, 299]
    out = torch.empty(T, hkv, d, dtype=torch.bfloat16, device=DEV)
    gdn.gdn_attn_packed(h, i32([0, T]), [0, T], i32([T]), i32(table), q, out)
    for r in pick:
        o, mass, dot = C.attention(f64(q[r:r + 1]), kr, vr, r, d ** -0.5)
        check_rows(out[r:r + 1], [(o[0], mass[0], dot[0], T)], d)


# --------------------------------------------------------- all of them --

class Server:
    """Requests on one cache: lengths, table and free pages live on the device."""

    def __init__(self, n, page, hkv, hq, d, code, n_pages, width, seed):
        self.rng = np.random.default_rng(seed)
        self.n, self.page, self.hkv, self.hq, self.d = n, page, hkv, hq, d
        self.dev = DevCache(n_pages, hkv, page, d, code)
        self.kv, self.table = i32([0] * n), torch.full((n, width), -1, dtype=torch.int32, device=DEV)
        self.free, self.count = i32(self.rng.permutation(n_pages)), i32([n_pages])
        self.freq = [float(np.float32(10000.0 ** (-i / (d // 4)))) for i in range(d // 4)]
        self.rope = gdn.make_rope(self.freq)
        self.cu, self.status = i32([0] * (n + 1)), i32([0] * n)

    def buffers(self, T):
        z = lambda h: torch.zeros(T, h, self.d, dtype=torch.bfloat16, device=DEV)
        return dict(row=torch.zeros(T, (self.hq + 2 * self.hkv) * self.d, dtype=torch.bfloat16, device=DEV), out=z(self.hq), rot=z(self.hq),
                    slots=torch.zeros(T, dtype=torch.int64, device=DEV), pos=torch.zeros(T, dtype=torch.int32, device=DEV),
                    want=torch.zeros(self.n, dtype=torch.int32, device=DEV))

    def enqueue(self, b, cu_host, n_tok=0, max_kv=0, ws=None):
        """One layer's pass: plan, rotate and write, attend."""
        T, hq, hkv, d = b["row"].shape[0], self.hq, self.hkv, self.d
        gdn.gdn_plan_pages(self.page, b["want"], self.kv, self.kv, self.table, self.free, self.count, self.count, self.cu, b["slots"],
                           b["pos"], self.status)
        q, k, v = (b["row"][:, a * d:e * d].view(T, e - a, d) for a, e in ((0, hq), (hq, hq + hkv), (hq + hkv, hq + 2 * hkv)))
        gdn.gdn_rope_append(self.rope, self.dev.handle, self.cu, cu_host, q, k, v, b["pos"], b["slots"], b["rot"])
        if n_tok:
            gdn.gdn_attn_decode(self.dev.handle, n_tok, self.kv, self.table, b["rot"], b["out"], max_kv, None, ws)
        else:
            gdn.gdn_attn_packed(self.dev.handle, self.cu, cu_host, self.kv, self.table, b["rot"], b["out"])

    def draw(self, T):
        return bf(self.rng.standard_normal((T, (self.hq + 2 * self.hkv) * self.d))).to(DEV)


def pools(server, lens):
    """What the cache holds for every request, in fp64."""
    k, v, ks, vs = server.dev.codes()
    t = server.table.cpu().numpy()
    P, out = server.page, []
    for i, x in enumerate(lens):
        pg, off = [t[i, p // P] for p in range(x)], [p % P for p in range(x)]
        out.append((k[pg, :, off] * ks[pg][:, :, None], v[pg, :, off] * vs[pg][:, :, None]))
    return out


@pytest.mark.parametrize("code,page,d", [("e4m3", 16, 128), ("int8", 64, 64), ("e4m3", 32, 256)])
def test_serving_run_prompts_decode_drafts_rejected_and_requests_ended(code, page, d):
    """Prompts in chunks, then decode steps of one and of four tokens with some
    drafted tokens rejected, an ended request's pages taken by another."""
    hkv, hq = 2, 6
    s = Server(4, page, hkv, hq, d, code, n_pages=4 * (-(-400 // page)) // 2, width=-(-400 // page), seed=page)
    lens = [0] * 4
    plan = [("packed", [100, 37, 0, 1]), ("packed", [23, 40, 5, 64]), ("decode", 1), ("decode", 4), ("reject", [2, 0, 4, 1]), ("decode", 4),
            ("end", 0), ("packed", [0, 30, 150, 3]), ("decode", 1), ("decode", 1)]
    total = s.count.item()
    for kind, arg in plan:
        if kind in ("reject", "end"):
            want = [x - r for x, r in zip(lens, arg)] if kind == "reject" else [0 if i == arg else x for i, x in enumerate(lens)]
            b = s.buffers(1)
            b["want"].copy_(i32(want))
            gdn.gdn_plan_pages(page, b["want"], s.kv, s.kv, s.table, s.free, s.count, s.count, s.cu, b["slots"], b["pos"], s.status)
            lens = want
        else:
            new = arg if kind == "packed" else [arg] * 4
            lens = [x + y for x, y in zip(lens, new)]
            T = sum(new)
            b = s.buffers(T)
            b["row"].copy_(s.draw(T))
            b["want"].copy_(i32(lens))
            cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
            most = max(lens)
            ws = torch.empty(gdn.gdn_attn_decode_workspace(s.dev.handle, hq, 4, max(1, arg if kind == "decode" else 1), most),
                             dtype=torch.uint8, device=DEV)
            s.enqueue(b, cu, arg if kind == "decode" else 0, most, ws)
            rows = pools(s, lens)
            check_rows(b["out"], oracle_rows(f64(b["rot"]), rows, lens, new, d ** -0.5), d, (kind, arg))
        torch.cuda.synchronize()
        assert s.status.cpu().tolist() == [0] * 4 and s.kv.cpu().tolist() == lens
        assert s.count.item() == total - sum(-(-x // page) for x in lens)


def test_a_captured_decode_step_follows_the_lengths():
    """Plan, rotation with the write, and attention captured once; replayed step
    after step, with eager work between, against an eager twin."""
    n, page, d, hkv, hq = 5, 16, 128, 2, 8
    twin = [Server(n, page, hkv, hq, d, "e4m3", 60, 12, seed=1) for _ in range(2)]
    start = [17, 3, 0, 60, 31]
    cu0 = np.concatenate([[0], np.cumsum(start)]).astype(np.int32)
    first = twin[0].draw(int(cu0[-1]))
    for s in twin:
        b = s.buffers(int(cu0[-1]))
        b["row"].copy_(first)
        b["want"].copy_(i32(start))
        s.enqueue(b, cu0)
    cu = np.arange(n + 1, dtype=np.int32)
    size = gdn.gdn_attn_decode_workspace(twin[0].dev.handle, hq, n, 1, 12 * page)
    bs = [s.buffers(n) for s in twin]
    ws = [torch.empty(size, dtype=torch.uint8, device=DEV) for _ in twin]
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        twin[1].enqueue(bs[1], cu, 1, 12 * page, ws[1])
    lens = list(start)
    for step in range(20):
        lens = [x + 1 for x in lens]
        row = twin[0].draw(n)
        for s, b in zip(twin, bs):
            b["row"].copy_(row)
            b["want"].copy_(i32(lens))
        twin[0].enqueue(bs[0], cu, 1, 12 * page, ws[0])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(bs[0]["out"], bs[1]["out"]) and torch.equal(bs[0]["slots"], bs[1]["slots"])
        assert torch.equal(twin[0].table, twin[1].table) and torch.equal(twin[0].kv, twin[1].kv)
        assert torch.equal(twin[0].dev.k.view(torch.uint8), twin[1].dev.k.view(torch.uint8))
    assert twin[1].kv.cpu().tolist() == lens


def test_two_streams_at_once():
    """Two caches, two workspaces, two streams at the same time: each as alone."""
    rng = np.random.default_rng(12)
    got, alone = [], []
    streams = [torch.cuda.Stream() for _ in range(2)]
    sides = []
    for i in range(2):
        lens = [1500, 300 + i, 64]
        ref, dev, table, rows = filled(rng, lens, 2, 16, 128, "int8")
        q = bf(rng.standard_normal((3, 8, 128))).to(DEV)
        size = gdn.gdn_attn_decode_workspace(dev.handle, 8, 3, 1, 1504)
        sides.append((dev, i32(lens), i32(table), q, torch.empty(size, dtype=torch.uint8, device=DEV)))
        alone.append(decode_call(dev, 1, lens, table, q))
    torch.cuda.synchronize()
    for rep in range(5):
        outs = [torch.empty_like(s[3]) for s in sides]
        torch.cuda.synchronize()
        for (dev, lens, table, q, ws), st, o in zip(sides, streams, outs):
            gdn.gdn_attn_decode(dev.handle, 1, lens, table, q, o, 1504, None, ws, stream=st)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, alone))

"""The operators of the paged 8-bit key/value cache: page planning, rotary positions with the cache's write,
the cache's read back, and attention over it for decoding requests and for packed prompts.

``listed`` and ``draw`` give cases, ``prepare`` a case's inputs, ``run`` one pass: in elementary torch
operations, or, where ``own`` is set, through the library's entry points.
"""
import math
import random

import numpy as np
import torch

own = False

DEV = "cuda"
S_MIN = 2.0 ** -100          # scale of a page that holds only zeros
MAXCODE = {"e4m3": 448.0, "int8": 127.0}


# ------------------------------------------------------------------ cases --

def listed():
    """Head counts 16 and 32 and head size 128 are the layer geometry of this repository's workloads, as are
    the chat wave (32 x 1,024 tokens), the long prompts (4 x 8,192), ragged prompts of 17 to 2,048 tokens and
    passes of 1,024 prompt tokens beside 32 decoding requests; head sizes 64 and 256 and the pages are generic."""
    return [
        # a decode step's bookkeeping: every request grows by one token, a few have ended
        dict(name="pages decode step", op="plan", n=64, lo=17, hi=2048, new_lo=1, new_hi=1, fresh=0, done=4, page=16, mix=1),
        # admission of a chat wave beside running requests: fresh prompts get all their pages, others grow by one
        dict(name="pages chat wave", op="plan", n=512, lo=17, hi=8192, new_lo=1024, new_hi=1024, fresh=32, done=16, page=64, mix=2),
        # one decode step's keys and values: latency
        dict(name="append decode step", op="append", n=64, ctx_lo=17, ctx_hi=2048, new_lo=1, new_hi=1, hq=32, hkv=8, d=128,
             rot=64, axes=3, adjacent=False, page=16, code="e4m3", mix=3),
        # prompt chunks that continue cached prefixes in the middle of a page
        dict(name="append ragged pass", op="append", n=8, ctx_lo=0, ctx_hi=1024, new_lo=64, new_hi=512, hq=16, hkv=4, d=256,
             rot=64, axes=1, adjacent=True, page=32, code="int8", mix=4),
        # the chat wave's prompts, image positions on three axes
        dict(name="append chat wave", op="append", n=32, ctx_lo=0, ctx_hi=0, new_lo=1024, new_hi=1024, hq=32, hkv=8, d=128,
             rot=128, axes=3, adjacent=False, page=64, code="e4m3", mix=5),
        # one prompt's prefix moved out of the cache
        dict(name="read one prefix", op="gather", n=1, lo=1000, hi=1000, hkv=8, d=128, page=16, code="int8", mix=6),
        # the long prompts moved out of the cache
        dict(name="read long prompts", op="gather", n=4, lo=8192, hi=8192, hkv=8, d=128, page=64, code="e4m3", mix=7),
        # one user alone: the smallest decode call
        dict(name="decode one request", op="decode", n=1, lo=1000, hi=1000, n_tok=1, hq=16, hkv=4, d=128, page=16, code="int8", mix=8),
        # a decode batch in mid-flight
        dict(name="decode ragged batch", op="decode", n=32, lo=17, hi=8192, n_tok=1, hq=32, hkv=8, d=128, page=64, code="e4m3", mix=9),
        # verification of drafted tokens on long contexts, wide heads
        dict(name="decode 4 tokens long", op="decode", n=16, lo=4096, hi=32768, n_tok=4, hq=16, hkv=2, d=256, page=128, code="int8", mix=10),
        # ragged prompts that continue prefixes found in the cache
        dict(name="prompts on prefixes", op="packed", n=8, ctx_lo=0, ctx_hi=4096, new_lo=17, new_hi=2048, hq=32, hkv=8, d=128, page=64, code="e4m3", mix=11),
        # the long prompts, whole
        dict(name="long prompts", op="packed", n=4, ctx_lo=0, ctx_hi=0, new_lo=8192, new_hi=8192, hq=16, hkv=4, d=128, page=64, code="int8", mix=12),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["plan", "append", "gather", "decode", "decode", "packed"])
    page, mix = rng.choice([16, 32, 64, 128]), rng.randrange(1 << 20)
    code, d = rng.choice(["e4m3", "int8"]), rng.choice([64, 128, 128, 256])
    hkv = rng.choice([1, 2, 3, 4, 8])
    hq = hkv * rng.choice([1, 2, 3, 4, 5, 6, 8])
    if op == "plan":
        n = _log(rng, 1, 512)
        fresh = rng.randrange(0, min(n, 32) + 1)
        return dict(op=op, n=n, lo=1, hi=_log(rng, 64, 8192), new_lo=1, new_hi=_log(rng, 1, 1024), fresh=fresh,
                    done=rng.randrange(0, n - fresh + 1), page=page, mix=mix)
    if op == "append":
        axes = rng.choice([1, 3])
        n = _log(rng, 1, 64)
        hi = _log(rng, 1, 8192 // n)
        return dict(op=op, n=n, ctx_lo=0, ctx_hi=_log(rng, 1, 2048), new_lo=rng.randint(1, hi), new_hi=hi, hq=hq, hkv=hkv, d=d,
                    rot=rng.choice([d // 4, d // 2, d]), axes=axes, adjacent=rng.random() < 0.5, page=page, code=code, mix=mix)
    if op == "gather":
        n = _log(rng, 1, 16)
        hi = _log(rng, 1, 16384 // n)
        return dict(op=op, n=n, lo=rng.randint(1, hi), hi=hi, hkv=hkv, d=d, page=page, code=code, mix=mix)
    if op == "decode":
        n = _log(rng, 1, 64)
        hi = _log(rng, 16, min(32768, 262144 // (n * max(1, hkv * d // 512))))
        return dict(op=op, n=n, lo=rng.randint(1, hi), hi=hi, n_tok=rng.choice([1, 1, 1, 2, 3, 4]), hq=hq, hkv=hkv, d=d, page=page,
                    code=code, mix=mix)
    n = _log(rng, 1, 8)
    hi = _log(rng, 17, 2048)
    return dict(op=op, n=n, ctx_lo=0, ctx_hi=_log(rng, 1, 4096), new_lo=rng.randint(1, hi), new_hi=hi, hq=hq, hkv=hkv, d=d, page=page,
                code=code, mix=mix)


def _lengths(case):
    """(length held before, length wanted) of each request, from the case alone."""
    r, n, op = random.Random(case["mix"]), case["n"], case["op"]
    if op == "plan":
        kv = [r.randint(case["lo"], case["hi"]) for _ in range(n)]
        want = [x + 1 for x in kv]
        order = r.sample(range(n), n)
        for i in order[:case["fresh"]]:
            kv[i], want[i] = 0, r.randint(case["new_lo"], case["new_hi"])
        for i in order[case["fresh"]:case["fresh"] + case["done"]]:
            want[i] = 0
        return kv, want
    if op in ("append", "packed"):
        kv = [r.randint(case["ctx_lo"], case["ctx_hi"]) for _ in range(n)]
        return kv, [x + r.randint(case["new_lo"], case["new_hi"]) for x in kv]
    n_tok = case.get("n_tok", 0)
    want = [max(n_tok, r.randint(case["lo"], case["hi"])) for _ in range(n)]
    return [x - n_tok for x in want], want


def _pages(x, page):
    return -(-x // page)


# ----------------------------------------------------------------- inputs --

def _scale_of(amax, code):
    """The smallest power of two at or above amax / maxcode."""
    m, e = torch.frexp(amax.float())                 # amax = m 2^e, 1/2 <= m < 1
    top, te = math.frexp(MAXCODE[code])
    s = torch.ldexp(torch.ones_like(m), e - te + (m > top).to(e.dtype))
    return torch.where(amax > 0, s.clamp(min=S_MIN), torch.full_like(s, S_MIN))


def _to_codes(x, code):
    x = torch.nan_to_num(x, nan=0.0 if code == "int8" else float("nan"), posinf=MAXCODE[code], neginf=-MAXCODE[code])
    x = x.clamp(-MAXCODE[code], MAXCODE[code])
    return x.round().to(torch.int8) if code == "int8" else x.to(torch.float8_e4m3fn)


def _cache(g, case, kv, want):
    """A cache whose requests hold kv tokens (each page quantised with its own scale) and have pages for `want`,
    the pages dealt out in a random order; every 16th channel of the keys is eight times the others."""
    n, page, hkv, d, code = case["n"], case["page"], case["hkv"], case["d"], case["code"]
    need = [_pages(w, page) for w in want]
    m = max(max(need), 1)
    n_pages = sum(need) + 3
    perm = torch.randperm(n_pages, generator=g, device=DEV)
    rows = torch.full((n, m), -1, dtype=torch.int32, device=DEV)
    held = torch.arange(m, device=DEV)[None, :] < torch.tensor(need, device=DEV)[:, None]
    rows[held] = perm[:sum(need)].to(torch.int32)
    chan = torch.ones(d, device=DEV)
    chan[::16] = 8.0
    k = torch.randn(n_pages, hkv, page, d, generator=g, device=DEV, dtype=torch.float32) * chan
    v = torch.randn(n_pages, hkv, page, d, generator=g, device=DEV, dtype=torch.float32)
    ks, vs = _scale_of(k.abs().amax((2, 3)), code), _scale_of(v.abs().amax((2, 3)), code)
    kc = _to_codes(k / ks[:, :, None, None], code)
    vc = _to_codes(v / vs[:, :, None, None], code)
    vc = vc.reshape(n_pages, hkv, page // 16, 16, d).transpose(3, 4).contiguous()
    return dict(k=kc, v=vc, ks=ks, vs=vs, table=rows, page=page, code=code)


def _slots(table, kv, want, page):
    """slot and index of every new token (requests one after the other)."""
    new = torch.tensor([w - x for x, w in zip(kv, want)], device=DEV)
    first = torch.tensor(kv, device=DEV)
    who = torch.repeat_interleave(torch.arange(len(kv), device=DEV), new)
    start = torch.cumsum(new, 0) - new
    pos = torch.arange(int(sum(want) - sum(kv)), device=DEV) - start[who] + first[who]
    return table[who, pos // page].long() * page + pos % page, pos


def _rope_plan(case):
    """freq and axis of every pair: base 10,000, the axes dealt out in turn (first, second, third, first, ...)."""
    half = case["rot"] // 2
    freq = [float(torch.tensor(10000.0 ** (-i / half), dtype=torch.float32)) for i in range(half)]
    return freq, [i % case["axes"] for i in range(half)]


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    kv, want = _lengths(case)
    n, page, op = case["n"], case["page"], case["op"]
    s = dict(case=case, op=op)
    if op == "plan":
        now, need = [_pages(x, page) for x in kv], [_pages(w, page) for w in want]
        m = max(max(now), max(need)) + 2
        n_pages = sum(max(a, b) for a, b in zip(now, need)) + 64
        perm = torch.randperm(n_pages, generator=g, device=DEV).to(torch.int32)
        table = torch.full((n, m), -1, dtype=torch.int32, device=DEV)
        table[torch.arange(m, device=DEV)[None, :] < torch.tensor(now, device=DEV)[:, None]] = perm[:sum(now)]
        free = torch.zeros(n_pages, dtype=torch.int32, device=DEV)
        free[:n_pages - sum(now)] = perm[sum(now):]
        total = sum(max(0, w - x) for x, w in zip(kv, want))
        s.update(want=_i32(want), kv=_i32(kv), table=table, free=free, count=_i32([n_pages - sum(now)]),
                 total=total, kv_out=torch.empty(n, dtype=torch.int32, device=DEV),
                 count_out=torch.empty(1, dtype=torch.int32, device=DEV),
                 cu=torch.empty(n + 1, dtype=torch.int32, device=DEV), status=torch.empty(n, dtype=torch.int32, device=DEV),
                 slots=torch.empty(total, dtype=torch.int64, device=DEV), pos=torch.empty(total, dtype=torch.int32, device=DEV))
        return s
    hkv, d = case["hkv"], case["d"]
    s["cache"] = c = _cache(g, case, kv, want)
    if op == "gather":
        s["slots"], _ = _slots(c["table"], [0] * n, want, page)
        t = s["slots"].numel()
        s["k_out"] = torch.empty(t, hkv, d, dtype=torch.bfloat16, device=DEV)
        s["v_out"] = torch.empty(t, hkv, d, dtype=torch.bfloat16, device=DEV)
        return s
    hq = case["hq"]
    new = [w - x for x, w in zip(kv, want)]
    cu = [0]
    for x in new:
        cu.append(cu[-1] + x)
    t = cu[-1]
    s.update(kv_len=_i32(want), cu=_i32(cu), cu_host=np.array(cu, dtype=np.int32), n_max=max(new), max_kv=max(want),
             q=torch.randn(t, hq, d, generator=g, device=DEV).bfloat16(), out=torch.empty(t, hq, d, dtype=torch.bfloat16, device=DEV))
    if op != "append":
        return s
    chan = torch.ones(d, device=DEV)
    chan[::16] = 8.0
    # one row of q, k and v per token, as a merged projection gives them
    row = torch.empty(t, (hq + 2 * hkv) * d, dtype=torch.bfloat16, device=DEV)
    row[:, :hq * d] = s["q"].reshape(t, -1)
    row[:, hq * d:(hq + hkv) * d] = (torch.randn(t, hkv, d, generator=g, device=DEV) * chan).reshape(t, -1)
    row[:, (hq + hkv) * d:] = torch.randn(t, hkv * d, generator=g, device=DEV)
    s["q"] = row[:, :hq * d].view(t, hq, d)
    s["k"] = row[:, hq * d:(hq + hkv) * d].view(t, hkv, d)
    s["v"] = row[:, (hq + hkv) * d:].view(t, hkv, d)
    s["slots"], pos = _slots(c["table"], kv, want, page)
    # text positions on every axis, then an offset for the further ones as inside an image
    s["pos"] = torch.stack([pos + (0 if a == 0 else torch.randint(0, 32, (t,), generator=g, device=DEV))
                            for a in range(case["axes"])]).to(torch.int32)
    freq, axis = _rope_plan(case)
    s["freq_host"], s["axis_host"] = freq, axis
    s["freq"], s["axis"] = torch.tensor(freq, dtype=torch.float64, device=DEV), torch.tensor(axis, device=DEV)
    s["runs"] = sum(_pages(w, page) - x // page for x, w in zip(kv, want))
    # every slot of the pages that the call touches up to the requests' lengths: what it may have changed
    s["touched"], _ = _slots(c["table"], [x // page * page for x in kv], want, page)
    tt = s["touched"].numel()
    s["k_out"] = torch.empty(tt, hkv, d, dtype=torch.bfloat16, device=DEV)
    s["v_out"] = torch.empty(tt, hkv, d, dtype=torch.bfloat16, device=DEV)
    return s


# --------------------------------------------------- the library's calls --

_lib = None


def _gdn():
    global _lib
    if _lib is None:
        import gated_deltanet_prefill_varlen_amd as lib
        _lib = lib
    return _lib


def _handle(s):
    """The cache's handle, the rotary plan's, the decode step's workspace: made once, kept by the program."""
    if "handle" not in s:
        gdn, c, case = _gdn(), s["cache"], s["case"]
        s["handle"] = gdn.make_cache(c["k"], c["v"], c["ks"], c["vs"])
        if s["op"] == "append":
            s["rope"] = gdn.make_rope(s["freq_host"], s["axis_host"], n_axes=case["axes"], adjacent=case["adjacent"])
        if s["op"] == "decode":
            size = gdn.gdn_attn_decode_workspace(s["handle"], case["hq"], case["n"], case["n_tok"], s["max_kv"])
            s["workspace"] = torch.empty(size, dtype=torch.uint8, device=DEV)
    return s["handle"]


def _run_own(s):
    gdn, op = _gdn(), s["op"]
    if op == "plan":
        gdn.gdn_plan_pages(s["case"]["page"], s["want"], s["kv"], s["kv_out"], s["table"], s["free"], s["count"], s["count_out"],
                           s["cu"], s["slots"], s["pos"], s["status"])
        return [s["kv_out"], s["count_out"], s["cu"], s["status"], s["table"], s["free"], s["slots"], s["pos"]]
    h = _handle(s)
    if op == "append":
        gdn.gdn_rope_append(s["rope"], h, s["cu"], s["cu_host"], s["q"], s["k"], s["v"], s["pos"], s["slots"], s["out"])
        gdn.gdn_cache_gather(h, s["touched"], s["k_out"], s["v_out"])
        return [s["out"], s["k_out"], s["v_out"], s["cache"]["ks"], s["cache"]["vs"]]
    if op == "gather":
        gdn.gdn_cache_gather(h, s["slots"], s["k_out"], s["v_out"])
        return [s["k_out"], s["v_out"]]
    if op == "decode":
        gdn.gdn_attn_decode(h, s["case"]["n_tok"], s["kv_len"], s["cache"]["table"], s["q"], s["out"], max_kv_len=s["max_kv"],
                            workspace=s["workspace"])
        return [s["out"]]
    gdn.gdn_attn_packed(h, s["cu"], s["cu_host"], s["kv_len"], s["cache"]["table"], s["q"], s["out"])
    return [s["out"]]


# --------------------------------------------------------- the plain form --

def _run_plan(s):
    page, want, kv, table, n = s["case"]["page"], s["want"].long(), s["kv"].long(), s["table"], s["case"]["n"]
    n_pages, m = s["free"].numel(), table.shape[1]
    count = s["count"].long()
    have, need = (kv + page - 1) // page, (want + page - 1) // page
    cols = torch.arange(m, device=DEV)[None, :]
    # ended or shortened requests: their pages onto the stack, in request order
    back = (have - need).clamp(min=0)
    total_back = back.sum()
    at = count + (torch.cumsum(back, 0) - back)[:, None] + cols - need[:, None]
    gone = (cols >= need[:, None]) & (cols < have[:, None])
    free = torch.cat([s["free"], s["free"].new_zeros(1)])
    free = free.scatter(0, torch.where(gone, at, n_pages).reshape(-1), table.reshape(-1))[:n_pages]
    # grown requests: their pages from the top
    more = (need - have).clamp(min=0)
    upto = torch.cumsum(more, 0)
    left = count + total_back
    fits = want <= m * page
    ok = (want <= kv) | (fits & ((more == 0) | (upto <= left)))
    kv_out = torch.where(ok, want, kv)
    got = (cols >= have[:, None]) & (cols < need[:, None]) & ok[:, None]
    src = (left - 1 - (upto - more)[:, None] - (cols - have[:, None])).clamp(0, n_pages - 1)
    table = torch.where(got, free[src], table)
    count_out = left - torch.where(ok, more, 0).sum()
    # the pack of the new tokens
    new = (want - kv).clamp(min=0)
    cu = torch.cat([new.new_zeros(1), torch.cumsum(new, 0)])
    who = torch.repeat_interleave(torch.arange(n, device=DEV), new, output_size=s["total"])
    pos = torch.arange(s["total"], device=DEV) - cu[who] + kv[who]
    slots = torch.where(ok[who], table[who, pos // page].long() * page + pos % page, -1)
    i32 = torch.int32
    return [kv_out.to(i32), count_out.to(i32), cu.to(i32), torch.where(ok, 0, torch.where(fits, 1, 2)).to(i32), table, free, slots, pos.to(i32)]


def _rotate(x, cos, sin, rot, adjacent):
    x = x.float()
    cos, sin = cos[:, None, :], sin[:, None, :]
    if adjacent:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
    return torch.cat([y, x[..., rot:]], -1).bfloat16()


def _write(codes, scale, x, rid, off, first, code):
    """Pages (codes [U, Hkv, P, d] as fp32, scales [U, Hkv]) with the tokens x [T, Hkv, d] written at [rid, :, off]."""
    x = x.float()
    finite = torch.where(x.isfinite(), x.abs(), 0.0).amax(-1)
    amax = torch.zeros_like(scale).scatter_reduce(0, rid[:, None].expand_as(finite), finite, "amax")
    old = torch.where((first == 0)[:, None] | ~(scale >= S_MIN), S_MIN, scale)
    now = torch.maximum(old, _scale_of(amax, code))
    held = torch.arange(codes.shape[2], device=DEV)[None, :] < first[:, None]
    again = _to_codes(codes * (old / now)[:, :, None, None], code).float()
    codes = torch.where(held[:, None, :, None], again, codes)
    codes[rid, :, off] = _to_codes(x / now[rid][..., None], code).float()
    return codes, now


def _run_append(s):
    case, c = s["case"], s["cache"]
    page, code, rot, adjacent = case["page"], case["code"], case["rot"], case["adjacent"]
    ang = s["pos"][s["axis"]].t().double() * s["freq"]
    cos, sin = ang.cos().float(), ang.sin().float()
    q = _rotate(s["q"], cos, sin, rot, adjacent)
    k = _rotate(s["k"], cos, sin, rot, adjacent)
    pages, off = s["slots"] // page, s["slots"] % page
    lead = torch.cat([pages.new_ones(1), (pages[1:] != pages[:-1]).long()])
    rid = torch.cumsum(lead, 0) - 1
    u = pages.new_zeros(s["runs"]).scatter(0, rid, pages)
    first = torch.full_like(u, page).scatter_reduce(0, rid, off, "amin")
    hkv, d = case["hkv"], case["d"]
    kind = c["k"].dtype
    kc, ks = _write(c["k"].view(torch.uint8)[u].view(kind).float(), c["ks"][u], k, rid, off, first, code)
    vc = c["v"].view(torch.uint8)[u].view(kind).float().transpose(3, 4).reshape(-1, hkv, page, d)
    vc, vs = _write(vc, c["vs"][u], s["v"], rid, off, first, code)
    c["k"].view(torch.uint8)[u] = kc.to(kind).view(torch.uint8)
    c["v"].view(torch.uint8)[u] = vc.reshape(-1, hkv, page // 16, 16, d).transpose(3, 4).contiguous().to(kind).view(torch.uint8)
    c["ks"][u], c["vs"][u] = ks, vs
    return [q, *_gathered(c, s["touched"]), c["ks"], c["vs"]]


def _gathered(c, slots):
    page = c["page"]
    p, o = slots // page, slots % page
    k = c["k"].view(torch.uint8)[p, :, o].view(c["k"].dtype).float() * c["ks"][p][..., None]
    v = c["v"].view(torch.uint8)[p, :, o // 16, :, o % 16].view(c["v"].dtype).float() * c["vs"][p][..., None]
    return k.bfloat16(), v.bfloat16()


def _held(c, dtype):
    """Keys and values [n, Hkv, M * P, d] of every request, from its pages."""
    t = c["table"].clamp(min=0).long()
    n, m = t.shape
    k = c["k"].view(torch.uint8)[t].view(c["k"].dtype).to(dtype) * c["ks"][t][..., None, None].to(dtype)
    v = c["v"].view(torch.uint8)[t].view(c["v"].dtype).to(dtype) * c["vs"][t][..., None, None, None].to(dtype)
    hkv, page, d = k.shape[2:]
    v = v.transpose(4, 5).reshape(n, m, hkv, page, d)
    return k.transpose(1, 2).reshape(n, hkv, m * page, d), v.transpose(1, 2).reshape(n, hkv, m * page, d)


def _run_attn(s):
    case = s["case"]
    hq, hkv, d, n = case["hq"], case["hkv"], case["d"], case["n"]
    k, v = _held(s["cache"], torch.float32)
    cu, kv_len, rows = s["cu"].long(), s["kv_len"].long(), s["n_max"]
    new = cu[1:] - cu[:-1]
    i = torch.arange(rows, device=DEV)[None, :]
    at = (cu[:-1, None] + torch.minimum(i, new[:, None] - 1).clamp(min=0))
    q = s["q"][at].float().reshape(n, rows, hkv, hq // hkv, d).permute(0, 2, 3, 1, 4).reshape(n, hkv, -1, d)
    p = torch.matmul(q * d ** -0.5, k.transpose(2, 3).contiguous())
    last = (kv_len - new)[:, None] + i                                      # the last key that row i sees
    seen = torch.arange(k.shape[2], device=DEV)[None, None, :] <= last[:, :, None]
    p = p.reshape(n, hkv, hq // hkv, rows, -1).masked_fill_(~seen[:, None, None], float("-inf"))
    p = p.sub_(p.amax(-1, keepdim=True)).exp_()
    p = p.div_(p.sum(-1, keepdim=True)).reshape(n, hkv, -1, k.shape[2])
    o = torch.matmul(p, v).reshape(n, hkv, hq // hkv, rows, d).permute(0, 3, 1, 2, 4).reshape(n, rows, hq, d)
    return [o[i < new[:, None]].bfloat16()]


def run(state):
    if own:
        return _run_own(state)
    op = state["op"]
    if op == "plan":
        return _run_plan(state)
    if op == "append":
        return _run_append(state)
    if op == "gather":
        return list(_gathered(state["cache"], state["slots"]))
    return _run_attn(state)


# ------------------------------------------------------------------- work --

def work(case):
    kv, want = _lengths(case)
    n, page, op = case["n"], case["page"], case["op"]
    new = [max(0, w - x) for x, w in zip(kv, want)]
    t = sum(new)
    if op == "plan":
        moved = sum(abs(_pages(w, page) - _pages(x, page)) for x, w in zip(kv, want))
        return {"bytes": 4 * (2 * n + 3 * n + 2) + 8 * moved + 12 * t, "flops": 0}
    hkv, d = case["hkv"], case["d"]
    if op == "gather":
        return {"bytes": sum(want) * (hkv * d * 6 + 8), "flops": 2 * sum(want) * hkv * d}
    hq = case["hq"]
    if op == "append":
        held = sum(w - x // page * page for x, w in zip(kv, want))
        write = t * ((2 * hq + 2 * hkv) * d * 2 + 2 * hkv * d + 4 * case["axes"] + 8)
        return {"bytes": write + held * (hkv * d * 6 + 8), "flops": 6 * t * (hq + hkv) * case["rot"] // 2}
    pairs = sum(x * m + m * (m + 1) // 2 for x, m in zip(kv, new))
    held = sum(want) * 2 * hkv * d + sum(_pages(w, page) for w in want) * (8 * hkv + 4)
    return {"bytes": held + 4 * t * hq * d, "flops": 4 * d * hq * pairs}


# ------------------------------------------------------------------ exact --

def exact(case, seed):
    """The operators' definition in 64 bits, request by request."""
    op = case["op"]
    if op == "plan":
        return None                                    # whole numbers only
    s = prepare(case, seed)
    c, page = s["cache"], case["page"]
    kv, want = _lengths(case)
    hkv, d = case["hkv"], case["d"]

    def held(r, upto):
        """codes as numbers [upto, Hkv, d] and scales [upto, Hkv] of request r's first tokens, in 64 bits."""
        t = c["table"][r, :_pages(upto, page)].long()
        k = c["k"].view(torch.uint8).index_select(0, t).view(c["k"].dtype).double()
        v = c["v"].view(torch.uint8).index_select(0, t).view(c["v"].dtype).double()
        k = k.permute(0, 2, 1, 3).reshape(-1, hkv, d)[:upto]
        v = v.permute(0, 2, 4, 1, 3).reshape(-1, hkv, d)[:upto]
        ks = c["ks"].double()[t].repeat_interleave(page, 0)[:upto]
        vs = c["vs"].double()[t].repeat_interleave(page, 0)[:upto]
        return k, v, ks, vs

    if op == "gather":
        got = [held(r, w) for r, w in enumerate(want)]
        return [torch.cat([k * ks[..., None] for k, _, ks, _ in got]), torch.cat([v * vs[..., None] for _, v, _, vs in got])]
    hq = case["hq"]
    if op in ("decode", "packed"):
        if work(case)["flops"] > 4e12:
            return None
        out = torch.empty(s["q"].shape, dtype=torch.float64, device=DEV)
        for r, (x, w) in enumerate(zip(kv, want)):
            k, v, ks, vs = held(r, w)
            k, v = k * ks[..., None], v * vs[..., None]
            rows = slice(int(s["cu_host"][r]), int(s["cu_host"][r + 1]))
            hidden = torch.arange(w, device=DEV)[None, :] > torch.arange(x, w, device=DEV)[:, None]
            for h in range(hq):
                kh, vh = k[:, h // (hq // hkv)], v[:, h // (hq // hkv)]
                a = s["q"][rows, h].double() @ kh.t().contiguous() / math.sqrt(d)
                a[hidden] = -math.inf
                out[rows, h] = torch.softmax(a, -1) @ vh
        return [out]
    # append: rotation by a complex factor, then page by page
    rot, half, code = case["rot"], case["rot"] // 2, case["code"]
    where = s["pos"].double()[s["axis"]].t() * s["freq"]                        # [T, half]
    turn = torch.polar(torch.ones_like(where), where)[:, None, :]

    def rotated(x):
        y = x.double().clone()
        lo = slice(0, rot, 2) if case["adjacent"] else slice(0, half)
        hi = slice(1, rot, 2) if case["adjacent"] else slice(half, rot)
        z = torch.complex(y[..., lo].contiguous(), y[..., hi].contiguous()) * turn
        y[..., lo], y[..., hi] = z.real, z.imag
        return y

    top = MAXCODE[code]

    def stored(x, step):
        y = x / step
        return (y.round() if code == "int8" else y.float().to(torch.float8_e4m3fn).double()) * step

    q_out, k_new, v_new = rotated(s["q"]), rotated(s["k"]).bfloat16().double(), s["v"].double()
    k_all, v_all = [], []
    ks_all, vs_all = c["ks"].double().clone(), c["vs"].double().clone()
    for r, (x, w) in enumerate(zip(kv, want)):
        k, v, ks, vs = held(r, w)
        rows = slice(int(s["cu_host"][r]), int(s["cu_host"][r + 1]))
        lo = x // page * page
        n_p = _pages(w, page) - x // page
        t = c["table"][r, x // page:_pages(w, page)].long()
        for new_rows, codes, sc, keep, into in ((k_new[rows], k, ks, k_all, ks_all), (v_new[rows], v, vs, v_all, vs_all)):
            values = torch.cat([(codes * sc[..., None])[lo:x], new_rows])       # [w - lo, Hkv, d]
            fresh = torch.cat([torch.zeros_like(values[:x - lo]), new_rows]).abs()
            pad = torch.zeros(n_p * page - values.shape[0], hkv, d, dtype=torch.float64, device=DEV)
            most = torch.cat([fresh, pad]).reshape(n_p, page, hkv, d).amax((1, 3))
            step = torch.exp2(torch.ceil(torch.log2((most / top).clamp(min=2.0 ** -100))))
            if x % page:
                step[0] = torch.maximum(step[0], sc[lo])
            per = step.repeat_interleave(page, 0)[:values.shape[0], :, None]
            keep.append(stored(values, per))
            into[t] = step
    return [q_out, torch.cat(k_all), torch.cat(v_all), ks_all, vs_all]

"""fp64 definitions of the paged 8-bit key/value cache's operators, written
token by token and request by request: codes and scales, the cache's write and
read, rotary positions, the page planner and causal attention.  Shares no code
with the library."""
from __future__ import annotations

import math

import numpy as np

from .gdn_oracle import round_bf16

MIN_SCALE = 2.0 ** -100
TOP = {"e4m3": 448.0, "int8": 127.0}


def e4m3_value(code: int) -> float:
    """Sign, 4 exponent bits (bias 7), 3 fraction bits; 0x7F and 0xFF are NaN."""
    sign = -1.0 if code & 0x80 else 1.0
    e, f = (code >> 3) & 15, code & 7
    if e == 15 and f == 7:
        return math.nan
    return sign * (f * 2.0 ** -9 if e == 0 else (8 + f) * 2.0 ** (e - 10))


_E4M3 = np.array([e4m3_value(c) for c in range(127)])          # 0 .. 448, ascending


def code_round(x: np.ndarray, code: str) -> np.ndarray:
    """x (already divided by its scale) as the value of its code: nearest, ties
    to the even code, infinities the largest; NaN: NaN (e4m3) or 0 (int8)."""
    x = np.asarray(x, np.float64)
    a = np.minimum(np.abs(np.where(np.isnan(x), 0.0, x)), TOP[code])
    if code == "int8":
        return np.copysign(np.rint(a), np.where(np.isnan(x), 0.0, x))
    hi = np.clip(np.searchsorted(_E4M3, a, side="left"), 1, 126)
    lo = hi - 1
    down, up = a - _E4M3[lo], _E4M3[hi] - a
    pick = np.where(down < up, lo, np.where(up < down, hi, np.where(lo % 2 == 0, lo, hi)))
    return np.where(np.isnan(x), np.nan, np.copysign(_E4M3[pick], x))


def scale_for(amax: float, code: str) -> float:
    """The smallest power of two s >= 2^-100 with amax <= s * largest code."""
    s = MIN_SCALE
    while amax > s * TOP[code]:
        s *= 2.0
    return s


class PagedCache:
    """Codes as numbers and scales, [n_pages, Hkv, page, d] and [n_pages, Hkv]."""

    def __init__(self, n_pages, hkv, page, d, code):
        self.page, self.code = page, code
        self.k = np.zeros((n_pages, hkv, page, d))
        self.v = np.zeros((n_pages, hkv, page, d))
        self.ks = np.full((n_pages, hkv), MIN_SCALE)
        self.vs = np.full((n_pages, hkv), MIN_SCALE)

    def _put(self, codes, scales, pg, h, first, rows):
        """rows: {offset: values [d]} written at once into one page and head."""
        amax = max((np.max(np.abs(np.where(np.isfinite(x), x, 0.0))) for x in rows.values()), default=0.0)
        old = MIN_SCALE if first == 0 else scales[pg, h]
        new = max(old, scale_for(float(amax), self.code))
        for o in range(first):
            if new > old:
                codes[pg, h, o] = code_round(codes[pg, h, o] * (old / new), self.code)
        for o, x in rows.items():
            codes[pg, h, o] = code_round(x / new, self.code)
        scales[pg, h] = new

    def append(self, cu, slots, k, v):
        """k, v [T, Hkv, d] (k already rotated) at slots, prompt by prompt and
        page by page; slots that break their page's run are not written."""
        P = self.page
        for s in range(len(cu) - 1):
            t = cu[s]
            if t == cu[s + 1]:
                continue
            off = int(slots[t]) % P if slots[t] >= 0 else 0
            while t < cu[s + 1]:
                n = min(P - off, cu[s + 1] - t)
                lead = int(slots[t])
                if lead >= 0 and lead % P == off and lead // P < self.k.shape[0]:
                    ok = [i for i in range(n) if slots[t + i] == lead + i]
                    for h in range(k.shape[1]):
                        self._put(self.k, self.ks, lead // P, h, off, {off + i: k[t + i, h] for i in ok})
                        self._put(self.v, self.vs, lead // P, h, off, {off + i: v[t + i, h] for i in ok})
                t += n
                off = 0

    def read(self, slots):
        P = self.page
        k = np.zeros((len(slots),) + (self.k.shape[1], self.k.shape[3]))
        v = np.zeros_like(k)
        for t, s in enumerate(slots):
            if 0 <= s < self.k.shape[0] * P:
                k[t] = self.k[s // P, :, s % P] * self.ks[s // P][:, None]
                v[t] = self.v[s // P, :, s % P] * self.vs[s // P][:, None]
        return k, v


def rotate(x, pos, freq, axis, adjacent=False, scale=1.0):
    """x [T, H, d] turned by the positions pos [n_axes, T]."""
    y = np.array(x, np.float64)
    half = len(freq)
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if adjacent else (i, i + half)
        ang = pos[axis[i]].astype(np.float64) * float(freq[i])
        c, s = scale * np.cos(ang)[:, None], scale * np.sin(ang)[:, None]
        y[:, :, a] = x[:, :, a] * c - x[:, :, b] * s
        y[:, :, b] = x[:, :, a] * s + x[:, :, b] * c
    return y


def plan_pages(page, want, kv, table, free, n_pages, slot_cap):
    """One request after the other.  table: list of lists (entries of held
    pages), free: the stack.  Returns (kv_out, table, free, cu, slots,
    positions, status)."""
    n, m = len(want), len(table[0]) if len(table) else 0
    pages = lambda x: -(-x // page)
    table, free, kv_out, status = [list(r) for r in table], list(free), list(kv), [0] * n
    for i in range(n):
        if want[i] < 0 or kv[i] < 0 or kv[i] > m * page:
            status[i] = 3
        elif want[i] > m * page:
            status[i] = 2
        elif want[i] < kv[i]:
            free += table[i][pages(want[i]):pages(kv[i])]
            kv_out[i] = want[i]
    new = [0 if status[i] == 3 else max(0, want[i] - kv[i]) for i in range(n)]
    cu = [0]
    for x in new:
        cu.append(cu[-1] + x)
    there, asked = len(free), 0
    for i in range(n):
        if status[i] or want[i] <= kv[i]:
            continue
        if cu[i + 1] > slot_cap:
            status[i] = 4
            continue
        more = pages(want[i]) - pages(kv[i])
        asked += more
        if more and asked > there:
            status[i] = 1
            continue
        for j in range(pages(kv[i]), pages(want[i])):
            table[i][j] = free.pop()
        kv_out[i] = want[i]
    slots, pos = [-1] * slot_cap, [0] * slot_cap
    for i in range(n):
        for e in range(new[i]):
            t, p = cu[i] + e, kv[i] + e
            if t < slot_cap:
                pos[t] = p
                if status[i] == 0:
                    slots[t] = table[i][p // page] * page + p % page
    return kv_out, table, free, cu, slots, pos, status


def attention(q, k, v, first, scale):
    """q [n, Hq, d]; k, v [L, Hkv, d]; row i sees the keys 0 .. first + i.
    Returns the outputs, and with the probabilities p: sum p |v| and the largest
    scale * sum |q k| of a seen key (for error bounds)."""
    n, hq, d = q.shape
    g = hq // k.shape[1]
    o, mass, dot = np.zeros((n, hq, d)), np.zeros((n, hq, d)), np.zeros((n, hq, 1))
    for i in range(n):
        m = min(len(k), first + i + 1)
        if m <= 0:
            continue
        for h in range(hq):
            kk, vv = k[:m, h // g], v[:m, h // g]
            s = scale * (kk @ q[i, h])
            p = np.exp(s - s.max())
            p /= p.sum()
            o[i, h], mass[i, h] = p @ vv, p @ np.abs(vv)
            dot[i, h] = abs(scale) * np.max(np.abs(kk) @ np.abs(q[i, h]))
    return o, mass, dot


__all__ = ["MIN_SCALE", "TOP", "e4m3_value", "code_round", "scale_for", "PagedCache", "rotate", "plan_pages",
           "attention", "round_bf16"]

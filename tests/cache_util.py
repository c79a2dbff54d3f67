"""Helpers of the paged-cache tests: seeded caches on the device beside the
fp64 oracle's, and the error bound of attention."""
from __future__ import annotations

import numpy as np
import torch

import gated_deltanet_prefill_varlen_amd as gdn
from oracle import cache_oracle as C

DEV = "cuda:0"
TORCH_CODE = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8}


def bf(a) -> torch.Tensor:
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(torch.bfloat16)


def f64(t: torch.Tensor) -> np.ndarray:
    return t.detach().float().cpu().numpy().astype(np.float64)


def i32(a) -> torch.Tensor:
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(DEV)


def i64(a) -> torch.Tensor:
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int64)).to(DEV)


class DevCache:
    """Pages on the device that hold what memory may hold: codes of all bits
    set (e4m3's NaN) and NaN scales."""

    def __init__(self, n_pages, hkv, page, d, code, device=DEV):
        dt = TORCH_CODE[code]
        self.page, self.code = page, code
        self.k = torch.full((n_pages, hkv, page, d), 0x7F, dtype=torch.uint8, device=device).view(dt)
        self.v = torch.full((n_pages, hkv, page // 16, d, 16), 0xFF, dtype=torch.uint8, device=device).view(dt)
        self.ks = torch.full((n_pages, hkv), float("nan"), device=device)
        self.vs = torch.full((n_pages, hkv), float("nan"), device=device)
        self.handle = gdn.make_cache(self.k, self.v, self.ks, self.vs)

    def load(self, ref: C.PagedCache, only=None):
        """The oracle's codes and scales, of the (page, offset) pairs in `only`
        (all when None); the rest stays as it is."""
        dt = TORCH_CODE[self.code]
        n, h, p, d = ref.k.shape
        keep = np.ones((n, p), bool)
        if only is not None:
            keep[:] = False
            for a, b in only:
                keep[a, b] = True
        keep = torch.from_numpy(keep).to(self.k.device)
        raw = lambda x: torch.from_numpy(x.astype(np.float32)).to(dt).view(torch.uint8).to(self.k.device)
        kk, vv = raw(ref.k), raw(ref.v)
        old_k = self.k.view(torch.uint8)
        old_v = self.v.view(torch.uint8).transpose(3, 4).reshape(n, h, p, d)
        m = keep[:, None, :, None]
        self.k.copy_(torch.where(m, kk, old_k).view(dt))
        self.v.copy_(torch.where(m, vv, old_v).reshape(n, h, p // 16, 16, d).transpose(3, 4).contiguous().view(dt))
        pages = keep.any(1)[:, None]
        self.ks.copy_(torch.where(pages, torch.from_numpy(ref.ks).float().to(self.ks.device), self.ks))
        self.vs.copy_(torch.where(pages, torch.from_numpy(ref.vs).float().to(self.vs.device), self.vs))

    def codes(self):
        """Codes as numbers [n_pages, Hkv, page, d] (both) and scales, in fp64."""
        n, h, p, d = self.k.shape
        return (f64(self.k), f64(self.v).transpose(0, 1, 2, 4, 3).reshape(n, h, p, d), f64(self.ks), f64(self.vs))


def tables(rng, lens, page, spare=3, width=None):
    """Random pages for requests of these lengths: (table, n_pages); entries
    past a request's pages hold ids that are nobody's."""
    need = [-(-x // page) for x in lens]
    n_pages = sum(need) + spare
    m = max([1] + need) + 1 if width is None else width
    ids = rng.permutation(n_pages)
    t = rng.integers(-(1 << 31), (1 << 31) - 1, size=(len(lens), m)).astype(np.int32)
    at = 0
    for i, x in enumerate(need):
        t[i, :x] = ids[at:at + x]
        at += x
    return t, n_pages


def slots_of(table, page, i, lo, hi):
    return [int(table[i, p // page]) * page + p % page for p in range(lo, hi)]


def filled(rng, lens, hkv, page, d, code, k_scale=1.0, v_scale=1.0):
    """An oracle cache that holds these requests' tokens, its device twin
    (everything else poisoned), the block table and the dequantised rows."""
    table, n_pages = tables(rng, lens, page)
    ref = C.PagedCache(n_pages, hkv, page, d, code)
    rows, only = [], []
    for i, x in enumerate(lens):
        k = C.round_bf16(rng.standard_normal((x, hkv, d)) * k_scale)
        v = C.round_bf16(rng.standard_normal((x, hkv, d)) * v_scale)
        sl = slots_of(table, page, i, 0, x)
        ref.append([0, x], sl, k, v)
        rows.append(ref.read(sl))
        only += [(s // page, s % page) for s in sl]
    dev = DevCache(n_pages, hkv, page, d, code)
    dev.load(ref, only)
    return ref, dev, table, rows


def attn_bound(o, mass, dot, d, keys):
    """Largest error of a bf16 output: half a step of the output (2^-8 of its
    value), half a bf16 step of each probability (2^-8 of sum p |v|), and the
    fp32 work.  Where the sum is of the rounded probabilities p (1 + e), |e| <=
    2^-8, the quotient sum p (1 + e) v / sum p (1 + e) has besides those e of
    the numerator a denominator between 1 - 2^-8 and 1 + 2^-8: another 2^-8 of
    the output (and a second order, below).  A score of `dot` = scale sum |q k| is summed from d products,
    each sum off by 2^-24 of it at most, and exponentiated with a relative error
    of 2^-22 of its size: p is off by that much of itself twice (numerator and
    sum); the sums over the keys add keys 2^-24."""
    p = 2 * dot * ((d + 4) * 2.0 ** -24 + 2.0 ** -22) + (keys + 8) * 2.0 ** -24 + 2.0 ** -20
    return (2 * 2.0 ** -8 * np.abs(o) + (2.0 ** -8 + p) * mass) * (1 + 2.0 ** -7) + 2.0 ** -126

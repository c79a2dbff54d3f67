"""Packs for the kernel of many rows: the limit below which a prompt goes to the
decoding requests' kernel instead, and a call on prompts above it."""
from __future__ import annotations

import os
import re

import numpy as np
import torch

import gated_deltanet_prefill_varlen_amd as gdn
from cache_util import f64, i32


def few_rows(d: int) -> int:
    """Rows (tokens x query heads of a kv head) up to which a prompt is taken
    for one of few rows: read where the library has it, so that tests of the
    other kernel cannot slip below a limit that moves."""
    src = os.path.join(os.path.dirname(gdn.__file__), "csrc", "cache_internal.h")
    with open(src) as f:
        m = re.search(r"few_rows\(int dim\) \{ return dim == 256 \? (\d+) : (\d+); \}", f.read())
    return int(m.group(1 if d == 256 else 2))


def packed_call(dev, new, lens, table, q, scale=None):
    cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    out = torch.full_like(q, 5.0)
    gdn.gdn_attn_packed(dev.handle, i32(cu), cu, i32(lens), i32(table), q, out, scale)
    return out


def many_rows_call(dev, new, lens, table, q, scale=None):
    """The same, for prompts that all have more rows than few_rows()."""
    g = q.shape[1] // dev.k.shape[1]
    assert min(new) * g > few_rows(dev.k.shape[3])
    return packed_call(dev, new, lens, table, q, scale)


__all__ = ["few_rows", "packed_call", "many_rows_call", "f64"]

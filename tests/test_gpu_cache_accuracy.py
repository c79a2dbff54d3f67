"""Errors of the kernel of decoding requests, which sums probabilities before
any of them is rounded: decode calls, and packs of prompts of few rows."""
import numpy as np
import pytest

from cache_util import DEV, attn_bound, bf, f64, filled
from packed_util import few_rows, packed_call
from test_gpu_cache import decode_call, oracle_rows

pytestmark = pytest.mark.gpu


def check_unrounded_sum(out, ref_rows, d, what):
    """attn_bound without the 2^-8 of the output that it allows a sum of rounded
    probabilities: this sum is of fp32 ones, whose errors its p covers."""
    got = f64(out)
    for r, (o, mass, dot, keys) in enumerate(ref_rows):
        err = np.abs(got[r] - o) - (attn_bound(o, mass, dot, d, keys) - 2.0 ** -8 * np.abs(o) * (1 + 2.0 ** -7))
        assert np.all(err <= 0), (what, r, float(err.max()))


@pytest.mark.parametrize("code", ["e4m3", "int8"])
@pytest.mark.parametrize("d,page,g,n_tok", [(64, 16, 3, 1), (64, 64, 8, 4), (128, 16, 4, 1), (128, 128, 16, 2), (256, 32, 8, 1), (256, 64, 12, 4)])
def test_sums_of_unrounded_probabilities(d, page, g, n_tok, code):
    rng = np.random.default_rng(d + g)
    lens = [n_tok, 17, 64, 65, 300, 1024, 1537, 2600]
    assert n_tok * g <= few_rows(d)
    for v_scale, q_scale in ((1.0, 1.0), (1.0, 0.0), (1.0, 6.0)):
        ref, dev, table, rows = filled(rng, lens, 1, page, d, code, 1.0, v_scale)
        if q_scale == 0.0:                              # all keys alike, values of one sign: errors of the sum do not cancel
            ref.v[:] = np.abs(ref.v)
            at = [(int(table[i, p // page]), p % page) for i, n in enumerate(lens) for p in range(n)]
            dev.load(ref, at)
            rows = [ref.read([int(table[i, p // page]) * page + p % page for p in range(n)]) for i, n in enumerate(lens)]
        q = bf(q_scale * rng.standard_normal((len(lens) * n_tok, g, d))).to(DEV)
        want = oracle_rows(f64(q), rows, lens, [n_tok] * len(lens), d ** -0.5)
        check_unrounded_sum(decode_call(dev, n_tok, lens, table, q), want, d, "decode")
        check_unrounded_sum(packed_call(dev, [n_tok] * len(lens), lens, table, q), want, d, "few rows")

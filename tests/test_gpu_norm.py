"""The root-mean-square norm against the fp64 oracle.

Bounds: a sum of squares of up to 32,768 values is formed as 8 products a
vector, up to 4 vectors and a tree: at most 8 + 4 + 6 + 64 additions in a row,
82 * 2^-24, whose root halves it; the quotient, the weight and the gate (two
hardware functions of 2^-22) add less than 2^-20: 2^-18 in all.  A bf16 result
is off by half a step more, 2^-8; an e4m3 code by 2^-4 of its value or half
the smallest step, 2^-10; an int8 code by half a step."""
import numpy as np
import pytest
import torch

import gated_deltanet_prefill_varlen_amd as gdn
from oracle import ssm_oracle as O
from tests.ssm_util import DEV, f64

pytestmark = pytest.mark.gpu
E = 2.0 ** -18
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def make(rows, dim, dtype=torch.bfloat16, pad=0, seed=0, scale=1.0, off=0):
    g = torch.Generator().manual_seed(seed)
    t = (torch.randn(rows, dim + pad + off, generator=g) * scale).to(dtype).to(DEV)
    return t[:, off:off + dim]


def check(rows, dim, dtype=torch.bfloat16, res=None, gate="none", groups=1, code=None, block=0, out=True, pad=0, off=0, weight="full", offset=0.0,
          scale=1.0, seed=0, in_place=False):
    x = make(rows, dim, dtype, pad, seed, scale, off)
    r = None if res is None else make(rows, dim, res, pad + 8, seed + 1, scale, off)
    z = None if gate == "none" else make(rows, dim, dtype, pad + 16, seed + 2, 1.0, off)
    w = None if weight == "none" else 1 + 0.3 * make(1, dim if weight == "full" else dim // groups, torch.float32, 0, seed + 3)[0]
    y, want_r = O.rms_norm(f64(x), f64(w), f64(r), f64(z), gate == "first", groups, 1e-5, offset)
    o = None if not out else torch.full((rows, dim), 7.0, dtype=dtype, device=DEV)
    ro = None if r is None else r if in_place else torch.empty_strided(r.shape, r.stride(), dtype=r.dtype, device=DEV)
    c = None if code is None else torch.zeros(rows, dim, dtype=code, device=DEV)
    s = None if code is None else torch.full((rows, dim // block if block else 1), float("nan"), device=DEV)
    shape = gdn.make_norm(dim, groups=groups, eps=1e-5, gate_first=gate == "first", scale_block=block, weight_offset=offset,
                          shared_weight=weight == "shared")
    gdn.gdn_rms_norm(shape, x, w, out=o, residual=r, residual_out=ro, gate=z, codes=c, scales=s)
    if out:
        assert np.all(np.abs(f64(o) - y) <= (HALF[dtype] + E) * (1 + 2.0 ** -6) * np.abs(y) + 1e-37)
    if r is not None:
        assert np.all(np.abs(f64(ro) - want_r) <= HALF[res] * (1 + 2.0 ** -6) * np.abs(want_r) + 2.0 ** -24 * np.abs(want_r))
    if code is not None:
        yb = y.reshape(rows, s.shape[1], -1)
        top = 448.0 if code == torch.float8_e4m3fn else 127.0
        step = np.maximum(np.abs(yb).max(-1) / top, 2.0 ** -100)
        assert np.all(np.abs(f64(s) - step) <= 2 * E * step)
        got = (f64(c).reshape(yb.shape) * f64(s)[..., None])
        tol = (2.0 ** -4 * np.abs(yb) + 2.0 ** -10 * step[..., None] if top == 448 else 0.5 * step[..., None]) * (1 + 4 * E) + 4 * E * np.abs(yb)
        assert np.all(np.abs(got - yb) <= tol)


@pytest.mark.parametrize("dim", [1, 2, 3, 7, 8, 9, 31, 64, 65, 100, 128, 200, 256, 511, 512, 513, 777, 1024, 2047, 2048, 2056, 4096, 5000, 8192, 8200,
                                 16384, 20001, 32768])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_widths(dim, dtype):
    check(5, dim, dtype, res=torch.bfloat16, code=torch.float8_e4m3fn)
    check(3, dim, dtype, gate="after", code=torch.int8)


@pytest.mark.parametrize("rows", [1, 2, 63, 300])
@pytest.mark.parametrize("dim", [8, 96, 512, 640])
def test_rows(rows, dim):
    check(rows, dim, res=torch.float32)


@pytest.mark.parametrize("groups,gd", [(2, 8), (3, 16), (5, 32), (8, 64), (32, 128), (3, 256), (4, 512), (2, 1024), (3, 1536), (4, 4096), (64, 512), (4, 64)])
@pytest.mark.parametrize("gate", ["none", "first", "after"])
def test_groups(groups, gd, gate):
    check(4, groups * gd, gate=gate, groups=groups, weight="shared", code=torch.int8)
    check(3, groups * gd, gate=gate, groups=groups, res=torch.bfloat16)


@pytest.mark.parametrize("res", [None, torch.bfloat16, torch.float32])
@pytest.mark.parametrize("gate", ["none", "first", "after"])
@pytest.mark.parametrize("code,block", [(None, 0), (torch.float8_e4m3fn, 0), (torch.float8_e4m3fn, 128), (torch.int8, 0), (torch.int8, 128)])
@pytest.mark.parametrize("dim", [256, 1280])
def test_options(res, gate, code, block, dim):
    check(6, dim, torch.bfloat16, res, gate, code=code, block=block, out=code is None or block == 0)
    check(6, dim, torch.float32, res, gate, code=code, block=block, out=True, offset=1.0)


@pytest.mark.parametrize("off", [0, 1, 3])
@pytest.mark.parametrize("dim", [129, 1024, 2777])
def test_strides(off, dim):
    """Rows of a wider row that begin at no alignment, the residual in place."""
    check(7, dim, res=torch.bfloat16, gate="after", pad=5, off=off, in_place=True)
    check(7, dim, torch.float32, res=torch.float32, pad=3, off=off, code=torch.int8)


@pytest.mark.parametrize("kw", [dict(weight="none"), dict(offset=1.0), dict(scale=2.0 ** 40), dict(scale=2.0 ** -60), dict(scale=1e-3)], ids=str)
def test_values(kw):
    check(5, 700, res=torch.bfloat16, code=torch.float8_e4m3fn, **kw)


def test_in_place():
    x = make(9, 600)
    y, _ = O.rms_norm(f64(x), eps=1e-5)
    x = x.contiguous()
    gdn.gdn_rms_norm(gdn.make_norm(600, eps=1e-5), x, out=x)
    assert np.all(np.abs(f64(x) - y) <= (2.0 ** -8 + E) * 1.02 * np.abs(y))


def test_zeros_and_not_finite():
    x = make(6, 384)
    x = x.contiguous()
    x[1] = 0
    x[2, 5] = float("nan")
    x[3, 6] = float("inf")
    x[4, 200:] = 0
    out = torch.zeros_like(x)
    for code in (torch.float8_e4m3fn, torch.int8):
        c, s = torch.zeros(6, 384, dtype=code, device=DEV), torch.zeros(6, 3, device=DEV)
        gdn.gdn_rms_norm(gdn.make_norm(384, scale_block=128), x, out=out, codes=c, scales=s)
        assert bool((out[1] == 0).all()) and bool((c[1].float() == 0).all()) and bool((s[1] == 2.0 ** -100).all())
        assert bool(out[2].isnan().all()) and bool(s[2].isfinite().all())
        assert bool((c[2].float() == 0).all()) if code == torch.int8 else bool(c[2].float().isnan().all())
        assert bool(out[3, 6].isnan()) and bool((out[3, :6] == 0).all())
        assert bool((s[4, 2] == 2.0 ** -100)) and bool((c[4, 256:].float() == 0).all())
        for i in (0, 5):
            y, _ = O.rms_norm(f64(x[i:i + 1]))
            assert np.all(np.abs(f64(out[i:i + 1]) - y) <= (2.0 ** -8 + E) * 1.02 * np.abs(y))


def test_row_bits_do_not_depend_on_the_batch():
    for dim in (100, 512, 3000):
        x, r = make(50, dim), make(50, dim, seed=1)
        shape = gdn.make_norm(dim)
        a, b = torch.zeros(50, dim, dtype=torch.bfloat16, device=DEV), torch.zeros(1, dim, dtype=torch.bfloat16, device=DEV)
        gdn.gdn_rms_norm(shape, x, out=a, residual=r)
        gdn.gdn_rms_norm(shape, x[37:38], out=b, residual=r[37:38])
        assert torch.equal(a[37:38], b)


def test_nothing_to_do():
    x = torch.zeros(0, 64, dtype=torch.bfloat16, device=DEV)
    gdn.gdn_rms_norm(gdn.make_norm(64), x, out=torch.zeros_like(x))


def test_after_the_delta_rule_scan():
    """The gated norm over each head of the packed delta-rule prefill's outputs."""
    T, H, d = 40, 4, 128
    g = torch.Generator().manual_seed(0)
    rnd = lambda *n: torch.randn(*n, generator=g)
    q, k, v = (rnd(T, 2, d).bfloat16().to(DEV), rnd(T, 2, d).bfloat16().to(DEV), rnd(T, H, d).bfloat16().to(DEV))
    gl, beta = -rnd(T, H).abs().to(DEV), torch.rand(T, H, generator=g).to(DEV)
    cu = np.array([0, 25, T], np.int32)
    out = torch.empty(T, H, d, dtype=torch.bfloat16, device=DEV)
    final = torch.empty(2, H, d, d, device=DEV)
    gdn.gdn_prefill_packed(gdn.make_shape(2, H, d, d), torch.from_numpy(cu).to(DEV), cu, q, k, v, gl, beta, None, None, None, out, final, None)
    z, w = rnd(T, H * d).bfloat16().to(DEV), rnd(d).to(DEV)
    y = torch.empty(T, H * d, dtype=torch.bfloat16, device=DEV)
    gdn.gdn_rms_norm(gdn.make_norm(H * d, groups=H, shared_weight=True), out.view(T, H * d), w, out=y, gate=z)
    want, _ = O.rms_norm(f64(out).reshape(T, -1), f64(w), gate=f64(z), groups=H)
    assert np.all(np.abs(f64(y) - want) <= (2.0 ** -8 + E) * 1.02 * np.abs(want) + 1e-37)

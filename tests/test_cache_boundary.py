"""The paged cache's entry points without a GPU: every refusal comes from the
host before any HIP call, in the C ABI and in the Python binding."""
import ctypes

import numpy as np
import pytest
import torch

import gated_deltanet_prefill_varlen_amd as gdn

FAKE = 0x100000     # only in calls that fail validation, or have no device to launch on
no_gpu = pytest.mark.skipif(torch.cuda.device_count() > 0,
                            reason="host-validation probes with fake device pointers run only without a GPU")
NULL, SHAPE, UNSUPPORTED, SEQLENS, CAPACITY, HIP = 1, 2, 3, 4, 6, 7


def cache(**kw):
    f = dict(num_kv_heads=2, head_dim=128, page=64, code_dtype=gdn.GDN_E4M3, n_pages=8, reserved=0,
             k=FAKE, v=FAKE, k_scale=FAKE, v_scale=FAKE)
    f.update(kw)
    return gdn.gdn_cache(*f.values())


BAD_CACHES = [(dict(num_kv_heads=0), SHAPE), (dict(n_pages=0), SHAPE), (dict(head_dim=96), UNSUPPORTED),
              (dict(head_dim=32), UNSUPPORTED), (dict(page=8), UNSUPPORTED), (dict(page=48), UNSUPPORTED),
              (dict(page=256), UNSUPPORTED), (dict(code_dtype=gdn.GDN_BF16), UNSUPPORTED)]
BAD_DATA = [(dict(k=None), NULL), (dict(v=None), NULL), (dict(k_scale=None), NULL), (dict(v_scale=None), NULL),
            (dict(k=FAKE + 8), SHAPE), (dict(v=FAKE + 4), SHAPE)]


def ref(c):
    return None if c is None else ctypes.byref(c)


def plan(page=16, n=2, want=FAKE, kv=FAKE, kvo=FAKE, table=FAKE, m=4, free=FAKE, fc=FAKE, fco=FAKE, pages=8, cu=FAKE,
         slot=FAKE, cap=32, pos=None, status=FAKE):
    return gdn.load().gdn_plan_pages(page, n, want, kv, kvo, table, m, free, fc, fco, pages, cu, slot, cap, pos, status, None)


@no_gpu
def test_plan_refusals():
    assert plan() == HIP
    for kw, st in [(dict(page=0), UNSUPPORTED), (dict(page=24), UNSUPPORTED), (dict(n=-1), SHAPE), (dict(m=-1), SHAPE),
                   (dict(pages=0), SHAPE), (dict(cap=-1), SHAPE), (dict(want=None), NULL), (dict(kv=None), NULL),
                   (dict(kvo=None), NULL), (dict(table=None), NULL), (dict(free=None), NULL), (dict(fc=None), NULL),
                   (dict(fco=None), NULL), (dict(cu=None), NULL), (dict(slot=None), NULL), (dict(status=None), NULL)]:
        assert plan(**kw) == st, kw
    assert plan(cap=0, slot=None) == HIP                       # no new tokens to slot
    assert plan(n=0, want=None, kv=None, kvo=None, table=None, status=None) == HIP


def append(rope=None, c=None, hq=4, cu=(0, 3, 7), T=None, q=FAKE, qs=0, k=FAKE, ks=0, v=FAKE, vs=0, pos=FAKE, ps=7,
           slot=FAKE, qo=FAKE, qos=0, cud=FAKE):
    rope = gdn.make_rope([1.0] * 32) if rope is None else rope
    c = cache() if c is None else c
    cu = np.asarray(cu, np.int32)
    T = int(cu[-1]) if T is None else T
    return gdn.load().gdn_rope_append(ref(rope), ref(c), hq, cud, cu.ctypes.data, len(cu) - 1, T, q, qs, k, ks, v, vs,
                                      pos, ps, slot, qo, qos, None)


@no_gpu
def test_append_refusals():
    assert append() == HIP
    assert append(q=None, qo=None, hq=0) == HIP                # the cache alone
    assert append(rope=gdn.make_rope([]), pos=None) == HIP     # no rotation
    assert append(cu=(0, 0, 0)) == 0                           # nothing to do
    assert append(ks=1024, vs=1024, qs=1024, qos=1024) == HIP  # columns of one row
    for kw, st in BAD_CACHES + BAD_DATA:
        assert append(c=cache(**kw)) == st, kw
    for kw, st in [(dict(cu=(1, 3)), SEQLENS), (dict(cu=(0, 5, 3)), SEQLENS), (dict(T=9), SEQLENS), (dict(k=None), NULL),
                   (dict(v=None), NULL), (dict(slot=None), NULL), (dict(pos=None), NULL), (dict(q=None), NULL),
                   (dict(qo=None), NULL), (dict(cud=None), NULL), (dict(hq=0), SHAPE), (dict(ks=128), SHAPE), (dict(ks=260), SHAPE),
                   (dict(vs=-256), SHAPE), (dict(qs=8), SHAPE), (dict(qos=511), SHAPE), (dict(k=FAKE + 2), SHAPE),
                   (dict(qo=FAKE + 8), SHAPE), (dict(ps=-1), SHAPE), (dict(qs=1024), SHAPE)]:
        assert append(**kw) == st, kw
    r = gdn.make_rope([1.0] * 32)
    for field, value, st in [("rot_dim", 24, UNSUPPORTED), ("rot_dim", -16, UNSUPPORTED), ("rot_dim", 144, UNSUPPORTED),
                             ("n_axes", 0, UNSUPPORTED), ("n_axes", 5, UNSUPPORTED), ("adjacent", 2, UNSUPPORTED),
                             ("scale", float("inf"), SHAPE)]:
        r = gdn.make_rope([1.0] * 32)
        setattr(r, field, value)
        assert append(rope=r) == st, field
    r = gdn.make_rope([1.0] * 32)
    r.axis[3] = 1
    assert append(rope=r) == SHAPE
    r = gdn.make_rope([1.0] * 31 + [float("nan")])
    assert append(rope=r) == SHAPE
    assert gdn.load().gdn_rope_append(None, ref(cache()), 4, FAKE, None, 0, 0, FAKE, 0, FAKE, 0, FAKE, 0, FAKE, 0,
                                      FAKE, FAKE, 0, None) == NULL


@no_gpu
def test_gather_refusals():
    g = lambda c=None, n=5, slot=FAKE, k=FAKE, v=FAKE: gdn.load().gdn_cache_gather(ref(c or cache()), n, slot, k, v, None)
    assert g() == HIP and g(k=None) == HIP and g(v=None) == HIP and g(n=0, slot=None) == 0
    for kw, st in BAD_CACHES + BAD_DATA:
        assert g(c=cache(**kw)) == st, kw
    assert g(n=-1) == SHAPE and g(slot=None) == NULL and g(k=None, v=None) == NULL and g(k=FAKE + 8) == SHAPE


def packed(c=None, hq=4, scale=0.1, cu=(0, 3, 7), T=None, kv=FAKE, table=FAKE, m=4, q=FAKE, qs=0, out=2 * FAKE, cud=FAKE):
    cu = np.asarray(cu, np.int32)
    return gdn.load().gdn_attn_packed(ref(c or cache()), hq, scale, cud, cu.ctypes.data, len(cu) - 1,
                                      int(cu[-1]) if T is None else T, kv, table, m, q, qs, out, None)


def decode(c=None, hq=4, scale=0.1, b=2, n_tok=1, kv=FAKE, table=FAKE, m=4, most=256, q=FAKE, qs=0, out=2 * FAKE, ws=4 * FAKE,
           size=1 << 40):
    return gdn.load().gdn_attn_decode(ref(c or cache()), hq, scale, b, n_tok, kv, table, m, most, q, qs, out, ws, size, None)


@no_gpu
@pytest.mark.parametrize("call", [packed, decode])
def test_attention_refusals(call):
    assert call() == HIP and call(m=0, table=None, **({"most": 0} if call is decode else {})) == HIP
    for kw, st in BAD_CACHES + BAD_DATA:
        assert call(c=cache(**kw)) == st, kw
    for kw, st in [(dict(hq=3), UNSUPPORTED), (dict(hq=130), UNSUPPORTED), (dict(hq=0), SHAPE), (dict(scale=float("nan")), SHAPE),
                   (dict(m=-1), SHAPE), (dict(kv=None), NULL), (dict(table=None), NULL), (dict(q=None), NULL), (dict(out=None), NULL),
                   (dict(qs=504), SHAPE), (dict(qs=516), SHAPE), (dict(q=FAKE + 8), SHAPE), (dict(out=2 * FAKE + 2), SHAPE),
                   (dict(out=FAKE), SHAPE), (dict(out=FAKE + 1024), SHAPE)]:
        assert call(**kw) == st, kw


@no_gpu
def test_packed_and_decode_refusals_of_their_own():
    for kw, st in [(dict(cu=(1, 3)), SEQLENS), (dict(cu=(0, 5, 3)), SEQLENS), (dict(T=9), SEQLENS), (dict(cud=None), NULL)]:
        assert packed(**kw) == st, kw
    assert packed(cu=(0, 0)) == 0
    for kw, st in [(dict(b=-1), SHAPE), (dict(n_tok=0), SHAPE), (dict(most=-1), SHAPE), (dict(most=257), SHAPE),
                   (dict(b=1 << 30, n_tok=4), SHAPE)]:
        assert decode(**kw) == st, kw
    assert decode(b=0, kv=None, table=None, q=None, out=None) == 0
    n = ctypes.c_int64(-1)
    lib, size = gdn.load(), lambda *a: gdn.load().gdn_attn_decode_workspace(ref(cache()), *a, ctypes.byref(n))
    assert size(4, 2, 1, 256) == 0 and n.value >= 0
    assert size(4, 64, 4, 1 << 20) == 0
    if n.value:
        assert decode(b=64, n_tok=4, m=1 << 14, most=1 << 20, out=1 << 40, size=n.value - 1) == CAPACITY
        assert decode(b=64, n_tok=4, m=1 << 14, most=1 << 20, out=1 << 40, ws=None) == NULL
        assert decode(b=64, n_tok=4, m=1 << 14, most=1 << 20, out=1 << 40, ws=4 * FAKE + 8) == SHAPE
    assert size(0, 2, 1, 256) == SHAPE and size(4, -1, 1, 256) == SHAPE and size(4, 2, 0, 256) == SHAPE
    assert size(4, 2, 1, -1) == SHAPE
    assert lib.gdn_attn_decode_workspace(ref(cache()), 4, 2, 1, 256, None) == NULL
    assert lib.gdn_attn_decode_workspace(None, 4, 2, 1, 256, ctypes.byref(n)) == NULL


@no_gpu
def test_sizes_that_no_launch_holds_are_refused():
    """A launch has fewer than 2^32 threads along its first axis, and 65,535
    workgroups along the others."""
    zeros = np.zeros((1 << 22) + 1, np.int32)
    assert packed(cu=zeros) == SHAPE and packed(cu=zeros[:-1]) == 0
    assert append(cu=zeros) == SHAPE and append(cu=zeros[:-1]) == 0
    assert append(T=1 << 25, cu=(0, 1 << 25), ps=1 << 25) == SHAPE
    assert gdn.load().gdn_cache_gather(ref(cache()), 2 ** 31 - 1, FAKE, FAKE, FAKE, None) == SHAPE
    far = dict(m=1 << 24, out=1 << 45, size=1 << 60, ws=1 << 50)
    assert decode(most=65535 * 1024, **far) == HIP and decode(most=65535 * 1024 + 1, **far) == SHAPE
    assert decode(most=2 ** 30, **far) == SHAPE
    assert decode(b=65535, n_tok=256, most=64, **far) == HIP and decode(b=65535, n_tok=257, most=64, **far) == SHAPE
    assert decode(m=(1 << 24) + 1, most=64) == SHAPE and packed(m=(1 << 24) + 1) == SHAPE
    n = ctypes.c_int64()
    big = cache(page=128)
    assert gdn.load().gdn_attn_decode_workspace(ref(big), 4, 1, 1, 2 ** 31 - 1, ctypes.byref(n)) == 0
    assert n.value == (1 << 21) * 4 * 130 * 4


@no_gpu
def test_workspace_apart_from_the_rows():
    assert gdn.load().gdn_attn_decode_workspace(ref(cache()), 4, 2, 1, 4096, ctypes.byref(n := ctypes.c_int64())) == 0 and n.value
    ok = dict(m=64, most=4096, q=1 << 30, out=1 << 31, ws=1 << 32)
    assert decode(**ok) == HIP
    for at in ("q", "out"):
        base = ok[at]
        for ws, st in [(base, SHAPE), (base + 1024, SHAPE), (base - n.value + 16, SHAPE), (base - n.value, HIP), (base + 2 * 4 * 128 * 2, HIP)]:
            assert decode(**{**ok, "ws": ws}) == st, (at, ws - base)


def test_binding_refusals():
    """Wrong shapes, types and places are Python errors before any call."""
    f8, i8 = torch.float8_e4m3fn, torch.int8
    z = lambda *s, dt=torch.float32: torch.zeros(*s).to(dt)
    for k, v, ks in [(z(4, 2, 16, 64), z(4, 2, 1, 64, 16), z(4, 2)),                       # not codes
                     (z(4, 2, 16, 64, dt=i8), z(4, 2, 1, 64, 16, dt=f8), z(4, 2)),
                     (z(4, 2, 16, 64, dt=i8), z(4, 2, 16, 64, dt=i8), z(4, 2)),
                     (z(4, 2, 16, 64, dt=i8), z(4, 2, 1, 64, 16, dt=i8), z(4, 3)),
                     (z(4, 2, 16, 64, dt=i8), z(4, 2, 1, 64, 16, dt=i8), z(4, 2))]:         # not on the GPU
        with pytest.raises(ValueError):
            gdn.make_cache(k, v, ks, ks)
    for freq, axis, n in [([1.0] * 129, None, 1), ([1.0], [1], 1), ([1.0, 2.0], [0], 1), ([1.0], [-1], 2)]:
        with pytest.raises(ValueError):
            gdn.make_rope(freq, axis, n)
    c = cache()
    i32 = lambda *s: z(*s, dt=torch.int32)
    q = z(3, 4, 128, dt=torch.bfloat16)
    with pytest.raises(ValueError):
        gdn.gdn_attn_decode(c, 1, i32(3), i32(3, 4), q, q.clone())                          # not on the GPU
    with pytest.raises(TypeError):
        gdn.gdn_attn_decode(c, 1, i32(3), i32(3, 4), q.float(), q)
    with pytest.raises(ValueError):
        gdn.gdn_attn_decode(c, 1, i32(4), i32(4, 4), q, q)                                  # q too short
    with pytest.raises(ValueError):
        gdn.gdn_attn_packed(c, i32(2), [0, 3], i32(1), i32(1, 4), q.transpose(0, 1), q)     # rows of other heads
    with pytest.raises(ValueError):
        gdn.gdn_cache_gather(c, z(3, dt=torch.int64), q, q)                                 # 4 heads, not 2
    with pytest.raises(ValueError):
        gdn.gdn_plan_pages(16, i32(3), i32(2), i32(3), i32(3, 4), i32(8), i32(1), i32(1), i32(4), z(4, dt=torch.int64), None, i32(3))

"""The state space layers' and the norm's entry points without a GPU: every
refusal comes from the host before any HIP call, in the C ABI and in the
Python binding."""
import ctypes

import numpy as np
import pytest
import torch

import gated_deltanet_prefill_varlen_amd as gdn

FAKE = 1 << 40     # only in calls that fail validation, or have no device to launch on
no_gpu = pytest.mark.skipif(torch.cuda.device_count() > 0,
                            reason="host-validation probes with fake device pointers run only without a GPU")
NULL, SHAPE, UNSUPPORTED, SEQLENS, CKPT, CAPACITY, HIP = 1, 2, 3, 4, 5, 6, 7
at = lambda i: FAKE + (i << 36)      # far apart


def ssm(**kw):
    s = gdn.make_ssm(4, 2, 64, 64)
    for k, v in kw.items():
        setattr(s, k, v)
    return s


BAD_SHAPES = [(dict(num_heads=0), SHAPE), (dict(num_groups=0), SHAPE), (dict(num_groups=3), UNSUPPORTED), (dict(head_dim=48), UNSUPPORTED),
              (dict(head_dim=256), UNSUPPORTED), (dict(state_dim=16), UNSUPPORTED), (dict(flags=2), UNSUPPORTED),
              (dict(dt_min=1.0, dt_max=0.5), SHAPE), (dict(dt_min=float("nan")), SHAPE), (dict(num_heads=70000), SHAPE),
              (dict(num_heads=60000, num_groups=60000), SHAPE)]
C = 4 * 64 + 2 * 2 * 64


def need(cu, s=None):
    n = ctypes.c_int64(-1)
    cu = np.asarray(cu, np.int32)
    st = gdn.load().gdn_ssm_prefill_workspace(ctypes.byref(ssm() if s is None else s), cu.ctypes.data, len(cu) - 1, int(cu[-1]), ctypes.byref(n))
    return st, n.value


def prefill(s=None, cu=(0, 3, 7), T=None, cud=at(0), x=at(1), xs=0, w=at(2), b=at(3), ci=at(4), co=at(5), dtt=0, dt=at(6), dts=0, A=at(7),
            bias=at(8), D=at(9), init=at(10), pos=(2, 7), posd=at(11), cc=at(12), out=at(13), final=at(14), kept=at(15), ws=at(16),
            size=1 << 34, shape_null=False):
    cu = np.asarray(cu, np.int32)
    ph = None if pos is None else np.asarray(pos, np.int32)
    return gdn.load().gdn_ssm_prefill_packed(
        None if shape_null else ctypes.byref(ssm() if s is None else s), cud, cu.ctypes.data, len(cu) - 1, int(cu[-1]) if T is None else T, x, xs, w, b,
        ci, co, gdn.GDN_BF16 if dtt == 0 else dtt, dt, dts, A, bias, D, init, posd, None if ph is None else ph.ctypes.data,
        0 if ph is None else len(ph), cc, out, final, kept, ws, size, None)


@no_gpu
def test_prefill_refusals():
    assert prefill() == HIP
    assert prefill(w=None, b=None, ci=None, co=None, cc=None) == HIP
    assert prefill(b=None, bias=None, D=None, init=None, final=None, pos=None, posd=None, kept=None, cc=None, ci=None, co=None) == HIP
    assert prefill(dtt=gdn.GDN_F32) == HIP and prefill(xs=C + 8, dts=9) == HIP
    assert prefill(shape_null=True) == NULL
    for kw, st in BAD_SHAPES:
        assert prefill(s=ssm(**kw)) == st, kw
    for kw, st in [(dict(cu=(1, 3)), SEQLENS), (dict(cu=(0, 5, 3)), SEQLENS), (dict(T=9), SEQLENS), (dict(cud=None), NULL),
                   (dict(x=None), NULL), (dict(dt=None), NULL), (dict(A=None), NULL), (dict(out=None), NULL), (dict(ws=None), NULL),
                   (dict(w=None), NULL), (dict(w=None, ci=None, co=None, cc=None), NULL), (dict(posd=None), NULL), (dict(kept=None), NULL),
                   (dict(pos=(2, 2)), CKPT), (dict(pos=(7, 2)), CKPT), (dict(pos=(0, 2)), CKPT), (dict(pos=(2, 8)), CKPT),
                   (dict(dtt=gdn.GDN_E4M3), UNSUPPORTED), (dict(xs=C - 8), SHAPE), (dict(xs=C + 4), SHAPE), (dict(xs=-C), SHAPE),
                   (dict(xs=1 << 23), SHAPE), (dict(dts=3), SHAPE), (dict(dts=1 << 31), SHAPE)]:
        assert prefill(**kw) == st, kw
    for name in ("x", "w", "b", "ci", "co", "init", "cc", "out", "final", "kept", "ws"):
        assert prefill(**{name: at(20) + 8}) == SHAPE, name


@no_gpu
def test_prefill_overlaps():
    head, row, rows = 4 * 64 * 64 * 4, 4 * 64 * 2, 7 * 4 * 64 * 2
    st, n = need((0, 3, 7))
    assert st == 0 and n > 0 and prefill(size=n) == HIP and prefill(size=n - 1) == CAPACITY
    assert prefill(co=at(4)) == HIP and prefill(final=at(10)) == HIP            # in place
    for kw in [dict(out=at(1)), dict(out=at(1) + 6 * C * 2), dict(x=at(13) + rows - 16), dict(co=at(4) + 16), dict(final=at(10) + 16),
               dict(final=at(10) - 2 * head + 16), dict(kept=at(10) + head), dict(kept=at(14) - 16), dict(ws=at(1) - n + 16), dict(ws=at(13)),
               dict(ws=at(10)), dict(ws=at(14) + 2 * head - 16), dict(ws=at(15))]:
        assert prefill(**kw) == SHAPE, kw
    for kw in [dict(out=at(1) + 7 * C * 2), dict(final=at(10) + 2 * head), dict(kept=at(10) + 2 * head), dict(ws=at(13) + rows)]:
        assert prefill(**kw) == HIP, kw


@no_gpu
def test_prefill_of_nothing():
    assert prefill(cu=(0,), cud=None, pos=None, x=None, dt=None, A=None, out=None, ws=None, size=0) == 0
    assert need((0,)) == (0, 0) and need((0, 0, 0)) == (0, 0)
    assert prefill(cu=(0, 0), pos=None, x=None, dt=None, A=None, out=None, ws=None, size=0) == HIP     # its state and window are written


@no_gpu
def test_workspace_refusals_and_growth():
    lib, n, cu = gdn.load(), ctypes.c_int64(), np.array([0, 4], np.int32)
    assert lib.gdn_ssm_prefill_workspace(None, cu.ctypes.data, 1, 4, ctypes.byref(n)) == NULL
    assert lib.gdn_ssm_prefill_workspace(ctypes.byref(ssm()), cu.ctypes.data, 1, 4, None) == NULL
    assert lib.gdn_ssm_prefill_workspace(ctypes.byref(ssm()), cu.ctypes.data, 1, 5, ctypes.byref(n)) == SEQLENS
    for kw, st in BAD_SHAPES:
        assert need((0, 4), ssm(**kw))[0] == st, kw
    sizes = [need((0, t))[1] for t in (1, 31, 32, 33, 1024, 1025, 8192, 100000)]
    assert sizes == sorted(sizes) and all(v % 256 == 0 for v in sizes)
    assert need((0, 1 << 30))[1] > 1 << 32                          # in 64 bits


@no_gpu
def test_sizes_that_no_launch_holds_are_refused():
    zeros = np.zeros((1 << 23) + 1, np.int32)
    assert prefill(cu=zeros, pos=None) == SHAPE
    assert step(B=1 << 24, pool=1 << 24, slot=None) == SHAPE
    assert norm(rows=(1 << 22) + 1, d=8192) == SHAPE and norm(rows=1 << 24, d=2048) == SHAPE


def step(s=None, B=2, n_tok=1, x=at(1), xs=0, w=at(2), b=at(3), cs=at(4), dtt=0, dt=at(6), dts=0, A=at(7), bias=at(8), D=at(9), state=at(10),
         pool=5, slot=at(11), slots=(3, 0), out=at(13), snap=at(15), shape_null=False):
    sh = None if slots is None else np.asarray(slots, np.int32)
    return gdn.load().gdn_ssm_decode(
        None if shape_null else ctypes.byref(ssm() if s is None else s), B, n_tok, x, xs, w, b, cs, gdn.GDN_BF16 if dtt == 0 else dtt, dt, dts, A, bias,
        D, state, pool, slot, None if sh is None else sh.ctypes.data, out, snap, None)


@no_gpu
def test_step_refusals():
    assert step() == HIP and step(w=None, b=None, cs=None) == HIP and step(snap=None, bias=None, D=None, b=None) == HIP
    assert step(slot=None, slots=None) == HIP and step(n_tok=3) == HIP and step(dtt=gdn.GDN_F32) == HIP
    assert step(B=0, x=None, dt=None, A=None, out=None, state=None, slot=None) == 0
    assert step(shape_null=True) == NULL
    for kw, st in BAD_SHAPES:
        assert step(s=ssm(**kw)) == st, kw
    for kw, st in [(dict(B=-1), SHAPE), (dict(pool=-1), SHAPE), (dict(n_tok=0), SHAPE), (dict(B=1 << 20, n_tok=1 << 12), SHAPE), (dict(w=None), NULL),
                   (dict(cs=None), NULL), (dict(w=None, cs=None), NULL), (dict(x=None), NULL), (dict(dt=None), NULL), (dict(A=None), NULL),
                   (dict(out=None), NULL), (dict(state=None), NULL), (dict(slots=None), NULL), (dict(slots=(3, 3)), CAPACITY),
                   (dict(slots=(3, 5)), CAPACITY), (dict(slots=(-1, 0)), CAPACITY), (dict(slot=None, pool=1), CAPACITY),
                   (dict(dtt=gdn.GDN_I8), UNSUPPORTED), (dict(xs=C - 8), SHAPE), (dict(xs=C + 2), SHAPE), (dict(dts=2), SHAPE), (dict(out=at(1)), SHAPE)]:
        assert step(**kw) == st, kw
    for name in ("x", "w", "b", "cs", "state", "out", "snap"):
        assert step(**{name: at(20) + 8}) == SHAPE, name


def norm(s=None, rows=4, d=256, xt=0, x=at(1), xs=0, rt=0, r=at(2), rs=0, ro=at(3), z=at(4), zs=0, w=at(5), out=at(6), ct=gdn.GDN_E4M3, codes=at(7),
         scales=at(8), shape_null=False, **kw):
    sh = gdn.make_norm(d) if s is None else s
    for k, v in kw.items():
        setattr(sh, k, v)
    bf = lambda t: gdn.GDN_BF16 if t == 0 else t
    return gdn.load().gdn_rms_norm(None if shape_null else ctypes.byref(sh), rows, bf(xt), x, xs, bf(rt), r, rs, ro, z, zs, w, out, ct, codes, scales,
                                   None)


@no_gpu
def test_norm_refusals():
    assert norm() == HIP and norm(shape_null=True) == NULL and norm(rows=0, x=None) == 0
    assert norm(r=None, ro=None, z=None, w=None, codes=None, scales=None) == HIP
    assert norm(out=None) == HIP and norm(out=None, codes=None, scales=None) == HIP            # the sum with the residual alone
    assert norm(xt=gdn.GDN_F32, rt=gdn.GDN_F32, ct=gdn.GDN_I8) == HIP and norm(flags=1) == HIP
    assert norm(d=1, weight_dim=1) == HIP and norm(d=32768) == HIP and norm(x=at(1) + 2, out=at(6) + 2, ro=at(3) + 2) == HIP
    assert norm(ro=at(2)) == HIP and norm(out=at(1)) == HIP                                    # in place
    for kw, st in [(dict(d=0), SHAPE), (dict(d=32769), UNSUPPORTED), (dict(groups=0), SHAPE), (dict(groups=3), SHAPE), (dict(rows=-1), SHAPE),
                   (dict(eps=-1.0), SHAPE), (dict(eps=float("nan")), SHAPE), (dict(eps=float("inf")), SHAPE), (dict(weight_offset=float("nan")), SHAPE),
                   (dict(flags=2), UNSUPPORTED), (dict(groups=64), UNSUPPORTED), (dict(d=768, groups=4), UNSUPPORTED), (dict(weight_dim=64), SHAPE),
                   (dict(scale_block=64), UNSUPPORTED), (dict(d=200, scale_block=128), UNSUPPORTED), (dict(xt=gdn.GDN_I8), UNSUPPORTED),
                   (dict(rt=gdn.GDN_E4M3), UNSUPPORTED), (dict(ct=gdn.GDN_BF16), UNSUPPORTED), (dict(xs=255), SHAPE), (dict(rs=255), SHAPE),
                   (dict(zs=255), SHAPE), (dict(xs=1 << 31), SHAPE), (dict(x=None), NULL), (dict(codes=None), NULL), (dict(scales=None), NULL),
                   (dict(r=None), NULL), (dict(out=None, codes=None, scales=None, ro=None), NULL), (dict(flags=1, z=None), NULL),
                   (dict(x=at(1) + 1), SHAPE), (dict(z=at(4) + 1), SHAPE), (dict(out=at(6) + 1), SHAPE), (dict(r=at(2) + 1), SHAPE),
                   (dict(w=at(5) + 2), SHAPE), (dict(scales=at(8) + 2), SHAPE), (dict(xt=gdn.GDN_F32, x=at(1) + 2), SHAPE),
                   (dict(out=at(1) + 256), SHAPE), (dict(out=at(1), xs=264), SHAPE), (dict(out=at(2)), SHAPE), (dict(out=at(4)), SHAPE),
                   (dict(ro=at(2) + 2), SHAPE), (dict(ro=at(1)), SHAPE), (dict(codes=at(6)), SHAPE), (dict(codes=at(3) + 100), SHAPE),
                   (dict(scales=at(5)), SHAPE), (dict(scales=at(7) + 1020), SHAPE)]:
        assert norm(**kw) == st, kw


@no_gpu
def test_binding_refusals(monkeypatch):
    """Wrong shapes, types and places are Python errors before any call.  (With
    the device that host tensors name, so that the shapes are looked at: a call
    that is not refused ends in the library's own error without a GPU.)"""
    with pytest.raises(ValueError, match="not on the GPU"):
        gdn.gdn_rms_norm(gdn.make_norm(8), torch.zeros(2, 8))
    monkeypatch.setattr(gdn, "_where", lambda stream: (-1, None))
    bf = torch.bfloat16
    z = lambda *s, dt=torch.float32: torch.zeros(*s).to(dt)
    cu = np.array([0, 3], np.int32)
    shape = ssm()

    def scan(**kw):
        a = dict(x=z(3, C, dt=bf), dt=z(3, 4, dt=bf), A=z(4), out=z(3, 4, 64, dt=bf))
        o = {k: kw.pop(k) for k in list(kw) if k in a}
        a.update(o)
        gdn.gdn_ssm_prefill_packed(shape, z(2, dt=torch.int32), cu, a["x"], a["dt"], a["A"], a["out"], **kw)

    def tokens(**kw):
        a = dict(x=z(2, C, dt=bf), dt=z(2, 4, dt=bf), A=z(4), state=z(5, 4, 64, 64), out=z(2, 4, 64, dt=bf), n_tok=1)
        o = {k: kw.pop(k) for k in list(kw) if k in a}
        a.update(o)
        gdn.gdn_ssm_decode(shape, a["n_tok"], a["x"], a["dt"], a["A"], a["state"], a["out"], **kw)

    def rms(**kw):
        a = dict(x=z(4, 256, dt=bf))
        a.update({k: kw.pop(k) for k in list(kw) if k in a})
        gdn.gdn_rms_norm(gdn.make_norm(256), a["x"], **kw)

    n = need(cu)[1]
    for call, good in ((scan, dict(workspace=z(n, dt=torch.uint8))), (tokens, {}), (rms, dict(out=z(4, 256, dt=bf)))):
        with pytest.raises(gdn.GdnError):
            call(**good)
    with pytest.raises(gdn.GdnError, match="CAPACITY"):
        scan(workspace=z(n - 1, dt=torch.uint8))
    for call in (scan, tokens):
        for bad in [dict(x=z(2, C + 8, dt=bf)), dict(x=z(1, 2, C, dt=bf)), dict(x=z(C, 3, dt=bf).T), dict(dt=z(3, 5, dt=bf)), dict(out=z(3, 2, 64, dt=bf)),
                    dict(A=z(5))]:
            with pytest.raises(ValueError):
                call(**bad)
        for bad in [dict(x=z(3, C)), dict(dt=z(3, 4, dt=torch.float16))]:
            with pytest.raises((TypeError, ValueError)):
                call(**bad)
    with pytest.raises(ValueError):
        tokens(n_tok=0)
    with pytest.raises(ValueError):
        tokens(x=z(3, C, dt=bf), n_tok=2)
    with pytest.raises(ValueError):
        tokens(slot=z(1, dt=torch.int32), slot_host=[0])
    for bad in [dict(x=z(4, 255, dt=bf)), dict(out=z(4, 128, dt=bf)), dict(residual_out=z(4, 256)), dict(residual=z(3, 256)), dict(gate=z(4, 255, dt=bf)),
                dict(residual=z(4, 256), residual_out=z(4, 512)[:, :256])]:
        with pytest.raises(ValueError):
            rms(**bad)
    for bad in [dict(conv_weight=z(C, 3)), dict(init_state=z(2, 4, 64, 64)), dict(final_state=z(1, 4, 64, 32)), dict(conv_state_in=z(1, 4, C, dt=bf)),
                dict(ckpt_positions=z(2, dt=torch.int32), ckpt_positions_host=[1, 2], ckpt_buf=z(1, 4, 64, 64)), dict(out=z(4, 3, 64, dt=bf).transpose(0, 1))]:
        with pytest.raises(ValueError):
            scan(**bad)
    for bad in [dict(conv_state=z(4, 3, C, dt=bf)), dict(snapshots=z(2, 2, 4, 64, 64)), dict(state=z(5, 4, 64, 128)[..., ::2])]:
        with pytest.raises((ValueError, TypeError)):
            tokens(**bad)
    with pytest.raises(TypeError):
        rms(codes=z(4, 256, dt=torch.uint8), scales=z(4, 1))

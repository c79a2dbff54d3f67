"""What the state space layers' calls accept and refuse at the limits of their
launches, and which of their buffers may lie over one another; without a GPU."""
import numpy as np

import gated_deltanet_prefill_varlen_amd as gdn
from tests.test_ssm_boundary import HIP, SHAPE, at, need, no_gpu, prefill, ssm, step


@no_gpu
def test_many_groups():
    """A launch's second axis holds 65,535: a group each, and eight heads each."""
    wide = dict(head_dim=32, state_dim=32)
    most = 58253                                   # 58,253 + 7,282 = 65,535
    s = ssm(num_heads=most, num_groups=most, **wide)
    assert need((0, 4), s)[0] == 0 and prefill(s=s, xs=0, dts=0, pos=None, size=1 << 40) == HIP and step(s=s, snap=None) == HIP
    s = ssm(num_heads=most + 1, num_groups=most + 1, **wide)
    assert need((0, 4), s)[0] == SHAPE


@no_gpu
def test_many_prompts_and_tokens():
    """A launch's first axis holds fewer than 2^32 threads, 256 a workgroup."""
    s = gdn.make_ssm(1, 1, 32, 32)
    args = dict(s=s, pos=None, ci=None, co=None, cc=None, w=None, b=None, init=None, final=None, x=1 << 50, out=1 << 60, ws=1 << 52, dt=1 << 58,
                size=1 << 56)
    assert prefill(cu=(0, 500_000_000), **args) == HIP
    assert prefill(cu=(0, 540_000_000), **args) == SHAPE
    assert prefill(cu=np.zeros((1 << 23) + 1, np.int32), **args) == HIP


def check_overlaps(call, spans, written, allowed):
    """Every buffer written, laid over the first and the last 16 bytes of every other, is refused; beside them it is not."""
    base = 1 << 43                                             # far from every default address
    for w in written:
        for r in spans:
            if r == w:
                continue
            nw, nr = spans[w], spans[r]
            for p in (base - nw + 16, base + nr - 16, base - nw, base + nr):
                p -= p % 16                                    # (starts stay aligned)
                got = call(**{r: base, w: p})
                assert got == (SHAPE if p < base + nr and base < p + nw else HIP), (w, r, p - base, got)
            if (w, r) not in allowed and (r, w) not in allowed:
                assert call(**{r: base, w: base}) == SHAPE, (w, r)
            else:
                assert call(**{r: base, w: base}) == HIP, (w, r)


@no_gpu
def test_scan_overlaps():
    H, P, N, T, n, k = 4, 64, 64, 7, 2, 2
    C = H * P + 2 * 2 * N
    ws = need((0, 3, 7))[1]
    spans = dict(x=T * C * 2, dt=T * H * 2, A=H * 4, bias=H * 4, D=H * 4, w=C * 16, b=C * 4, ci=n * 3 * C * 2, init=n * H * P * N * 4, cud=12, posd=8,
                 co=n * 3 * C * 2, cc=k * 3 * C * 2, out=T * H * P * 2, final=n * H * P * N * 4, kept=k * H * P * N * 4, ws=ws)
    check_overlaps(lambda **kw: prefill(size=ws, **kw), spans, ("out", "final", "kept", "co", "cc", "ws"), {("co", "ci"), ("final", "init")})
    assert prefill(x=1 << 43, init=1 << 43, final=1 << 43) == SHAPE      # in place, but over another input
    assert prefill(cu=(0, 0, 0), pos=None, x=None, dt=None, A=None, out=None, ws=at(14) + 64, size=0) == HIP   # no workspace: no overlap


@no_gpu
def test_step_overlaps():
    H, P, N, B, pool = 4, 64, 64, 2, 2
    C = H * P + 2 * 2 * N
    spans = dict(x=B * 3 * C * 2, dt=B * 3 * H * 2, A=H * 4, bias=H * 4, D=H * 4, w=C * 16, b=C * 4, slot=B * 4, state=pool * H * P * N * 4,
                 cs=pool * 3 * C * 2, out=B * 3 * H * P * 2, snap=B * 3 * H * P * N * 4)
    check_overlaps(lambda **kw: step(n_tok=3, slots=(1, 0), pool=pool, **kw), spans, ("out", "state", "cs", "snap"), set())
    check_overlaps(lambda **kw: step(n_tok=3, slots=None, pool=pool, **{**kw, "slot": None}), {k: v for k, v in spans.items() if k != "slot"},
                   ("out", "state", "cs", "snap"), set())


@no_gpu
def test_step_in_spare_slots():
    """Slots that the call does not address are neither read nor written: they may hold its snapshots, or its rows."""
    head, window, pool = 4 * 64 * 64 * 4, 3 * (4 * 64 + 2 * 2 * 64) * 2, 8
    base = 1 << 43
    for slots in ((3, 0), (0, 3), (7, 6), None):
        kw = dict(pool=pool, slots=slots, **({"slot": None} if slots is None else {}))
        used = set(slots or (0, 1))
        for first in range(pool - 1):
            spare = not used & {first, first + 1}                        # the snapshots of two sequences
            assert step(state=base, snap=base + first * head, **kw) == (HIP if spare else SHAPE), (slots, first)
        for first in range(pool):
            want = SHAPE if first in used else HIP
            assert step(state=base, out=base + first * head, **kw) == want and step(cs=base, out=base + first * window, **kw) == want, (slots, first)
            assert step(state=base, x=base + first * head, **kw) == want, (slots, first)
    assert step(state=base, cs=base + 7 * head, pool=pool, slots=(3, 0)) == SHAPE

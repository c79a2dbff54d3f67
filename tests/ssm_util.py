"""Helpers of the state space layers' tests: seeded layers and rows, the
library's calls on them, and the error bounds.

Bounds.  A state is a sum of products dt x B, each decayed: its "mass" is that
sum of absolute values, with |u| + (|bias| + sum |w| |raw|) in place of |x| and
|B|, which also covers what the convolution's fp32 sum may err by (6 roundings
of 2^-24 of that sum, before a silu of slope below 1.1).  Products of values
held as fp16 pairs err by at most 3 * 2^-22 of themselves, decays (sums of up
to 64 steps in fp32, an exponential, one factor per chunk) by 2^-20 + 2^-23 a
chunk: 2^-18 + len 2^-27 of the mass bounds a state.  Outputs multiply
operands of 11 bits: x, B, C, the state and the weights within a chunk, each
off by at most 2^-11 of itself, and half a bf16 step of the result, 2^-8."""
from __future__ import annotations

import numpy as np
import torch

import gated_deltanet_prefill_varlen_amd as gdn
from oracle import ssm_oracle as O

DEV = "cuda:0"


def f64(t):
    return None if t is None else t.detach().float().cpu().numpy().astype(np.float64)


def state_tol(mass, length):
    return (2.0 ** -18 + length * 2.0 ** -27) * mass + 1e-30


def out_tol(y, mass):
    return 2.0 ** -8 * np.abs(y) * (1 + 2.0 ** -6) + 6 * 2.0 ** -11 * mass + 1e-30


def close(got, want, tol, what):
    got = f64(got) if isinstance(got, torch.Tensor) else got
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (what, int(bad.sum()), np.argwhere(bad)[:4].tolist(),
                           float(np.max(np.where(bad, np.abs(got - want) / np.maximum(tol, 1e-300), 0))))


class Layer:
    """A layer's constants and rows, as tensors on the device; the same values
    in 64 bits go to the oracle."""

    def __init__(self, H, G, P, N, lens, seed=0, conv=True, bias=True, D=True, dt_bias=True, softplus=True, dt_f32=False, init=False,
                 window=False, pad=0, a_scale=1.0, x_scale=1.0, dt_shift=0.0, device=DEV):
        g = torch.Generator().manual_seed(seed)
        randn = lambda *n: torch.randn(*n, generator=g)
        rand = lambda *n: torch.rand(*n, generator=g)
        self.dims, self.lens, self.dev = (H, G, P, N), list(lens), device
        self.C = C = H * P + 2 * G * N
        self.cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
        T, n = int(self.cu[-1]), len(lens)
        row = randn(T, 8 + C + 8 * ((H + 7) // 8) + pad).bfloat16()
        row[:, 8:8 + C] = (row[:, 8:8 + C].float() * x_scale).bfloat16()
        if not softplus:
            row[:, 8 + C:] = row[:, 8 + C:].float().abs().mul(0.1).bfloat16()
        row = row.to(device)
        self.x = row[:, 8:8 + C]
        self.dt = row[:, 8 + C:8 + C + H]
        if dt_f32:
            self.dt = row.float()[:, 8 + C:8 + C + H]
        to = lambda t: t.to(device)
        self.A = to(-(1 + 15 * rand(H)) * a_scale)
        dt = torch.exp(rand(H) * np.log(100.0) + np.log(0.001))
        self.dt_bias = to(dt + torch.log(-torch.expm1(-dt)) + dt_shift) if dt_bias else None
        self.D = to(1 + 0.1 * randn(H)) if D else None
        self.w = to(rand(C, 4) - 0.5) if conv else None
        self.b = to(0.2 * (rand(C) - 0.5)) if conv and bias else None
        self.window = to(randn(n, 3, C).mul(x_scale).bfloat16()) if conv and window else None
        self.init = to(0.5 * randn(n, H, P, N) * x_scale) if init else None
        self.shape = gdn.make_ssm(H, G, P, N, softplus=softplus)
        self.softplus = softplus

    def steps(self):
        return O.steps(f64(self.dt), f64(self.dt_bias), self.softplus)

    def oracle(self, ckpts=()):
        H, G, P, N = self.dims
        return O.prefill(H, G, P, N, self.cu, f64(self.x), self.steps(), f64(self.A), f64(self.D), f64(self.w), f64(self.b),
                         f64(self.window), f64(self.init), set(int(c) for c in ckpts))

    def run(self, ckpts=(), only=None, window_out="new", workspace=None, stream=None):
        """The packed scan over all prompts, or over one of them alone."""
        H, G, P, N = self.dims
        lo, hi = (0, len(self.lens)) if only is None else (only, only + 1)
        a, b = int(self.cu[lo]), int(self.cu[hi])
        cu = (self.cu[lo:hi + 1] - a).astype(np.int32)
        ck = np.array([c - a for c in ckpts if a < c <= b], np.int32)
        n, k = hi - lo, len(ck)
        win = None if self.window is None else self.window[lo:hi].clone()
        r = dict(out=torch.full((b - a + 2, H, P), 7.0, dtype=torch.bfloat16, device=self.dev),
                 final=torch.full((n, H, P, N), float("nan"), device=self.dev), kept=torch.full((k, H, P, N), float("nan"), device=self.dev))
        if self.w is not None:
            r["window"] = win if window_out == "in place" and win is not None else torch.zeros(n, 3, self.C, dtype=torch.bfloat16, device=self.dev)
            r["window_kept"] = torch.zeros(k, 3, self.C, dtype=torch.bfloat16, device=self.dev) if k else None
        if workspace is None:
            workspace = torch.full((gdn.gdn_ssm_prefill_workspace(self.shape, cu),), 0xFF, dtype=torch.uint8, device=self.dev)
        self.workspace = workspace
        i32 = lambda v: torch.from_numpy(np.ascontiguousarray(v)).to(self.dev)
        gdn.gdn_ssm_prefill_packed(
            self.shape, i32(cu), cu, self.x[a:b], self.dt[a:b], self.A, r["out"], dt_bias=self.dt_bias, D=self.D,
            init_state=None if self.init is None else self.init[lo:hi].contiguous(), final_state=r["final"], ckpt_positions=i32(ck),
            ckpt_positions_host=ck, ckpt_buf=r["kept"], conv_weight=self.w, conv_bias=self.b, conv_state_in=win,
            conv_state_out=r.get("window"), conv_ckpt=r.get("window_kept"), workspace=workspace, stream=stream)
        return r

    def check(self, r, want, ckpts=()):
        T, longest = int(self.cu[-1]), max(self.lens + [0])
        assert bool((r["out"][T:] == 7.0).all()), "rows behind the last prompt"
        close(r["out"][:T], want["out"], out_tol(want["out"], want["out_mass"]), "out")
        close(r["final"], want["final"], state_tol(want["final_mass"], longest), "final")
        if len(ckpts):
            close(r["kept"], want["kept"], state_tol(want["kept_mass"], longest), "kept")
        if self.w is not None:
            assert np.array_equal(f64(r["window"]), want["window"])
            if len(ckpts):
                assert np.array_equal(f64(r["window_kept"]), want["window_kept"])

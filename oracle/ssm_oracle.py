"""fp64 oracle of the state space layers and of the norm, token by token and
row by row, with the absolute sums ("masses") that error bounds are made of."""
from __future__ import annotations

import numpy as np


def conv(x, w, bias, before):
    """silu(bias + four taps) of one prompt's rows x [L, C] after its window
    `before` [3, C]; and |bias| + sum |w| |x|, what a rounded sum errs by."""
    ext = np.concatenate([before, x])
    L = len(x)
    z = np.zeros_like(x) if bias is None else np.broadcast_to(bias, x.shape).copy()
    m = np.abs(z)
    for k in range(4):
        z = z + w[:, k] * ext[k:k + L]
        m = m + np.abs(w[:, k] * ext[k:k + L])
    with np.errstate(over="ignore"):
        return z / (1.0 + np.exp(-z)), m


def steps(raw, bias, softplus=True, lo=0.0, hi=np.inf):
    v = raw if bias is None else raw + bias
    if softplus:
        v = np.maximum(v, 0.0) + np.log1p(np.exp(-np.abs(v)))
    return np.clip(v, lo, hi)


class Scan:
    """One sequence's recurrence: state [H, P, N], and its mass."""

    def __init__(self, H, G, P, N, A, D, state=None):
        self.H, self.G, self.P, self.N, self.A = H, G, P, N, A
        self.D = np.zeros(H) if D is None else D
        self.S = np.zeros((H, P, N)) if state is None else state.copy()
        self.mass = np.abs(self.S)

    def split(self, u):
        H, G, P, N = self.H, self.G, self.P, self.N
        rep = lambda a: np.repeat(a.reshape(G, N), H // G, axis=0)
        return u[:H * P].reshape(H, P), rep(u[H * P:H * P + G * N]), rep(u[H * P + G * N:])

    def token(self, u, um, dt):
        """Output [H, P] and its mass; um: magnitudes that |u| may stand for."""
        x, B, C = self.split(u)
        xm, Bm, Cm = self.split(um)
        al = np.exp(self.A * dt)[:, None, None]
        self.S = al * self.S + (dt[:, None] * x)[:, :, None] * B[:, None, :]
        self.mass = al * self.mass + (np.abs(dt)[:, None] * xm)[:, :, None] * Bm[:, None, :]
        y = np.einsum("hpn,hn->hp", self.S, C) + self.D[:, None] * x
        return y, np.einsum("hpn,hn->hp", self.mass, Cm) + np.abs(self.D)[:, None] * xm


def prefill(H, G, P, N, cu, x, dt, A, D=None, conv_w=None, conv_b=None, window=None, init=None, ckpts=()):
    """dict of out, out_mass [T, H, P], final, final_mass [n, H, P, N], kept,
    kept_mass [k, H, P, N], window, window_kept."""
    n = len(cu) - 1
    T, C = x.shape
    r = dict(out=np.zeros((T, H, P)), out_mass=np.zeros((T, H, P)), final=[], final_mass=[], kept=[], kept_mass=[], window=[],
             window_kept=[])
    for s in range(n):
        rows = x[cu[s]:cu[s + 1]]
        before = np.zeros((3, C)) if window is None else window[s]
        u, um = (rows, np.abs(rows)) if conv_w is None else conv(rows, conv_w, conv_b, before)
        um = np.abs(u) + um
        ext = np.concatenate([before, rows])
        sc = Scan(H, G, P, N, A, D, None if init is None else init[s])
        for i in range(len(rows)):
            t = cu[s] + i
            r["out"][t], r["out_mass"][t] = sc.token(u[i], um[i], dt[t])
            if t + 1 in ckpts:
                r["kept"].append(sc.S.copy())
                r["kept_mass"].append(sc.mass.copy())
                r["window_kept"].append(ext[i + 1:i + 4])
        r["final"].append(sc.S)
        r["final_mass"].append(sc.mass)
        r["window"].append(ext[-3:])
    return {k: v if isinstance(v, np.ndarray) else np.array(v) for k, v in r.items()}


def silu(z):
    return z / (1.0 + np.exp(-z))


def rms_norm(x, w=None, residual=None, gate=None, gate_first=False, groups=1, eps=1e-6, offset=0.0):
    """(y, r): the normed rows and the sums x + residual."""
    r = x if residual is None else x + residual
    v = r * silu(gate) if gate is not None and gate_first else r
    g = v.reshape(len(v), groups, -1)
    y = (g / np.sqrt((g * g).mean(-1, keepdims=True) + eps)).reshape(v.shape)
    if w is not None:
        y = y * np.tile(w + offset, v.shape[1] // len(w))
    if gate is not None and not gate_first:
        y = y * silu(gate)
    return y, r

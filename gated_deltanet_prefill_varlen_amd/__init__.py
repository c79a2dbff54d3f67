"""Python binding of libgdn (packed gated-delta-rule prefill, checkpoints,
decode, short conv and checkpoint copy; the paged 8-bit key/value cache of the
softmax-attention layers with the attention over it; the scan and decode step of
state space layers; and the norm around these layers, on MI355X / gfx950).

Argument marshalling only: every function here passes torch tensor data
pointers, sizes and the current HIP stream to the C entry point of the same
name in ``libgdn.so`` and raises ``GdnError`` on a non-OK status.  All compute
runs in the library's HIP kernels; there is no other implementation behind
these names, and importing fails loudly when the library is not built.

torch is imported before the library is loaded so that the process holds a
single HIP runtime (torch's), which makes torch streams, events and device
pointers valid handles for libgdn.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional, Sequence

import numpy as np
import torch

__all__ = [
    "GdnError", "gdn_shape", "make_shape", "load", "GDN_BF16", "GDN_F32", "GDN_QK_L2NORM",
    "gdn_status_string", "gdn_plan_checkpoints", "gdn_prefill_packed", "gdn_prefill_conv_packed",
    "gdn_decode_step", "gdn_decode_tokens",
    "gdn_conv1d_silu_packed", "gdn_snapshot_copy", "LIB_PATH", "EXPORTED",
    "gdn_cache", "gdn_rope", "make_cache", "make_rope", "GDN_E4M3", "GDN_I8",
    "gdn_plan_pages", "gdn_rope_append", "gdn_cache_gather", "gdn_attn_packed", "gdn_attn_decode",
    "gdn_attn_decode_workspace",
    "gdn_ssm_shape", "gdn_norm_shape", "make_ssm", "make_norm", "gdn_ssm_prefill_workspace",
    "gdn_ssm_prefill_packed", "gdn_ssm_decode", "gdn_rms_norm",
]

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libgdn.so")
GDN_BF16, GDN_F32, GDN_E4M3, GDN_I8 = 0, 1, 2, 3
GDN_QK_L2NORM = 1
GDN_SSM_SOFTPLUS = 1
GDN_NORM_GATE_FIRST = 1
STATUS = {0: "GDN_OK", 1: "GDN_ERR_NULL", 2: "GDN_ERR_SHAPE", 3: "GDN_ERR_UNSUPPORTED",
          4: "GDN_ERR_SEQLENS", 5: "GDN_ERR_CKPT", 6: "GDN_ERR_CAPACITY", 7: "GDN_ERR_HIP"}
EXPORTED = ("gdn_status_string", "gdn_plan_checkpoints", "gdn_conv1d_silu_packed",
            "gdn_prefill_packed", "gdn_prefill_conv_packed", "gdn_decode_step",
            "gdn_decode_tokens", "gdn_snapshot_copy", "gdn_plan_pages", "gdn_rope_append",
            "gdn_cache_gather", "gdn_attn_packed", "gdn_attn_decode", "gdn_attn_decode_workspace",
            "gdn_ssm_prefill_workspace", "gdn_ssm_prefill_packed", "gdn_ssm_decode", "gdn_rms_norm")


class GdnError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {gdn_status_string(status)}")


class gdn_shape(ctypes.Structure):
    _fields_ = [
        ("num_qk_heads", ctypes.c_int32), ("num_v_heads", ctypes.c_int32),
        ("head_k_dim", ctypes.c_int32), ("head_v_dim", ctypes.c_int32),
        ("chunk", ctypes.c_int32), ("io_dtype", ctypes.c_int32), ("flags", ctypes.c_uint32),
        ("scale", ctypes.c_float), ("l2_eps", ctypes.c_float), ("reserved", ctypes.c_int32),
        ("q_tok_stride", ctypes.c_int64), ("k_tok_stride", ctypes.c_int64),
        ("v_tok_stride", ctypes.c_int64),
    ]


def make_shape(Hqk: int, Hv: int, dk: int, dv: int, chunk: int = 64, io_dtype: int = GDN_BF16,
               l2norm: bool = True, scale: float = 1.0, l2_eps: float = 1e-6,
               q_tok_stride: int = 0, k_tok_stride: int = 0, v_tok_stride: int = 0) -> gdn_shape:
    return gdn_shape(Hqk, Hv, dk, dv, chunk, io_dtype, GDN_QK_L2NORM if l2norm else 0,
                     scale, l2_eps, 0, q_tok_stride, k_tok_stride, v_tok_stride)


class gdn_cache(ctypes.Structure):
    _fields_ = [
        ("num_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32), ("page", ctypes.c_int32),
        ("code_dtype", ctypes.c_int32), ("n_pages", ctypes.c_int32), ("reserved", ctypes.c_int32),
        ("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
        ("v_scale", ctypes.c_void_p),
    ]
    device = -1


class gdn_rope(ctypes.Structure):
    _fields_ = [
        ("rot_dim", ctypes.c_int32), ("n_axes", ctypes.c_int32), ("adjacent", ctypes.c_int32),
        ("scale", ctypes.c_float), ("freq", ctypes.c_float * 128), ("axis", ctypes.c_uint8 * 128),
    ]


class gdn_ssm_shape(ctypes.Structure):
    _fields_ = [
        ("num_heads", ctypes.c_int32), ("num_groups", ctypes.c_int32), ("head_dim", ctypes.c_int32),
        ("state_dim", ctypes.c_int32), ("flags", ctypes.c_uint32), ("dt_min", ctypes.c_float),
        ("dt_max", ctypes.c_float), ("reserved", ctypes.c_int32),
    ]


def make_ssm(H: int, G: int, P: int, N: int, softplus: bool = True, dt_min: float = 0.0,
             dt_max: float = float("inf")) -> gdn_ssm_shape:
    """A state space layer of H heads of P channels, G groups of B and C, N state columns."""
    return gdn_ssm_shape(H, G, P, N, GDN_SSM_SOFTPLUS if softplus else 0, dt_min, dt_max, 0)


class gdn_norm_shape(ctypes.Structure):
    _fields_ = [
        ("dim", ctypes.c_int32), ("groups", ctypes.c_int32), ("weight_dim", ctypes.c_int32),
        ("scale_block", ctypes.c_int32), ("flags", ctypes.c_uint32), ("eps", ctypes.c_float),
        ("weight_offset", ctypes.c_float), ("reserved", ctypes.c_int32),
    ]


def make_norm(dim: int, groups: int = 1, eps: float = 1e-6, gate_first: bool = False, scale_block: int = 0,
              weight_offset: float = 0.0, shared_weight: bool = False) -> gdn_norm_shape:
    """A norm over dim channels in groups; shared_weight: one weight of dim / groups for all groups."""
    return gdn_norm_shape(dim, groups, dim // groups if shared_weight and groups > 0 else dim, scale_block,
                          GDN_NORM_GATE_FIRST if gate_first else 0, eps, weight_offset, 0)


_CODES = {torch.float8_e4m3fn: GDN_E4M3, torch.int8: GDN_I8}


def make_cache(k: torch.Tensor, v: torch.Tensor, k_scale: torch.Tensor,
               v_scale: torch.Tensor) -> gdn_cache:
    """Handle of a paged cache: k [n_pages, Hkv, page, d] and v [n_pages, Hkv,
    page/16, d, 16] of torch.float8_e4m3fn or torch.int8, scales [n_pages, Hkv]
    fp32.  The handle keeps its tensors alive; nothing needs clearing."""
    if k.dim() != 4 or k.dtype not in _CODES:
        raise ValueError("k must be [n_pages, Hkv, page, d] of float8_e4m3fn or int8")
    n, h, page, d = k.shape
    if v.dtype != k.dtype or tuple(v.shape) != (n, h, page // 16, d, 16):
        raise ValueError("v must be [n_pages, Hkv, page/16, d, 16] of k's dtype")
    for t in (k_scale, v_scale):
        if t.dtype != torch.float32 or tuple(t.shape) != (n, h):
            raise ValueError("scales must be fp32 [n_pages, Hkv]")
    dev = k.get_device()
    c = gdn_cache(h, d, page, _CODES[k.dtype], n, 0, _buf(k, k.dtype, dev, "k"), _buf(v, k.dtype, dev, "v"),
                  _buf(k_scale, torch.float32, dev, "k_scale"), _buf(v_scale, torch.float32, dev, "v_scale"))
    if dev < 0:
        raise ValueError("the cache is not on the GPU")
    c.device = dev
    c.tensors = (k, v, k_scale, v_scale)
    return c


def make_rope(freq: Sequence[float], axis: Optional[Sequence[int]] = None, n_axes: int = 1,
              adjacent: bool = False, scale: float = 1.0) -> gdn_rope:
    """Rotary plan: freq in radians per position (up to 65,536 in size) of each
    of rot_dim / 2 pairs, axis the position row (below n_axes) that turns each
    pair (default 0)."""
    freq = [float(f) for f in freq]
    axis = [0] * len(freq) if axis is None else [int(i) for i in axis]
    if len(freq) > 128 or len(axis) != len(freq) or any(not 0 <= i < n_axes for i in axis):
        raise ValueError("at most 128 pairs, each with an axis below n_axes")
    return gdn_rope(2 * len(freq), n_axes, int(adjacent), scale, (ctypes.c_float * 128)(*freq),
                    (ctypes.c_uint8 * 128)(*axis))


_lib: Optional[ctypes.CDLL] = None
_P = ctypes.c_void_p
_I32 = ctypes.c_int32
_I64 = ctypes.c_int64
_SP = ctypes.POINTER(gdn_shape)


def load() -> ctypes.CDLL:
    """Load libgdn.so (built in-tree); raises if it is missing."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"libgdn.so is not built ({LIB_PATH}); run __graft_entry__.build() "
                           "or python gated_deltanet_prefill_varlen_amd/build.py")
    lib = ctypes.CDLL(LIB_PATH)
    lib.gdn_status_string.restype = ctypes.c_char_p
    lib.gdn_status_string.argtypes = [_I32]
    lib.gdn_plan_checkpoints.restype = _I32
    lib.gdn_plan_checkpoints.argtypes = [_P, _I32, _P, _I32, _I32, _P, _I32, _P]
    lib.gdn_prefill_packed.restype = _I32
    lib.gdn_prefill_packed.argtypes = [_SP, _P, _P, _I32, _I32, _P, _P, _P, _P, _P, _P,
                                       _P, _P, _I32, _P, _P, _P, _P]
    lib.gdn_prefill_conv_packed.restype = _I32
    lib.gdn_prefill_conv_packed.argtypes = [_SP, _P, _P, _I32, _I32, _P, _I64, _P, _P, _P, _P, _P,
                                            _P, _P, _P, _I32, _P, _P, _P, _P, _P]
    lib.gdn_decode_step.restype = _I32
    lib.gdn_decode_step.argtypes = [_SP, _I32, _P, _P, _P, _P, _P, _P, _I64, _P, _P, _P, _P, _P, _P]
    lib.gdn_decode_tokens.restype = _I32
    lib.gdn_decode_tokens.argtypes = [_SP, _I32, _I32, _P, _P, _P, _P, _P, _P, _I64, _P, _P, _P, _P,
                                      _P, _P, _P]
    lib.gdn_conv1d_silu_packed.restype = _I32
    lib.gdn_conv1d_silu_packed.argtypes = [_SP, _P, _P, _I32, _I32, _P, _I64, _P, _P, _P, _I64,
                                           _P, _P, _P, _I32, _P, _P]
    lib.gdn_snapshot_copy.restype = _I32
    lib.gdn_snapshot_copy.argtypes = [_P, _I32, _I64, _P, _I64, _P, _P, _P, _P, _P]
    lib.gdn_plan_pages.restype = _I32
    lib.gdn_plan_pages.argtypes = [_I32, _I32, _P, _P, _P, _P, _I32, _P, _P, _P, _I32, _P, _P, _I32,
                                   _P, _P, _P]
    lib.gdn_rope_append.restype = _I32
    lib.gdn_rope_append.argtypes = [_P, _P, _I32, _P, _P, _I32, _I32, _P, _I64, _P, _I64, _P, _I64,
                                    _P, _I64, _P, _P, _I64, _P]
    lib.gdn_cache_gather.restype = _I32
    lib.gdn_cache_gather.argtypes = [_P, _I32, _P, _P, _P, _P]
    lib.gdn_attn_packed.restype = _I32
    lib.gdn_attn_packed.argtypes = [_P, _I32, ctypes.c_float, _P, _P, _I32, _I32, _P, _P, _I32, _P,
                                    _I64, _P, _P]
    lib.gdn_attn_decode.restype = _I32
    lib.gdn_attn_decode.argtypes = [_P, _I32, ctypes.c_float, _I32, _I32, _P, _P, _I32, _I32, _P,
                                    _I64, _P, _P, _I64, _P]
    lib.gdn_attn_decode_workspace.restype = _I32
    lib.gdn_attn_decode_workspace.argtypes = [_P, _I32, _I32, _I32, _I32, _P]
    lib.gdn_ssm_prefill_workspace.restype = _I32
    lib.gdn_ssm_prefill_workspace.argtypes = [_P, _P, _I32, _I32, _P]
    lib.gdn_ssm_prefill_packed.restype = _I32
    lib.gdn_ssm_prefill_packed.argtypes = [_P, _P, _P, _I32, _I32, _P, _I64, _P, _P, _P, _P, _I32, _P, _I64, _P, _P, _P,
                                           _P, _P, _P, _I32, _P, _P, _P, _P, _P, _I64, _P]
    lib.gdn_ssm_decode.restype = _I32
    lib.gdn_ssm_decode.argtypes = [_P, _I32, _I32, _P, _I64, _P, _P, _P, _I32, _P, _I64, _P, _P, _P, _P, _I64, _P, _P,
                                   _P, _P, _P]
    lib.gdn_rms_norm.restype = _I32
    lib.gdn_rms_norm.argtypes = [_P, _I32, _I32, _P, _I64, _I32, _P, _I64, _P, _P, _I64, _P, _P, _I32, _P, _P, _P]
    _lib = lib
    return lib


def gdn_status_string(status: int) -> str:
    return load().gdn_status_string(int(status)).decode()


# ------------------------------------------------------------ marshalling --

def _dev(t) -> Optional[int]:
    """Device pointer of a tensor (None passes NULL)."""
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError("device arguments must be torch tensors")
    if not t.is_cuda:
        raise ValueError("device argument is not on the GPU")
    return t.data_ptr()


def _buf(t: Optional[torch.Tensor], dtype: torch.dtype, dev: int, what: str = "argument") -> Optional[int]:
    """Device pointer of a dense tensor of one type on device dev."""
    if t is None:
        return None
    if t.dtype is not dtype or not t.is_contiguous() or t.get_device() != dev:
        _refuse(t, dtype, what)
    return t.data_ptr()


def _refuse(t: torch.Tensor, dtype: torch.dtype, what: str) -> None:
    if t.dtype is not dtype:
        raise TypeError(f"{what} must be {dtype}, got {t.dtype}")
    raise ValueError(f"{what} must be contiguous" if t.is_cuda and not t.is_contiguous() else
                     f"{what} is not on the current device" if t.is_cuda else f"{what} is not on the GPU")


def _rows(t: torch.Tensor, rows: int, heads: Optional[int], d: int, dev: int, what: str):
    """Pointer, token stride and head count of bf16 rows [>= rows, heads, d]
    whose heads are dense (columns of a wider row will do)."""
    if t.dtype is not torch.bfloat16 or t.get_device() != dev:
        _refuse(t, torch.bfloat16, what)
    n, h, e = t.shape if t.dim() == 3 else (0, 0, 0)
    if e != d or n < rows or (heads is not None and h != heads):
        raise ValueError(f"{what} must be [{rows}, {'heads' if heads is None else heads}, {d}], got {tuple(t.shape)}")
    st = t.stride()
    if st[2] != 1 or (h > 1 and st[1] != d):
        raise ValueError(f"{what}: the heads of a token must be dense")
    if n > 1 and st[0] < h * d:   # (0 would mean dense rows)
        raise ValueError(f"{what}: the rows overlap")
    return t.data_ptr(), (st[0] if n > 1 else h * d), h


def _where(stream):
    """Current device (one that no tensor is on while there is none) and the
    stream's handle."""
    if not torch.cuda.is_initialized():
        return -2, None
    dev = torch.cuda.current_device()
    if isinstance(stream, torch.cuda.Stream) and stream.device_index != dev:
        raise ValueError("the stream is not on the current device")
    return dev, (torch._C._cuda_getCurrentRawStream(dev) or None) if stream is None else _stream(stream)


def _host_i32(a) -> Optional[np.ndarray]:
    if type(a) is np.ndarray and a.dtype == np.int32 and a.flags.c_contiguous:
        return a
    if a is None:
        return None
    if isinstance(a, torch.Tensor):
        a = a.detach().cpu().numpy()
    return np.ascontiguousarray(np.asarray(a), dtype=np.int32)


def _host_i64(a) -> Optional[np.ndarray]:
    if a is None:
        return None
    if isinstance(a, torch.Tensor):
        a = a.detach().cpu().numpy()
    return np.ascontiguousarray(np.asarray(a), dtype=np.int64)


def _hp(a: Optional[np.ndarray]) -> Optional[int]:
    return None if a is None else a.ctypes.data


def _stream(stream) -> Optional[int]:
    if stream is None:
        stream = torch.cuda.current_stream()
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream or None
    return int(stream) or None


def _event(ev) -> Optional[int]:
    if ev is None:
        return None
    if isinstance(ev, torch.cuda.Event):
        return ev.cuda_event or None
    return int(ev) or None


def _record_target(ev) -> Optional[int]:
    """Handle of an event the library records.  torch makes an event's HIP
    handle only at its first record, and a null handle would leave the event
    unrecorded (a later wait on it would not wait), so a fresh torch event is
    recorded once on the current stream first; the library's own record after
    its work is the one every later wait sees."""
    if isinstance(ev, torch.cuda.Event) and not ev.cuda_event:
        ev.record()
    return _event(ev)


def _check(status: int, where: str) -> None:
    if status != 0:
        raise GdnError(status, where)


# -------------------------------------------------------------- functions --

def gdn_plan_checkpoints(cu_seqlens_host, block: int, tail: int = 16,
                         p0_host=None) -> np.ndarray:
    """Checkpoint positions (int32 global offsets) for a pack; host only."""
    lib = load()
    cu = _host_i32(cu_seqlens_host)
    p0 = _host_i32(p0_host)
    n = ctypes.c_int32(0)
    st = lib.gdn_plan_checkpoints(_hp(cu), len(cu) - 1, _hp(p0), block, tail, None, 0,
                                  ctypes.byref(n))
    if st not in (0, 6):
        _check(st, "gdn_plan_checkpoints")
    out = np.zeros(max(n.value, 1), dtype=np.int32)
    _check(lib.gdn_plan_checkpoints(_hp(cu), len(cu) - 1, _hp(p0), block, tail, _hp(out),
                                    n.value, ctypes.byref(n)), "gdn_plan_checkpoints")
    return out[:n.value]


def gdn_prefill_packed(shape: gdn_shape, cu_seqlens, cu_seqlens_host, q, k, v, g, beta,
                       init_state, ckpt_positions, ckpt_positions_host, out, final_state,
                       ckpt_buf, stream=None) -> None:
    cu_h = _host_i32(cu_seqlens_host)
    ck_h = _host_i32(ckpt_positions_host)
    n_ckpt = 0 if ck_h is None else len(ck_h)
    n_tokens = int(cu_h[-1]) if len(cu_h) else 0
    _check(load().gdn_prefill_packed(
        ctypes.byref(shape), _dev(cu_seqlens), _hp(cu_h), len(cu_h) - 1, n_tokens,
        _dev(q), _dev(k), _dev(v), _dev(g), _dev(beta), _dev(init_state),
        _dev(ckpt_positions), _hp(ck_h), n_ckpt, _dev(out), _dev(final_state), _dev(ckpt_buf),
        _stream(stream)), "gdn_prefill_packed")


def gdn_prefill_conv_packed(shape: gdn_shape, cu_seqlens, cu_seqlens_host, x, conv_weight, g,
                            beta, init_state, ckpt_positions, ckpt_positions_host, out,
                            final_state, ckpt_buf, conv_state_in=None, conv_state_out=None,
                            conv_ckpt=None, x_tok_stride: int = 0, stream=None) -> None:
    """The packed prefill reading pre-conv rows x (the short conv fused into
    the scan's loads)."""
    cu_h = _host_i32(cu_seqlens_host)
    ck_h = _host_i32(ckpt_positions_host)
    n_ckpt = 0 if ck_h is None else len(ck_h)
    n_tokens = int(cu_h[-1]) if len(cu_h) else 0
    _check(load().gdn_prefill_conv_packed(
        ctypes.byref(shape), _dev(cu_seqlens), _hp(cu_h), len(cu_h) - 1, n_tokens,
        _dev(x), x_tok_stride, _dev(conv_weight), _dev(conv_state_in), _dev(conv_state_out),
        _dev(g), _dev(beta), _dev(init_state), _dev(ckpt_positions), _hp(ck_h), n_ckpt,
        _dev(conv_ckpt), _dev(out), _dev(final_state), _dev(ckpt_buf), _stream(stream)),
        "gdn_prefill_conv_packed")


def gdn_decode_step(shape: gdn_shape, q, k, v, g, beta, state, slot=None, slot_host=None,
                    out=None, conv_w=None, conv_state=None, stream=None) -> None:
    """One token per sequence; with conv_w and conv_state, q, k, v are the
    conv's inputs and the slots' conv windows move on by one token."""
    sl_h = _host_i32(slot_host)
    _check(load().gdn_decode_step(
        ctypes.byref(shape), int(q.shape[0]), _dev(q), _dev(k), _dev(v), _dev(g), _dev(beta),
        _dev(state), int(state.shape[0]), _dev(slot), _hp(sl_h), _dev(out), _dev(conv_w),
        _dev(conv_state), _stream(stream)), "gdn_decode_step")


def gdn_decode_tokens(shape: gdn_shape, n_tok: int, q, k, v, g, beta, state, slot=None,
                      slot_host=None, out=None, snapshots=None, conv_w=None, conv_state=None,
                      stream=None) -> None:
    """n_tok tokens per sequence (rows b * n_tok + i), states kept per token."""
    sl_h = _host_i32(slot_host)
    batch = int(q.shape[0]) // int(n_tok)
    _check(load().gdn_decode_tokens(
        ctypes.byref(shape), batch, int(n_tok), _dev(q), _dev(k), _dev(v), _dev(g), _dev(beta),
        _dev(state), int(state.shape[0]), _dev(slot), _hp(sl_h), _dev(out), _dev(snapshots),
        _dev(conv_w), _dev(conv_state), _stream(stream)), "gdn_decode_tokens")


def gdn_conv1d_silu_packed(shape: gdn_shape, cu_seqlens, cu_seqlens_host, x, weight, y,
                           conv_state_in=None, conv_state_out=None, ckpt_positions=None,
                           ckpt_positions_host=None, conv_ckpt=None, x_tok_stride: int = 0,
                           y_tok_stride: int = 0, stream=None) -> None:
    cu_h = _host_i32(cu_seqlens_host)
    ck_h = _host_i32(ckpt_positions_host)
    n_ckpt = 0 if ck_h is None else len(ck_h)
    _check(load().gdn_conv1d_silu_packed(
        ctypes.byref(shape), _dev(cu_seqlens), _hp(cu_h), len(cu_h) - 1, int(cu_h[-1]),
        _dev(x), x_tok_stride, _dev(weight), _dev(conv_state_in), _dev(y), y_tok_stride,
        _dev(conv_state_out), _dev(ckpt_positions), _hp(ck_h), n_ckpt, _dev(conv_ckpt),
        _stream(stream)), "gdn_conv1d_silu_packed")


def gdn_snapshot_copy(ckpt_buf, n: int, bytes_each: int, dst_pool, dst_slot, dst_slot_host,
                      pool_slots: int, wait_event=None, copy_stream=None, done_event=None) -> None:
    """Copy n checkpoint items of bytes_each bytes into pool slots.  dst_pool is
    a device tensor, or an int device address of mapped pinned host memory.
    copy_stream first waits for wait_event; done_event is recorded on
    copy_stream after the copy."""
    sl_h = _host_i64(dst_slot_host)
    dst = dst_pool if isinstance(dst_pool, int) else _dev(dst_pool)
    _check(load().gdn_snapshot_copy(
        _dev(ckpt_buf), int(n), int(bytes_each), dst, int(pool_slots), _dev(dst_slot), _hp(sl_h),
        _event(wait_event), _stream(copy_stream), _record_target(done_event)), "gdn_snapshot_copy")


def _cache(cache: gdn_cache, dev: int) -> int:
    """Address of a cache's handle; its tensors must be on device dev."""
    if cache.device != dev:
        raise ValueError("the cache is not on the current device")
    return ctypes.addressof(cache)


def gdn_plan_pages(page: int, want_len, kv_len, kv_len_out, block_table, free_pages, free_count,
                   free_count_out, cu_seqlens, slot_map, positions, status, stream=None) -> None:
    """Block tables, the pack of new tokens and its slot map, from the lengths
    that the requests hold (kv_len) and want; all on the device.  No two rows of
    block_table may share a page: it is free again when its request ends."""
    i32 = torch.int32
    dev, st = _where(stream)
    n, (rows, max_pages) = want_len.numel(), block_table.shape
    if (rows < n or kv_len.numel() < n or kv_len_out.numel() < n or status.numel() < n or
            cu_seqlens.numel() < n + 1):
        raise ValueError("a buffer is shorter than the requests")
    if positions is not None and positions.numel() < slot_map.numel():
        raise ValueError("positions is shorter than slot_map")
    if free_count.numel() < 1 or free_count_out.numel() < 1:
        raise ValueError("free_count is empty")
    _check(load().gdn_plan_pages(
        page, n, _buf(want_len, i32, dev, "want_len"), _buf(kv_len, i32, dev, "kv_len"),
        _buf(kv_len_out, i32, dev, "kv_len_out"), _buf(block_table, i32, dev, "block_table"), max_pages,
        _buf(free_pages, i32, dev, "free_pages"), _buf(free_count, i32, dev, "free_count"),
        _buf(free_count_out, i32, dev, "free_count_out"), free_pages.numel(),
        _buf(cu_seqlens, i32, dev, "cu_seqlens"), _buf(slot_map, torch.int64, dev, "slot_map"),
        slot_map.numel(), _buf(positions, i32, dev, "positions"), _buf(status, i32, dev, "status"),
        st), "gdn_plan_pages")


def gdn_rope_append(rope: gdn_rope, cache: gdn_cache, cu_seqlens, cu_seqlens_host, q, k, v, positions,
                    slot_map, q_out, stream=None) -> None:
    """q_out = rotated q; rotated k and v into their cache slots.  q, k, v are
    [T, heads, d] bf16, views of one wider row if need be; positions [n_axes, T],
    or [T] for every axis; q and q_out None: only the cache is written."""
    dev, st = _where(stream)
    cu_h = _host_i32(cu_seqlens_host)
    n = len(cu_h) - 1
    T, d, hkv = int(cu_h[-1]), cache.head_dim, cache.num_kv_heads
    qp = qs = qo = qos = None
    hq = 0
    if (q is None) != (q_out is None):
        raise ValueError("q and q_out go together")
    if q is not None:
        qp, qs, hq = _rows(q, T, None, d, dev, "q")
        qo, qos, _ = _rows(q_out, T, hq, d, dev, "q_out")
    kp, ks, _ = _rows(k, T, hkv, d, dev, "k")
    vp, vs, _ = _rows(v, T, hkv, d, dev, "v")
    pos_stride = 0
    if positions is not None:
        if positions.shape[-1] < T or (positions.dim() == 2 and positions.shape[0] < rope.n_axes) or positions.dim() > 2:
            raise ValueError("positions must be [T] or [n_axes, T]")
        pos_stride = positions.shape[-1] if positions.dim() == 2 else 0
    if slot_map.numel() < T or cu_seqlens.numel() < n + 1:
        raise ValueError("slot_map or cu_seqlens is shorter than the pack")
    _check(load().gdn_rope_append(
        ctypes.addressof(rope), _cache(cache, dev), hq, _buf(cu_seqlens, torch.int32, dev, "cu_seqlens"),
        cu_h.ctypes.data, n, T, qp, qs or 0, kp, ks, vp, vs, _buf(positions, torch.int32, dev, "positions"),
        pos_stride, _buf(slot_map, torch.int64, dev, "slot_map"), qo, qos or 0, st),
        "gdn_rope_append")


def gdn_cache_gather(cache: gdn_cache, slot_map, k_out=None, v_out=None, stream=None) -> None:
    """k_out, v_out [T, Hkv, d] bf16: the values held at the T slots."""
    dev, st = _where(stream)
    T = slot_map.numel()
    for t in (k_out, v_out):
        if t is not None and tuple(t.shape) != (T, cache.num_kv_heads, cache.head_dim):
            raise ValueError("outputs must be [T, Hkv, d]")
    _check(load().gdn_cache_gather(
        _cache(cache, dev), T, _buf(slot_map, torch.int64, dev, "slot_map"),
        _buf(k_out, torch.bfloat16, dev, "k_out"), _buf(v_out, torch.bfloat16, dev, "v_out"), st),
        "gdn_cache_gather")


def gdn_attn_packed(cache: gdn_cache, cu_seqlens, cu_seqlens_host, kv_len, block_table, q, out,
                    scale: Optional[float] = None, stream=None) -> None:
    """Causal attention of a pack's rows over the cache (which holds them);
    scale defaults to d ** -0.5."""
    dev, st = _where(stream)
    cu_h = _host_i32(cu_seqlens_host)
    n = len(cu_h) - 1
    T, d = int(cu_h[-1]), cache.head_dim
    qp, qs, hq = _rows(q, T, None, d, dev, "q")
    if tuple(out.shape[1:]) != (hq, d) or out.shape[0] < T:
        raise ValueError("out must be [T, Hq, d]")
    if kv_len.numel() < n or block_table.shape[0] < n or cu_seqlens.numel() < n + 1:
        raise ValueError("kv_len, block_table or cu_seqlens is shorter than the prompts")
    _check(load().gdn_attn_packed(
        _cache(cache, dev), hq, d ** -0.5 if scale is None else scale,
        _buf(cu_seqlens, torch.int32, dev, "cu_seqlens"), cu_h.ctypes.data, n, T,
        _buf(kv_len, torch.int32, dev, "kv_len"), _buf(block_table, torch.int32, dev, "block_table"),
        block_table.shape[1], qp, qs, _buf(out, torch.bfloat16, dev, "out"), st),
        "gdn_attn_packed")


def gdn_attn_decode_workspace(cache: gdn_cache, num_q_heads: int, batch: int, n_tok: int,
                              max_kv_len: int) -> int:
    """Bytes of workspace of gdn_attn_decode."""
    n = ctypes.c_int64(0)
    _check(load().gdn_attn_decode_workspace(ctypes.addressof(cache), num_q_heads, batch, n_tok,
                                            max_kv_len, ctypes.byref(n)), "gdn_attn_decode_workspace")
    return n.value


def gdn_attn_decode(cache: gdn_cache, n_tok: int, kv_len, block_table, q, out,
                    max_kv_len: Optional[int] = None, scale: Optional[float] = None, workspace=None,
                    stream=None) -> None:
    """Causal attention of n_tok rows per request (q [batch * n_tok, Hq, d])
    over the cache.  workspace: a uint8 tensor of gdn_attn_decode_workspace()
    bytes; max_kv_len: an upper bound of kv_len (default: the table's pages)."""
    dev, st = _where(stream)
    B, max_pages = kv_len.numel(), block_table.shape[1]
    d = cache.head_dim
    qp, qs, hq = _rows(q, B * n_tok, None, d, dev, "q")
    if tuple(out.shape[1:]) != (hq, d) or out.shape[0] < B * n_tok:
        raise ValueError("out must be [batch * n_tok, Hq, d]")
    if block_table.shape[0] < B:
        raise ValueError("block_table is shorter than the batch")
    _check(load().gdn_attn_decode(
        _cache(cache, dev), hq, d ** -0.5 if scale is None else scale, B, n_tok,
        _buf(kv_len, torch.int32, dev, "kv_len"), _buf(block_table, torch.int32, dev, "block_table"), max_pages,
        min(max_pages * cache.page, 2**31 - 1) if max_kv_len is None else max_kv_len, qp, qs,
        _buf(out, torch.bfloat16, dev, "out"), _buf(workspace, torch.uint8, dev, "workspace"),
        0 if workspace is None else workspace.numel(), st), "gdn_attn_decode")


# ------------------------------------------------- state space layers, norm --

_IO = {torch.bfloat16: GDN_BF16, torch.float32: GDN_F32}


def _row_stride(t: torch.Tensor, rows: int, width: int, dev: int, what: str, dtype=None, exact: bool = False):
    """Pointer and row stride of rows [>= rows, width] (exact: [rows, width])
    with dense channels (columns of a wider row will do); 0 rows: no pointer."""
    if t.get_device() != dev or (t.dtype not in _IO if dtype is None else t.dtype is not dtype):
        _refuse(t, dtype or (t.dtype if t.dtype in _IO else torch.bfloat16), what)
    n, w = t.shape if t.dim() == 2 else (-1, -1)
    if w != width or (n != rows if exact else n < rows):
        raise ValueError(f"{what} must be [{rows}, {width}], got {tuple(t.shape)}")
    row, one = t.stride()
    if one != 1 and width > 1:
        raise ValueError(f"{what}: the channels of a row must be dense")
    if n < 2:
        row = 0
    elif row < width:
        raise ValueError(f"{what}: the rows overlap")
    return (t.data_ptr() if rows else None), row


def _sized(t, dtype, dev: int, shape, what: str) -> Optional[int]:
    """Pointer of a dense tensor of one type and shape (None passes NULL)."""
    if t is None:
        return None
    if t.shape != shape:
        raise ValueError(f"{what} must be {list(shape)}, got {tuple(t.shape)}")
    if t.dtype is not dtype or not t.is_contiguous() or t.get_device() != dev:
        _refuse(t, dtype, what)
    return t.data_ptr()


def _ssm_dims(shape: gdn_ssm_shape):
    return shape.num_heads, shape.head_dim, shape.state_dim, (shape.num_heads * shape.head_dim +
                                                              2 * shape.num_groups * shape.state_dim)


def _ssm_dt(dt: torch.Tensor, rows: int, H: int, dev: int):
    p, st = _row_stride(dt, rows, H, dev, "dt")
    return _IO[dt.dtype], p, st


def gdn_ssm_prefill_workspace(shape: gdn_ssm_shape, cu_seqlens_host) -> int:
    """Bytes of workspace of gdn_ssm_prefill_packed for a pack."""
    cu_h = _host_i32(cu_seqlens_host)
    n = ctypes.c_int64(0)
    _check(load().gdn_ssm_prefill_workspace(ctypes.addressof(shape), cu_h.ctypes.data, len(cu_h) - 1, int(cu_h[-1]),
                                            ctypes.byref(n)), "gdn_ssm_prefill_workspace")
    return n.value


def gdn_ssm_prefill_packed(shape: gdn_ssm_shape, cu_seqlens, cu_seqlens_host, x, dt, A, out, dt_bias=None, D=None,
                           init_state=None, final_state=None, ckpt_positions=None, ckpt_positions_host=None,
                           ckpt_buf=None, conv_weight=None, conv_bias=None, conv_state_in=None, conv_state_out=None,
                           conv_ckpt=None, workspace=None, stream=None) -> None:
    """The packed scan of a state space layer: x [T, conv_dim] bf16 (columns
    [x | B | C], before the short convolution where conv_weight is given), dt
    [T, H] raw steps in bf16 or fp32, both columns of a wider row if need be;
    out [T, H, P] bf16.  workspace: a uint8 tensor of
    gdn_ssm_prefill_workspace() bytes."""
    dev, st = _where(stream)
    f32, bf16 = torch.float32, torch.bfloat16
    cu_h, ck_h = _host_i32(cu_seqlens_host), _host_i32(ckpt_positions_host)
    n, T, k = len(cu_h) - 1, int(cu_h[-1]), 0 if ck_h is None else len(ck_h)
    H, P, N, C = _ssm_dims(shape)
    xp, xs = _row_stride(x, T, C, dev, "x", bf16)
    dtt, dtp, dts = _ssm_dt(dt, T, H, dev)
    if tuple(out.shape[1:]) != (H, P) or out.shape[0] < T:
        raise ValueError("out must be [T, H, P]")
    if cu_seqlens.numel() < n + 1 or (k and ckpt_positions is not None and ckpt_positions.numel() < k):
        raise ValueError("cu_seqlens or ckpt_positions is shorter than its host mirror")
    _check(load().gdn_ssm_prefill_packed(
        ctypes.addressof(shape), _buf(cu_seqlens, torch.int32, dev, "cu_seqlens"), cu_h.ctypes.data, n, T, xp, xs,
        _sized(conv_weight, f32, dev, (C, 4), "conv_weight"), _sized(conv_bias, f32, dev, (C,), "conv_bias"),
        _sized(conv_state_in, bf16, dev, (n, 3, C), "conv_state_in"),
        _sized(conv_state_out, bf16, dev, (n, 3, C), "conv_state_out"), dtt, dtp, dts,
        _sized(A, f32, dev, (H,), "A"), _sized(dt_bias, f32, dev, (H,), "dt_bias"), _sized(D, f32, dev, (H,), "D"),
        _sized(init_state, f32, dev, (n, H, P, N), "init_state"),
        _buf(ckpt_positions, torch.int32, dev, "ckpt_positions"), _hp(ck_h), k,
        _sized(conv_ckpt, bf16, dev, (k, 3, C), "conv_ckpt"), _buf(out, bf16, dev, "out"),
        _sized(final_state, f32, dev, (n, H, P, N), "final_state"),
        _sized(ckpt_buf, f32, dev, (k, H, P, N), "ckpt_buf"), _buf(workspace, torch.uint8, dev, "workspace"),
        0 if workspace is None else workspace.numel(), st), "gdn_ssm_prefill_packed")


def gdn_ssm_decode(shape: gdn_ssm_shape, n_tok: int, x, dt, A, state, out, dt_bias=None, D=None, conv_weight=None,
                   conv_bias=None, conv_state=None, slot=None, slot_host=None, snapshots=None, stream=None) -> None:
    """n_tok tokens per sequence (rows b * n_tok + i of x [batch * n_tok,
    conv_dim] and dt [batch * n_tok, H]) in place on the pools state
    [slots, H, P, N] and conv_state [slots, 3, conv_dim]."""
    dev, st = _where(stream)
    f32, bf16 = torch.float32, torch.bfloat16
    H, P, N, C = _ssm_dims(shape)
    rows, n_tok = x.shape[0], int(n_tok)
    if n_tok < 1 or rows % n_tok != 0:
        raise ValueError("x must have n_tok rows per sequence")
    B, pool = rows // n_tok, state.shape[0]
    sl_h = _host_i32(slot_host)
    if slot is not None and (slot.numel() < B or (sl_h is not None and len(sl_h) < B)):
        raise ValueError("slot is shorter than the batch")
    xp, xs = _row_stride(x, rows, C, dev, "x", bf16, exact=True)
    dtt, dtp, dts = _ssm_dt(dt, rows, H, dev)
    _check(load().gdn_ssm_decode(
        ctypes.addressof(shape), B, n_tok, xp, xs, _sized(conv_weight, f32, dev, (C, 4), "conv_weight"),
        _sized(conv_bias, f32, dev, (C,), "conv_bias"), _sized(conv_state, bf16, dev, (pool, 3, C), "conv_state"),
        dtt, dtp, dts, _sized(A, f32, dev, (H,), "A"), _sized(dt_bias, f32, dev, (H,), "dt_bias"),
        _sized(D, f32, dev, (H,), "D"), _sized(state, f32, dev, (pool, H, P, N), "state"), pool,
        _buf(slot, torch.int32, dev, "slot"), _hp(sl_h), _sized(out, bf16, dev, (rows, H, P), "out"),
        _sized(snapshots, f32, dev, (B, n_tok, H, P, N), "snapshots"), st), "gdn_ssm_decode")


def gdn_rms_norm(shape: gdn_norm_shape, x, weight=None, out=None, residual=None, residual_out=None, gate=None,
                 codes=None, scales=None, stream=None) -> None:
    """Root-mean-square norm of x [rows, dim] (bf16 or fp32), after the addition
    of a residual (its sum to residual_out), gated by silu(gate); to out (x's
    type) and / or to codes (float8_e4m3fn or int8) with fp32 scales [rows, 1]
    or [rows, dim / scale_block]."""
    dev, st = _where(stream)
    rows, d = x.shape[0], shape.dim
    xp, xs = _row_stride(x, rows, d, dev, "x", exact=True)
    rp = rs = zp = zs = rop = ros = None
    rt = ct = 0
    if residual is not None:
        rp, rs = _row_stride(residual, rows, d, dev, "residual", exact=True)
        rt = _IO[residual.dtype]
    if residual_out is not None:
        if residual is None:
            raise ValueError("residual_out needs a residual")
        rop, ros = _row_stride(residual_out, rows, d, dev, "residual_out", residual.dtype, exact=True)
        if ros != rs:
            raise ValueError("residual_out must have residual's row stride")
    if gate is not None:
        zp, zs = _row_stride(gate, rows, d, dev, "gate", x.dtype, exact=True)
    if codes is not None:
        if codes.dtype not in _CODES:
            raise TypeError("codes must be float8_e4m3fn or int8")
        ct = _CODES[codes.dtype]
    n_sc = d // shape.scale_block if shape.scale_block > 0 else 1
    _check(load().gdn_rms_norm(
        ctypes.addressof(shape), rows, _IO[x.dtype], xp, xs, rt, rp, rs or 0, rop, zp, zs or 0,
        _sized(weight, torch.float32, dev, (shape.weight_dim,), "weight"), _sized(out, x.dtype, dev, (rows, d), "out"),
        ct, None if codes is None else _sized(codes, codes.dtype, dev, (rows, d), "codes"),
        _sized(scales, torch.float32, dev, (rows, n_sc), "scales"), st), "gdn_rms_norm")

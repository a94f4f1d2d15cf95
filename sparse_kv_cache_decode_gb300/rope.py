"""Binding of the kvs_rope entry points: norms of queries and keys for each head and their rotation by position.

`Rope` wraps a kvs_rope (what turns, by which frequency, along which axis).  It holds no device memory: one serves all layers,
devices and streams.  Tensors:

  q, k         [n_tok][H][head_dim] bf16, any strides that keep a head's elements together (slices of a fused projection or of longer rows)
  pos          [n_axis][n_tok] int32, or [n_tok] for all axes
  q_norm ...   [head_dim] fp32
"""
from __future__ import annotations

import ctypes

import torch

from . import KvsError, KvsRopeConfig, _check, calls
from . import fast as _fast

_BF16 = (torch.bfloat16, torch.int16)
_I32, _F32 = (torch.int32,), (torch.float32,)


def rope_axes(sections, cycle: bool = False) -> list:
    """The axis of each pair: `sections` pairs of axis 0, then of axis 1, ...; with `cycle` the axes take turns for as long as they have pairs left."""
    if not cycle:
        return [a for a, n in enumerate(sections) for _ in range(n)]
    left, out = list(sections), []
    while any(left):
        for a, n in enumerate(left):
            if n:
                out.append(a)
                left[a] -= 1
    return out


def make_rope_config(head_dim: int, rot_dim: int | None = None, theta: float = 10000.0, adjacent: bool = False, axes=None, inv_freq=None,
                     rot_scale: float = 1.0, norm_eps: float = 1e-6) -> KvsRopeConfig:
    """axes: the axis of each of the rot_dim / 2 pairs (see rope_axes), or None for one axis; inv_freq: radians per position of each
    pair, or None for theta^(-2 i / rot_dim)."""
    rot_dim = head_dim if rot_dim is None else rot_dim
    for x, name in ((head_dim, "head_dim"), (rot_dim, "rot_dim")):
        if not 0 <= x < 1 << 31:
            raise ValueError(f"{name}: {x}")
    cfg = KvsRopeConfig(head_dim, rot_dim, int(bool(adjacent)), 1, None, None, float(theta), float(rot_scale), float(norm_eps))
    if axes is not None:
        axes = [int(a) for a in axes]
        if len(axes) != rot_dim // 2 or any(not 0 <= a < 256 for a in axes):
            raise ValueError(f"axes: {len(axes)} of them, expected one for each of {rot_dim // 2} pairs")
        cfg.n_axis = max(axes, default=0) + 1
        cfg.axis = ctypes.cast((ctypes.c_ubyte * max(1, len(axes)))(*axes), ctypes.POINTER(ctypes.c_ubyte))
    if inv_freq is not None:
        inv_freq = [float(f) for f in inv_freq]
        if len(inv_freq) != rot_dim // 2:
            raise ValueError(f"inv_freq: {len(inv_freq)} of them, expected one for each of {rot_dim // 2} pairs")
        cfg.inv_freq = ctypes.cast((ctypes.c_double * max(1, len(inv_freq)))(*inv_freq), ctypes.POINTER(ctypes.c_double))
    return cfg


def _rows(t, name, d, index):
    """Rows [n_tok][heads][d] of bf16: (pointer, token stride, head stride, tokens, heads)."""
    x = _fast.rows(t, _BF16, -1, d, index)
    if x is not None:
        return x
    if t.dtype not in _BF16:
        raise ValueError(f"{name}: dtype {t.dtype}, expected {_BF16[0]}")
    if t.dim() != 3 or t.shape[2] != d:
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected (n_tok, heads, {d})")
    if t.stride(2) != 1:
        raise ValueError(f"{name}: a head's elements must be contiguous")
    raise ValueError(f"{name}: on {t.device}")


def _norm(t, name, d, index):
    if t is None:
        return None
    p = _fast.whole(t, _F32, (d,), index)
    if p is None:
        raise ValueError(f"{name}: {t.dtype} {tuple(t.shape)} on {t.device}, expected contiguous torch.float32 ({d},)")
    return p


def _positions(t, n_axis, n, index):
    """(pointer, elements between axes) of positions [n_axis][n] or [n]."""
    p = _fast.whole(t, _I32, (n,), index)
    if p is not None:
        return p, 0
    p = _fast.whole(t, _I32, (n_axis, n), index)
    if p is not None:
        return p, n if n_axis > 1 else 0
    if t.dtype != torch.int32:
        raise ValueError(f"pos: dtype {t.dtype}, expected torch.int32")
    shape, stride = t.shape, t.stride()
    if shape[-1:] != (n,) or len(shape) > 2 or (len(shape) == 2 and shape[0] != n_axis):
        raise ValueError(f"pos: shape {tuple(shape)}, expected ({n_axis}, {n}) or ({n},)")
    if n > 1 and stride[-1] != 1:
        raise ValueError("pos: an axis' positions must be contiguous")
    if t.get_device() != index:
        raise ValueError(f"pos: on {t.device}")
    return t.data_ptr(), stride[0] if len(shape) == 2 and n_axis > 1 else 0


class Rope:
    def __init__(self, cfg: KvsRopeConfig):
        self.h = None
        self.cfg = cfg
        self.d, self.n_axis = cfg.head_dim, cfg.n_axis
        self.L = calls
        h = ctypes.c_void_p()
        _check(self.L.kvs_rope_create(ctypes.byref(cfg), ctypes.byref(h)), "kvs_rope_create")
        self.h, self.address = h, h.value

    def close(self):
        if getattr(self, "h", None):
            self.L.kvs_rope_destroy(self.h)
            self.h = self.address = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def rotate(self, q, pos, q_out, k=None, k_out=None, q_norm=None, k_norm=None, stream=None):
        """kvs_rotate: q [n_tok][H_q][d] into q_out and, if given, k [n_tok][H_k][d] into k_out (in place: the same tensor)."""
        if self.h is None:
            raise ValueError("Rope: closed")
        status = _fast.rotate(self.address, self.d, self.n_axis, q, pos, q_out, k, k_out, q_norm, k_norm, stream)
        if status == 0:
            return
        if status is not None:
            raise KvsError(status, "kvs_rotate")
        d, index = self.d, q.get_device()
        if index < 0:
            raise ValueError("q: must be a CUDA tensor")
        qp, qs, qh, n, hq = _rows(q, "q", d, index)
        op, os, oh, n_o, h_o = _rows(q_out, "q_out", d, index)
        if n_o != n or h_o != hq:
            raise ValueError("q_out: another shape than q")
        kp = ks = kh = hk = kop = kos = koh = 0
        if (k is None) != (k_out is None):
            raise ValueError("k and k_out: one without the other")
        if k is not None:
            kp, ks, kh, n_k, hk = _rows(k, "k", d, index)
            kop, kos, koh, n_o, h_o = _rows(k_out, "k_out", d, index)
            if n_k != n or n_o != n or h_o != hk:
                raise ValueError("k and k_out: another number of tokens than q, or shapes that differ")
        pp, ps = _positions(pos, self.n_axis, n, index)
        qn, kn = _norm(q_norm, "q_norm", d, index), _norm(k_norm, "k_norm", d, index)
        if stream is None:
            stream = _fast.stream(index)
        elif not isinstance(stream, int):
            stream = stream.cuda_stream
        args = (self.h, qp, qs, qh, hq, qn, op, os, oh, kp, ks, kh, hk, kn, kop, kos, koh, pp, ps, n, stream)
        if _fast.device() == index:
            status = self.L.kvs_rotate(*args)
        else:
            with torch.cuda.device(index):
                status = self.L.kvs_rotate(*args)
        if status != 0:
            raise KvsError(status, "kvs_rotate")

"""Binding of the kvs_pool entry points: paged KV caches that stay whole in device memory.

`Pool` wraps a kvs_pool over the caller's K and V tensors, with a workspace from torch.  Its methods check
what the tensors are (ValueError) and forward to the C ABI (KvsError).  Tensors:

  k, v         [n_layer][n_slots][H_kv][block_size][d]; bf16 pools torch.bfloat16 (or int16 patterns), E4M3 pools
               torch.float8_e4m3fn (or uint8 codes)
  q            [n_tok][H_q][d] bf16, contiguous within a token (a slice of a fused projection will do)
  cu_q         [n_req + 1] int32;  ctx_len [n_req] int32;  block2slot [n_req][nb_max] int32
  out          [n_tok][H_q][d] bf16;  lse [n_tok][H_q] fp32;  weight [n_req][H_kv][max_ctx] fp32
  place        [n_tok] int64;  pos [n_axis][n_tok] or [n_tok] int32;  norms [d] fp32

`BlockTables` keeps the block table of a batch over a pool and the ring of its free slots.
"""
from __future__ import annotations

import ctypes
import functools

import torch

from . import KV_DTYPE, KvsError, KvsPoolConfig, _check, calls
from . import fast as _fast
from .rope import Rope, _norm, _positions

_BF16 = (torch.bfloat16, torch.int16)
_FP8 = (torch.float8_e4m3fn, torch.uint8)
_I32, _I64, _F32 = (torch.int32,), (torch.int64,), (torch.float32,)


def _int(x: int, name: str) -> int:
    """x, if the ABI's 32 bits hold it (ctypes would cut it to its low bits)."""
    if -0x80000000 <= x < 0x80000000:
        return x
    raise ValueError(f"{name}: {x} does not fit 32 bits")


def make_pool_config(n_layer: int, n_slots: int, n_q_head: int, n_kv_head: int, head_dim: int, block_size: int,
                     max_ctx: int, max_req: int, max_tokens: int, max_prefix_tokens: int = 0, kv_dtype: str = "bf16",
                     k_scale: float = 1.0, v_scale: float = 1.0, softmax_scale: float = 0.0,
                     wait_timeout_us: int = 0) -> KvsPoolConfig:
    ints = dict(n_layer=n_layer, n_slots=n_slots, n_q_head=n_q_head, n_kv_head=n_kv_head, head_dim=head_dim, block_size=block_size,
                max_ctx=max_ctx, max_req=max_req, max_tokens=max_tokens, max_prefix_tokens=max_prefix_tokens)
    if not 0 <= wait_timeout_us < 1 << 32:
        raise ValueError(f"wait_timeout_us: {wait_timeout_us} does not fit 32 bits")
    return KvsPoolConfig(*(_int(x, name) for name, x in ints.items()), KV_DTYPE[kv_dtype], float(k_scale), float(v_scale),
                         float(softmax_scale), wait_timeout_us)


class Pool:
    """A kvs_pool over K and V tensors of the caller, with its device workspace (allocated through torch): keep it, and every
    tensor of a call, until the calls on them are through."""
    h = _address = None       # the handle (None: closed), and its address

    def __init__(self, cfg: KvsPoolConfig, k: torch.Tensor, v: torch.Tensor):
        self.cfg = cfg
        self.L = calls
        nbytes = self.L.kvs_pool_workspace_bytes(ctypes.byref(cfg))
        if nbytes == 0:
            raise KvsError(1, "kvs_pool_workspace_bytes")
        self.nb_max = (cfg.max_ctx + cfg.block_size - 1) // cfg.block_size
        self.device = k.device
        self.index = k.get_device()          # -1 on the CPU
        shape = (cfg.n_layer, cfg.n_slots, cfg.n_kv_head, cfg.block_size, cfg.head_dim)
        kinds = _FP8 if cfg.kv_dtype == KV_DTYPE["fp8"] else _BF16
        self._whole(k, "k", kinds, shape)
        self._whole(v, "v", kinds, shape)
        if k.device.type != "cuda":
            raise ValueError("Pool: k and v must be CUDA tensors")
        self.k, self.v = k, v
        with torch.cuda.device(self.device):
            self.workspace = torch.empty(nbytes + 256, dtype=torch.uint8, device=self.device)
            aligned = (self.workspace.data_ptr() + 255) // 256 * 256
            h = ctypes.c_void_p()
            _check(self.L.kvs_pool_create(ctypes.byref(cfg), k.data_ptr(), v.data_ptr(), aligned, nbytes,
                                          ctypes.byref(h)), "kvs_pool_create")
        self.h, self._address = h, h.value

    def close(self):
        if self.h is not None:
            self.L.kvs_pool_destroy(self.h)
            self.h = self._address = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    # ------------------------------------------------------------------ checks (every call: kept short)
    def _whole(self, t, name, dtypes, shape):
        """Pointer of a contiguous tensor of this device."""
        p = _fast.whole(t, dtypes, shape, self.index)
        if p is not None:
            return p
        if t.dtype not in dtypes:
            raise ValueError(f"{name}: dtype {t.dtype}, expected {dtypes[0]}")
        if t.shape != shape:
            raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
        if not t.is_contiguous():
            raise ValueError(f"{name}: not contiguous")
        raise ValueError(f"{name}: on {t.device}, the pool is on {self.device}")

    def _tokens(self, t, name, heads):
        """Rows [n_tok][heads][d] of bf16, contiguous within a token: (pointer, token stride, tokens)."""
        d = self.cfg.head_dim
        x = _fast.rows(t, _BF16, heads, d, self.index)
        if x is not None and (x[2] == d or heads == 1) and x[1] >= heads * d:
            return x[0], x[1], x[3]
        if t.dtype not in _BF16:
            raise ValueError(f"{name}: dtype {t.dtype}, expected {_BF16[0]}")
        if t.dim() != 3 or t.shape[1] != heads or t.shape[2] != d:
            raise ValueError(f"{name}: shape {tuple(t.shape)}, expected (n_tok, {heads}, {d})")
        n = t.shape[0]
        s0, s1, s2 = t.stride()
        if s2 != 1 or (heads > 1 and s1 != d):
            raise ValueError(f"{name}: a token's rows must be contiguous")
        if t.get_device() != self.index:
            raise ValueError(f"{name}: on {t.device}, the pool is on {self.device}")
        if n <= 1:
            s0 = heads * d
        elif s0 < heads * d:
            raise ValueError(f"{name}: tokens overlap")
        return t.data_ptr(), s0, n

    def _batch(self, ctx_len, block2slot, cu_q=None):
        n_req = ctx_len.shape[0]
        ctx = self._whole(ctx_len, "ctx_len", _I32, (n_req,))
        tab = self._whole(block2slot, "block2slot", _I32, (n_req, self.nb_max))
        return (n_req, ctx, tab) if cu_q is None else (n_req, self._whole(cu_q, "cu_q", _I32, (n_req + 1,)), ctx, tab)

    def _stream(self, stream):
        if stream is None:
            return _fast.stream(self.index)
        return stream if isinstance(stream, int) else stream.cuda_stream

    def _call(self, fn, where, *args):
        if self.h is None:
            raise ValueError("Pool: closed")
        if _fast.device() == self.index:
            status = fn(self.h, *args)
        else:
            with torch.cuda.device(self.index):
                status = fn(self.h, *args)
        if status != 0:
            raise KvsError(status, where)

    # ------------------------------------------------------------------ C-ABI forwards
    def append(self, layer, k_new, v_new, cu_q, ctx_len, block2slot, stream=None):
        """kvs_pool_append: the call's new tokens, k_new and v_new [n_tok][H_kv][d] bf16, into the pool."""
        kp, ks, n_tok = self._tokens(k_new, "k_new", self.cfg.n_kv_head)
        vp, vs, n_v = self._tokens(v_new, "v_new", self.cfg.n_kv_head)
        if n_v != n_tok or ks != vs:
            raise ValueError("k_new and v_new: different numbers or strides of tokens")
        n_req, cu, ctx, tab = self._batch(ctx_len, block2slot, cu_q)
        self._call(self.L.kvs_pool_append, "kvs_pool_append", _int(layer, "layer"), kp, vp, ks, cu, ctx, tab, n_req, n_tok, self._stream(stream))

    def attn(self, layer, q, cu_q, ctx_len, block2slot, out, window=0, n_sink=0, lse=None, weight=None, stream=None):
        """kvs_pool_attn: causal attention (window, n_sink: a sliding window and first tokens that stay visible);
        weight accumulates each key's softmax weight."""
        c = self.cfg
        # no key is further away than the longest context
        window, n_sink = _int(min(window, c.max_ctx), "window"), _int(min(n_sink, c.max_ctx), "n_sink")
        qp, qs, n_tok = self._tokens(q, "q", c.n_q_head)
        n_req, cu, ctx, tab = self._batch(ctx_len, block2slot, cu_q)
        o = self._whole(out, "out", _BF16, (n_tok, c.n_q_head, c.head_dim))
        ls = None if lse is None else self._whole(lse, "lse", _F32, (n_tok, c.n_q_head))
        w = None if weight is None else self._whole(weight, "weight", _F32, (n_req, c.n_kv_head, c.max_ctx))
        self._call(self.L.kvs_pool_attn, "kvs_pool_attn", _int(layer, "layer"), qp, qs, cu, ctx, tab, n_req, n_tok, window, n_sink, o, ls, w,
                   self._stream(stream))

    def prefix_attn(self, layer, q, cu_q, ctx_len, block2slot, prefix_req, prefix_len, prefix2slot, out, lse=None,
                    stream=None):
        """kvs_pool_prefix_attn: requests [prefix_req[i], prefix_req[i + 1]) see prefix i, then their own tokens."""
        c = self.cfg
        qp, qs, n_tok = self._tokens(q, "q", c.n_q_head)
        n_req, cu, ctx, tab = self._batch(ctx_len, block2slot, cu_q)
        n_pre = prefix_len.shape[0]
        pr = self._whole(prefix_req, "prefix_req", _I32, (n_pre + 1,))
        pl = self._whole(prefix_len, "prefix_len", _I32, (n_pre,))
        pt = self._whole(prefix2slot, "prefix2slot", _I32, (n_pre, self.nb_max))
        o = self._whole(out, "out", _BF16, (n_tok, c.n_q_head, c.head_dim))
        ls = None if lse is None else self._whole(lse, "lse", _F32, (n_tok, c.n_q_head))
        self._call(self.L.kvs_pool_prefix_attn, "kvs_pool_prefix_attn", _int(layer, "layer"), qp, qs, cu, ctx, tab, n_req, n_tok, pr, pl, pt,
                   n_pre, o, ls, self._stream(stream))

    def evict(self, layer, weight, ctx_len, block2slot, keep, n_sink, n_recent, dst2slot, kept, n_kept, weight_out,
              stream=None):
        """kvs_pool_evict: the tokens each kv head keeps, gathered into the blocks of dst2slot."""
        c = self.cfg
        n_req, ctx, tab = self._batch(ctx_len, block2slot)
        w = self._whole(weight, "weight", _F32, (n_req, c.n_kv_head, c.max_ctx))
        dst = self._whole(dst2slot, "dst2slot", _I32, (n_req, self.nb_max))
        kp = self._whole(kept, "kept", _I32, (n_req, c.n_kv_head, keep))
        nk = self._whole(n_kept, "n_kept", _I32, (n_req,))
        wo = self._whole(weight_out, "weight_out", _F32, (n_req, c.n_kv_head, c.max_ctx))
        self._call(self.L.kvs_pool_evict, "kvs_pool_evict", _int(layer, "layer"), w, ctx, tab, n_req, keep, _int(n_sink, "n_sink"),
                   _int(n_recent, "n_recent"), dst, kp, nk, wo, self._stream(stream))

    def places(self, cu_q, ctx_len, block2slot, place, pos=None, pos_delta=None, stream=None):
        """kvs_pool_places: where the call's tokens go (place [n_tok]) and their positions, from tables kept by the caller."""
        n_req, cu, ctx, tab = self._batch(ctx_len, block2slot, cu_q)
        n_tok, pl, po, de = self._tokens_out(n_req, place, pos, pos_delta)
        self._call(self.L.kvs_pool_places, "kvs_pool_places", cu, ctx, tab, n_req, n_tok, de, pl, po, self._stream(stream))

    def _tokens_out(self, n_req, place, pos, pos_delta):
        n_tok = place.shape[0]
        pl = self._whole(place, "place", _I64, (n_tok,))
        po = None if pos is None else self._whole(pos, "pos", _I32, (n_tok,))
        return n_tok, pl, po, None if pos_delta is None else self._whole(pos_delta, "pos_delta", _I32, (n_req,))

    def _rope(self, rope):
        if not isinstance(rope, Rope) or rope.h is None:
            raise ValueError("rope: not an open Rope")
        return rope.h

    def rotate_append(self, layer, rope, q, k, v, pos, place, q_out, q_norm=None, k_norm=None, stream=None):
        """kvs_pool_rotate_append: q [n_tok][H_q][d] normed and rotated into q_out; k and v [n_tok][H_kv][d] to their places, k normed and
        rotated as well."""
        hq, hk, d = self._heads
        if self.h is not None and type(rope) is Rope and rope.h is not None:
            status = _fast.rotate_append(self._address, rope.address, self.index, hq, hk, d, rope.n_axis, layer, q, k, v, pos, place, q_out, q_norm, k_norm, stream)
            if status == 0:
                return
            if status is not None:
                raise KvsError(status, "kvs_pool_rotate_append")
        # another device than the current one, or something to complain of
        i, rows = self.index, _fast.rows
        a, b, c, o = rows(q, _BF16, hq, d, i), rows(k, _BF16, hk, d, i), rows(v, _BF16, hk, d, i), rows(q_out, _BF16, hq, d, i)
        if a is None or b is None or c is None or o is None or a[2] != d or b[2] != d or c[2] != d or o[2] != d:
            for t, name, heads in ((q, "q", hq), (k, "k", hk), (v, "v", hk), (q_out, "q_out", hq)):
                self._tokens(t, name, heads)
        n_tok = a[3]
        if b[3] != n_tok or c[3] != n_tok or o[3] != n_tok or b[1] != c[1]:
            raise ValueError("q, k, v and q_out: different numbers of tokens, or k and v of different strides")
        h = self._rope(rope)
        pp, ps = _positions(pos, rope.n_axis, n_tok, i)
        pl = self._whole(place, "place", _I64, (n_tok,))
        qn, kn = _norm(q_norm, "q_norm", d, i), _norm(k_norm, "k_norm", d, i)
        self._call(self.L.kvs_pool_rotate_append, "kvs_pool_rotate_append", h, _int(layer, "layer"), a[0], a[1], b[0], c[0], b[1], qn, kn, pp, ps, pl,
                   n_tok, o[0], o[1], _fast.stream(i) if stream is None else self._stream(stream))

    @functools.cached_property
    def _heads(self):
        """(H_q, H_kv, head_dim)"""
        return self.cfg.n_q_head, self.cfg.n_kv_head, self.cfg.head_dim

    def reposition(self, layer, rope, kept, n_kept, block2slot, stream=None):
        """kvs_pool_reposition: the keys that `evict` kept (its kept, n_kept and dst2slot), rotated to their new positions."""
        n_req, nk, tab = self._batch(n_kept, block2slot)
        kp = self._whole(kept, "kept", _I32, (n_req, self.cfg.n_kv_head, kept.shape[-1]))
        self._call(self.L.kvs_pool_reposition, "kvs_pool_reposition", self._rope(rope), _int(layer, "layer"), kp, nk, tab, n_req, kept.shape[-1],
                   self._stream(stream))

    def launch_count(self) -> int:
        return int(self.L.kvs_pool_launch_count(self.h))

    def poll_error(self) -> int:
        st = ctypes.c_int()
        with torch.cuda.device(self.device):
            _check(self.L.kvs_pool_poll_error(self.h, ctypes.byref(st)), "kvs_pool_poll_error")
        return st.value


class BlockTables:
    """The block table of a batch over a pool and the ring of the pool's free slots, kept in the caller's tensors:

      block2slot [n_req][nb_max] int32;  n_held [n_req] int32, the blocks each row owns;  ring [n_slots] int32;  ring_state [3] int32

    Several may share a ring (a batch, its shared prefixes, the blocks that an eviction gathers into)."""

    def __init__(self, pool: Pool, block2slot, n_held, ring, ring_state):
        self.pool, self.n_req = pool, block2slot.shape[0]
        self._ptrs = (pool._whole(n_held, "n_held", _I32, (self.n_req,)),
                      pool._whole(block2slot, "block2slot", _I32, (self.n_req, pool.nb_max)),
                      pool._whole(ring, "ring", _I32, (pool.cfg.n_slots,)), pool._whole(ring_state, "ring_state", _I32, (3,)))
        self.block2slot, self.n_held, self.ring, self.ring_state = block2slot, n_held, ring, ring_state

    @classmethod
    def empty(cls, pool: Pool, n_req: int, like: BlockTables | None = None):
        """Rows without blocks over a pool whose slots are all free, or over the ring of `like`."""
        i32 = dict(dtype=torch.int32, device=pool.device)
        n = pool.cfg.n_slots
        ring, state = (like.ring, like.ring_state) if like is not None else (torch.arange(n, **i32), torch.tensor([0, n, 0], **i32))
        return cls(pool, torch.full((n_req, pool.nb_max), -1, **i32), torch.zeros(n_req, **i32), ring, state)

    def reserve(self, ctx_len, cu_q=None, place=None, pos=None, pos_delta=None, stream=None):
        """kvs_pool_reserve: every row gets the blocks of its new length, or gives back those past it; with cu_q and place also where the
        call's tokens go, and their positions."""
        p, n_req = self.pool, self.n_req
        if p.h is not None:
            status = _fast.reserve(p._address, p.index, n_req, *self._ptrs, ctx_len, cu_q, place, pos, pos_delta, stream)
            if status == 0:
                return
            if status is not None:
                raise KvsError(status, "kvs_pool_reserve")
        # another device than the current one, or something to complain of
        ctx = p._whole(ctx_len, "ctx_len", _I32, (n_req,))
        cu = pl = po = de = None
        n_tok = 0
        if cu_q is not None and place is not None:
            cu = p._whole(cu_q, "cu_q", _I32, (n_req + 1,))
            n_tok, pl, po, de = p._tokens_out(n_req, place, pos, pos_delta)
        elif cu_q is not None or place is not None or pos is not None or pos_delta is not None:
            raise ValueError("cu_q and place: one without the other")
        held, tab, ring, state = self._ptrs
        p._call(p.L.kvs_pool_reserve, "kvs_pool_reserve", ctx, held, tab, ring, state, n_req, cu, de, n_tok, pl, po, p._stream(stream))

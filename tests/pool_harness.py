"""A paged pool filled with seeded rows for the pool tests.  Slots are handed out in random order, table
entries no request uses are -1, and every row of the pool that holds no token is NaN, so that a kernel that
uses one shows it."""
from __future__ import annotations

import numpy as np
import torch

import sparse_kv_cache_decode_gb300 as K

NAN = {"bf16": 0x7FC0, "fp8": 0x7F}


class PoolCase:
    def __init__(self, seed, ctx, q_len, hq, hk, d, bs, kv="bf16", prefixes=(), n_layer=1, layer=0, spare=0, max_ctx=None,
                 heavy=0.02, pad_tokens=0, k_scale=0.06, v_scale=0.04, key_shift=None, q_shift=0.0):
        r = np.random.default_rng(seed)
        self.rng = r
        self.ctx, self.q_len, self.hq, self.hk, self.d, self.bs, self.kv, self.layer = ctx, q_len, hq, hk, d, bs, kv, layer
        self.scales = (k_scale, v_scale) if kv == "fp8" else (1.0, 1.0)
        self.max_ctx = max_ctx or max([1] + list(ctx) + list(prefixes))
        self.nb = -(-self.max_ctx // bs)
        blocks = [-(-n // bs) for n in list(ctx) + list(prefixes)]
        self.n_used = sum(blocks)
        self.n_slots = self.n_used + spare + 2
        order = r.permutation(self.n_used + 2)      # two slots stay unused
        shape = (n_layer, self.n_slots, hk, bs, d)
        self.k = self._nan(shape)
        self.v = self._nan(shape)
        self.rows = []                              # per sequence: (k, v) [n][hk][d] fp64, as the pool holds them
        tables = np.full((len(blocks), self.nb), -1, np.int32)
        at = 0
        for s, n in enumerate(list(ctx) + list(prefixes)):
            tables[s, :blocks[s]] = order[at:at + blocks[s]]
            at += blocks[s]
            kv_rows = []
            for x, pool, scale in ((0, self.k, self.scales[0]), (1, self.v, self.scales[1])):
                a = r.standard_normal((n, hk, d)).astype(np.float32)
                if x == 0:
                    a *= np.where(r.random((n, hk, 1)) < heavy, 4, 1).astype(np.float32)
                    if key_shift is not None:       # added to every dim of a key, by position
                        a += key_shift(np.arange(n))[:, None, None].astype(np.float32)
                codes, val = self.encode(a, scale)
                for b in range(blocks[s]):
                    part = codes[b * bs:(b + 1) * bs]
                    pool[layer, tables[s, b], :, :len(part)] = part.transpose(0, 1)
                kv_rows.append(val)
            self.rows.append(tuple(kv_rows))
        self.table, self.prefix_table = tables[:len(ctx)], tables[len(ctx):]
        self.cu = np.concatenate([[0], np.cumsum(q_len)]).astype(np.int32)
        self.n_tok = int(self.cu[-1]) + pad_tokens
        self.q = torch.from_numpy(r.standard_normal((self.n_tok, hq, d)).astype(np.float32) + np.float32(q_shift)).to(torch.bfloat16)
        self.cfg = dict(n_layer=n_layer, n_slots=self.n_slots, n_q_head=hq, n_kv_head=hk, head_dim=d, block_size=bs, max_ctx=self.max_ctx,
                        max_req=max(1, len(ctx)), max_tokens=max(1, self.n_tok), max_prefix_tokens=max(1, self.n_tok) if prefixes else 0,
                        kv_dtype=kv, k_scale=self.scales[0], v_scale=self.scales[1])
        self.softmax_scale = float(np.float32(1 / np.sqrt(d)))

    def _nan(self, shape):
        if self.kv == "bf16":
            return torch.full(shape, float("nan"), dtype=torch.bfloat16)
        return torch.full(shape, NAN["fp8"], dtype=torch.uint8)

    def encode(self, a, scale):
        """(what the pool holds, the fp64 values it stands for) of fp32 values."""
        t = torch.from_numpy(np.ascontiguousarray(a))
        if self.kv == "bf16":
            t = t.to(torch.bfloat16)
            return t, t.double().numpy()
        t = (t / scale).clamp(-448, 448).to(torch.float8_e4m3fn)
        return t.view(torch.uint8), t.double().numpy() * np.float32(scale)

    def cuda(self, **over):
        dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
        self.dk, self.dv = self.k.cuda(), self.v.cuda()
        self.pool = K.Pool(K.make_pool_config(**(self.cfg | over)), self.dk, self.dv)
        self.d_q, self.d_cu = self.q.cuda(), dev(self.cu)
        self.d_ctx, self.d_table = dev(np.array(self.ctx, np.int32)), dev(self.table)
        return self

    def out(self, fill=7.0):
        return (torch.full((self.n_tok, self.hq, self.d), fill, dtype=torch.bfloat16, device="cuda"),
                torch.full((self.n_tok, self.hq), fill, device="cuda"))

    def query(self, r):
        return self.q[self.cu[r]:self.cu[r + 1]].double().numpy()


def check_out(got, lse, ref, ref_lse, mag, d, where="", S=40):
    """Outputs and log-sum-exps of one request against the oracle's.

    A weight p is computed with a relative error of at most 2^-8 (its rounding to bf16) plus e (its logit's
    error, below), so an output is off by at most (2^-8 + 2 e) mag, and its own rounding adds 2^-8 |ref|.
    A logit of |s| <= S (S = 40 covers most inputs, asserted) in fp32: d products of 24 + 8 bits summed
    in fp32 (each sum truncated at worst: 2^-23 a step relative to the largest partial sum, taken as 2 S),
    2^-23 (d + 4) * 2 S < 1.3e-3 at d = 128, in practice far less; the log-sum-exp carries the same."""
    e = 2.0 ** -23 * (d + 4) * 2 * S
    assert np.isneginf(ref_lse).all() or np.abs(ref_lse[~np.isneginf(ref_lse)]).max() < S
    tol = 2.0 ** -8 * np.abs(ref) + (2.0 ** -8 + 2 * e) * mag + 1e-30
    err = np.abs(got.astype(np.float64) - ref)
    assert (err <= tol).all(), f"{where}: out off by {err.max()} ({(err / tol).max():.2f} of the tolerance)"
    empty = np.isneginf(ref_lse)
    assert np.array_equal(np.isneginf(lse), empty), where
    if not empty.all():
        off = np.abs(lse.astype(np.float64)[~empty] - ref_lse[~empty])
        assert off.max() <= e + 2.0 ** -22 * S, f"{where}: lse off by {off.max()}"

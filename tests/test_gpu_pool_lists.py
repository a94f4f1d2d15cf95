"""Calls that give a CTA more pieces of work than it plans at a time (64): many short requests, in the kernels for few and
for many rows, for weights and behind prefixes.  A few requests are repeated hundreds of times over the same blocks, so that
their oracle serves for all: the smallest and the largest value of an output over the repeats are both checked against it."""
import numpy as np
import pytest
import torch

from oracle import pool_attend
from pool_harness import PoolCase, check_out

pytestmark = pytest.mark.gpu

SMS, LIST = 152, 64


def ends(x, n):
    """Smallest and largest over the n repeats (NaN stays NaN)."""
    x = x.reshape((n, -1) + tuple(x.shape[1:]))
    return x.amin(0).double().cpu().numpy(), x.amax(0).double().cpu().numpy()


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(np.array(a, np.int32))).cuda()


def repeated(seed, ctx, q_len, hq, hk, d, bs, kv, lists, prefixes=()):
    """(case, repeats) whose kv heads' items fill `lists` lists of pieces in each CTA and begin another."""
    n = -(-(lists * LIST + 8) * SMS // (len(ctx) * hk))
    c = PoolCase(seed, ctx, q_len, hq, hk, d, bs, kv, prefixes=prefixes)
    c.cuda(max_req=n * len(ctx), max_tokens=n * c.n_tok, max_prefix_tokens=n * c.n_tok if prefixes else 0)
    m = np.array(q_len)
    return c, n, dict(q=c.d_q.repeat(n, 1, 1), cu_q=dev(np.concatenate([[0], np.cumsum(np.tile(m, n))])), ctx_len=c.d_ctx.repeat(n),
                      block2slot=c.d_table.repeat(n, 1))


def check(c, n, out, lse, prefix_of=None):
    outs, lses = ends(out, n), ends(lse, n)
    want = []
    for r in range(len(c.ctx)):
        pre = {} if prefix_of is None else dict(zip(("prefix_k", "prefix_v"), c.rows[len(c.ctx) + prefix_of[r]]))
        ref, ref_lse, mag, wt = pool_attend(c.query(r), *c.rows[r], c.softmax_scale, **pre)
        a, b = c.cu[r], c.cu[r + 1]
        for o, ls in zip(outs, lses):
            check_out(o[a:b], ls[a:b], ref, ref_lse, mag, c.d, f"request {r}")
        want.append(wt)
    return want


CASES = [  # contexts, query tokens, heads, kv heads, head dim, block size, lists
    ([40], [16], 32, 8, 128, 16, 1),                              # many rows: one row tile and one tile of keys a piece
    ([1], [65], 16, 16, 64, 16, 2),                                # (most rows see no key)
    ([90, 40], [70, 40], 32, 8, 64, 32, 1),                       # two row tiles a piece
    ([40, 300, 7, 129, 200], [16, 40, 1, 129, 30], 64, 16, 128, 16, 2),   # one and two in turn, items cut between CTAs
    ([33], [1], 32, 8, 128, 16, 1),                               # few rows
    ([5, 140, 1, 17], [1, 3, 1, 5], 64, 16, 64, 16, 2),
    ([20, 0, 64], [1, 1, 1], 2048, 1024, 64, 16, 2),               # at most 32 requests: planned by one warp first
]


@pytest.mark.parametrize("weight", [False, True])
@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("i", range(len(CASES)))
def test_more_pieces_than_a_list(i, kv, weight):
    ctx, m, hq, hk, d, bs, lists = CASES[i]
    c, n, args = repeated(50 + i, ctx, m, hq, hk, d, bs, kv, lists)
    out = torch.full((n * c.n_tok, hq, d), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((n * c.n_tok, hq), 7.0, device="cuda")
    w0 = torch.from_numpy(c.rng.random((len(ctx), hk, c.max_ctx)).astype(np.float32))
    w = w0.cuda().repeat(n, 1, 1) if weight else None
    c.pool.attn(0, out=out, lse=lse, weight=w, **args)
    torch.cuda.synchronize()
    assert c.pool.poll_error() == 0
    want = check(c, n, out, lse)
    if not weight:
        return
    for got in ends(w, n):
        for r, (length, q) in enumerate(zip(ctx, m)):
            p0 = max(0, length - q)
            ref = w0[r].double().numpy()
            ref[:, :p0] += want[r][:p0].T
            ref[:, p0:length] = want[r][p0:].T
            # each weight is a sum of terms exp(s - lse), each of the two off by at most e of check_out; 2^-23 for its rounding
            # and the addition's
            tol = (2 * 2.0 ** -23 * (d + 4) * 80 + 2.0 ** -23) * np.abs(ref) + 1e-6
            assert (np.abs(got[r] - ref) <= tol).all(), f"request {r}: weights off by {np.abs(got[r] - ref).max()}"


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("m", [1, 16])
def test_more_prefix_groups_than_a_list(m, kv):
    """Many groups of two requests behind a short prefix each: the prefix part and the own part both go through several lists
    (m = 16: 32 rows a request in the own part, 64 a group)."""
    hk = 16
    c, n, args = repeated(80 + m, [30, 21], [m, m], 4 * hk, hk, 64, 16, kv, 2, prefixes=[50])
    off, pre = dev(np.arange(0, 2 * n + 1, 2)), torch.full((n,), 50, dtype=torch.int32, device="cuda")
    out, lse = torch.full((n * c.n_tok, 4 * hk, 64), 7.0, dtype=torch.bfloat16, device="cuda"), torch.full((n * c.n_tok, 4 * hk), 7.0, device="cuda")
    c.pool.prefix_attn(0, prefix_req=off, prefix_len=pre, prefix2slot=dev(c.prefix_table).repeat(n, 1), out=out, lse=lse, **args)
    torch.cuda.synchronize()
    assert c.pool.poll_error() == 0
    check(c, n, out, lse, prefix_of=[0, 0])

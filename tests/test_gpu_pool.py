"""Device-resident pools on the GPU against the oracle (fp64)."""
import numpy as np
import pytest
import torch

import sparse_kv_cache_decode_gb300 as K
from oracle import pool_attend, pool_kept
from pool_harness import PoolCase, check_out

pytestmark = pytest.mark.gpu


def run_attn(c, window=0, sink=0, weight=False):
    out, lse = c.out()
    w0 = None
    if weight:
        w0 = torch.from_numpy(c.rng.random((len(c.ctx), c.hk, c.max_ctx)).astype(np.float32))
        w = w0.cuda()
    c.pool.attn(c.layer, c.d_q, c.d_cu, c.d_ctx, c.d_table, out, window=window, n_sink=sink, lse=lse, weight=w if weight else None)
    torch.cuda.synchronize()
    assert c.pool.poll_error() == 0
    return out.double().cpu().numpy(), lse.cpu().numpy(), (w.double().cpu().numpy(), w0.double().numpy()) if weight else None


def check_attn(c, got, lse, window=0, sink=0, weights=None):
    for r, n in enumerate(c.ctx):
        k, v = c.rows[r]
        ref, ref_lse, mag, wt = pool_attend(c.query(r), k, v, c.softmax_scale, window, sink)
        a, b = c.cu[r], c.cu[r + 1]
        check_out(got[a:b], lse[a:b], ref, ref_lse, mag, c.d, f"request {r}")
        if weights:
            w, w0 = weights
            m = c.q_len[r]
            want = w0[r].copy()
            p0 = max(0, n - m)
            want[:, :p0] += wt[:p0].T
            want[:, p0:n] = wt[p0:].T
            # each weight is a sum of terms exp(s - lse) off by at most e each (see check_out), twice
            tol = 2 * 2.0 ** -23 * (c.d + 4) * 80 * np.abs(want) + 1e-6
            assert (np.abs(w[r] - want) <= tol).all(), f"request {r}: weights off by {np.abs(w[r] - want).max()}"
            assert (w[r, :, n:] == w0[r, :, n:]).all()
    end = c.cu[-1]
    assert (got[end:] == 7.0).all() and (lse[end:] == 7.0).all()     # rows behind the last request


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("m", [1, 5, 24])
def test_many_tiles_per_sm(m, d, kv):
    """Ranges of a dozen tiles and more per SM, where the tile rings wrap several times, cut inside items: equal
    queries against equal keys, so that one request's oracle serves for all."""
    hq, hk, n, b = 8, 2, 2500, 64
    c = PoolCase(m * d, [n], [m], hq, hk, d, 64, kv).cuda(max_req=b, max_tokens=m * b)
    q = c.d_q.repeat(b, 1, 1)
    cu = torch.arange(0, m * b + 1, m, dtype=torch.int32, device="cuda")
    out = torch.empty_like(q)
    lse = torch.empty((m * b, hq), device="cuda")
    c.pool.attn(0, q, cu, c.d_ctx.repeat(b), c.d_table.repeat(b, 1), out, lse=lse)
    torch.cuda.synchronize()
    assert c.pool.poll_error() == 0
    ref, ref_lse, mag, _ = pool_attend(c.query(0), *c.rows[0], c.softmax_scale)
    out, lse = out.view(b, m, hq, d).double().cpu().numpy(), lse.view(b, m, hq).cpu().numpy()
    for r in range(b):
        check_out(out[r], lse[r], ref, ref_lse, mag, d, f"request {r}")


HEADS = [(8, 2, 128), (4, 4, 64), (12, 4, 128), (7, 1, 64), (16, 2, 64), (32, 2, 128)]

@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("m,g", [(1, 4), (5, 3), (30, 4), (200, 3), (300, 4)])
@pytest.mark.parametrize("shape", ["rising", "step", "falling"])
def test_logits_that_outgrow_the_first_tile(shape, m, g, kv):
    """Logits that rise (or fall) by hundreds over the context, smoothly or in one key: what a kernel takes for the
    maximum of a row early on is passed by far later, and a weight of the first keys vanishes.  The queries have a
    common component of 2, the keys one that moves from -2 to 2.5 (a logit moves by 4.5 * 2 * sqrt(d) = 102)."""
    n, d = 900, 128
    move = {"rising": lambda t: -2 + 4.5 * t / n, "step": lambda t: np.where(t == 700, 2.5, -2.0), "falling": lambda t: 2.5 - 4.5 * t / n}
    c = PoolCase(m + g, [n, 400], [m, 1], 2 * g, 2, d, 32, kv, key_shift=move[shape], q_shift=2.0, heavy=0.0).cuda()
    out, lse = c.out()
    c.pool.attn(0, c.d_q, c.d_cu, c.d_ctx, c.d_table, out, lse=lse)
    torch.cuda.synchronize()
    assert c.pool.poll_error() == 0
    got, lse = out.double().cpu().numpy(), lse.cpu().numpy()
    for r in range(2):
        ref, ref_lse, mag, _ = pool_attend(c.query(r), *c.rows[r], c.softmax_scale)
        a, b = c.cu[r], c.cu[r + 1]
        check_out(got[a:b], lse[a:b], ref, ref_lse, mag, d, f"request {r}", S=200)


@pytest.mark.parametrize("m", [1, 3, 100, 700])
def test_lanes_without_a_row(m):
    """Groups of 3 and 7 heads leave places of a row tile empty, and what an earlier call left in them may be
    anything: here the largest queries there are.  Results and running time do not depend on it."""
    for g in (3, 7):
        big = PoolCase(1, [700, 64], [700, 64], 8, 2, 128, 64).cuda()
        big.d_q.copy_(torch.where(big.d_q > 0, 3e38, -3e38))
        out, _ = big.out()
        big.pool.attn(0, big.d_q, big.d_cu, big.d_ctx, big.d_table, out)
        c = PoolCase(m + g, [900, 300], [m, 1], g, 1, 128, 64).cuda()
        got, lse, _ = run_attn(c)
        check_attn(c, got, lse)


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("d", [64, 128])
def test_long_prompt_ranges(d, kv):
    """Items of two row tiles, a dozen tiles and more of K and V per SM."""
    c = PoolCase(d, [3000, 2500], [3000, 1200], 12, 4, d, 64, kv).cuda()
    got, lse, _ = run_attn(c, 1500, 5)
    check_attn(c, got, lse, 1500, 5)


SINGLE = [  # contexts, window, sink, block size
    ([1], 0, 0, 16), ([0, 5, 0], 0, 0, 16), ([1, 15, 16, 17], 0, 0, 16), ([127, 128, 129, 130], 0, 0, 32), ([700], 0, 0, 128),
    ([700, 333], 100, 0, 16), ([700, 333, 90], 100, 4, 64), ([1000], 1, 0, 16), ([1000], 1, 1, 128), ([513], 128, 130, 32),
    ([2049, 1, 0, 640], 257, 64, 64), ([300, 301], 1000, 3, 16), ([5000], 0, 0, 64), ([4097, 63], 2048, 7, 16),
]


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("m", [1, 3, 7])
def test_query_rows_of_every_size(m, d, kv):
    """Rows whose elements differ by many powers of two, rows of zeros, rows far larger or smaller than their neighbours.

    With an E4M3 pool a row of Q may be held to 2^-18 of its largest element (4 here) wherever an element is 2^-10 of that
    or smaller.  A key's |k| sum to less than 128 * 4 (4 times a normal's mean of 0.8 for heavy keys), so a logit is off by at
    most 512 * 4 * 2^-18 / sqrt(128) = 7e-4 by it, inside the logit error that check_out allows (1.3e-3 at d = 128, and half
    the sum and 0.7e-3 / sqrt(2) at d = 64)."""
    c = PoolCase(40 + m + d, [700, 129, 64], [m] * 3, 8, 2, d, 32, kv)
    q = c.q.float()
    t = torch.arange(c.n_tok * 8).view(c.n_tok, 8, 1) % 5
    spike = torch.zeros(d)
    spike[d // 3] = 4.0
    q = torch.where(t == 0, q * 2.0 ** -11 + spike, torch.where(t == 1, q * 0, torch.where(t == 2, q * 2.0 ** -30, torch.where(t == 3, q * 2.0 ** -125, q * 1.5))))
    c.q = q.to(torch.bfloat16)
    c.cuda()
    got, lse, _ = run_attn(c)
    check_attn(c, got, lse)


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("i", range(len(SINGLE)))
def test_single_tokens(i, kv):
    ctx, window, sink, bs = SINGLE[i]
    hq, hk, d = HEADS[i % len(HEADS)]
    c = PoolCase(100 + i, ctx, [1] * len(ctx), hq, hk, d, bs, kv).cuda()
    got, lse, _ = run_attn(c, window, sink)
    check_attn(c, got, lse, window, sink)


CHUNKS = [  # contexts, query tokens, window, sink, block size
    ([3], [3], 0, 0, 16), ([200], [200], 0, 0, 16), ([257], [257], 0, 0, 64), ([700], [130], 0, 0, 32),
    ([300, 40, 5, 129], [300, 1, 5, 64], 0, 0, 16), ([600], [600], 100, 4, 16), ([600, 1], [333, 1], 64, 0, 128),
    ([1025, 0, 511], [129, 0, 511], 200, 17, 64), ([5], [9], 0, 0, 16), ([20, 0], [33, 2], 4, 1, 16), ([900], [7], 300, 200, 32),
    ([1300], [1300], 0, 0, 128), ([400, 400, 400], [2, 3, 4], 33, 5, 16),
]


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("i", range(len(CHUNKS)))
def test_chunks(i, kv):
    ctx, m, window, sink, bs = CHUNKS[i]
    hq, hk, d = HEADS[(i + 2) % len(HEADS)]
    c = PoolCase(300 + i, ctx, m, hq, hk, d, bs, kv, pad_tokens=3).cuda()
    got, lse, _ = run_attn(c, window, sink)
    check_attn(c, got, lse, window, sink)


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("heads", HEADS)
def test_every_head_layout(heads, kv):
    hq, hk, d = heads
    c = PoolCase(hq + d, [150, 260, 33], [40, 1, 33], hq, hk, d, 32, kv).cuda()
    got, lse, w = run_attn(c, 90, 3, weight=True)
    check_attn(c, got, lse, 90, 3, w)


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("i", range(6))
def test_weights(i, kv):
    ctx, m, window, sink = [([300, 0, 1, 129], [1, 1, 1, 1], 0, 0), ([500], [500], 0, 0), ([400, 130], [32, 130], 0, 0),
                            ([700, 64], [3, 5], 100, 4), ([5], [8], 0, 0), ([2000], [1], 0, 0)][i]
    hq, hk, d = HEADS[i]
    c = PoolCase(500 + i, ctx, m, hq, hk, d, (16, 32, 64, 128)[i % 4], kv, pad_tokens=1, max_ctx=max(ctx) + 37).cuda()
    got, lse, w = run_attn(c, window, sink, weight=True)
    check_attn(c, got, lse, window, sink, w)


PREFIX = [  # prefixes, their request offsets, contexts, query tokens, block size
    ([100], [0, 1], [5], [1], 16), ([1000], [0, 4], [1, 17, 200, 64], [1, 1, 1, 1], 16),
    ([130, 1, 700], [0, 2, 3, 6], [9, 30, 4, 129, 5, 260], [5, 5, 4, 1, 3, 7], 32),
    ([257], [1, 3], [40, 50, 60, 70], [2, 1, 3, 1], 64),                 # the first and last request have no prefix
    ([0, 64], [0, 2, 4], [8, 0, 8, 3], [1, 1, 2, 5], 16),                # an empty prefix, an empty context, p < 0
    ([2000], [0, 40], [3] * 40, [1] * 40, 128), ([333], [0, 2], [150, 70], [150, 70], 16), ([64, 65], [0, 0, 2], [5, 6], [1, 1], 64),
]


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("i", range(len(PREFIX)))
def test_prefix(i, kv):
    pre, off, ctx, m, bs = PREFIX[i]
    hq, hk, d = HEADS[i % len(HEADS)]
    c = PoolCase(700 + i, ctx, m, hq, hk, d, bs, kv, prefixes=pre, pad_tokens=2).cuda()
    out, lse = c.out()
    dev = lambda a: torch.tensor(np.array(a, np.int32)).cuda()  # noqa: E731
    c.pool.prefix_attn(0, c.d_q, c.d_cu, c.d_ctx, c.d_table, dev(off), dev(pre), dev(c.prefix_table), out, lse=lse)
    torch.cuda.synchronize()
    assert c.pool.poll_error() == 0
    got, lse = out.double().cpu().numpy(), lse.cpu().numpy()
    for r in range(len(ctx)):
        g = [j for j in range(len(pre)) if off[j] <= r < off[j + 1]]
        pk, pv = c.rows[len(ctx) + g[0]] if g else (None, None)
        k, v = c.rows[r]
        ref, ref_lse, mag, _ = pool_attend(c.query(r), k, v, c.softmax_scale, prefix_k=pk, prefix_v=pv)
        a, b = c.cu[r], c.cu[r + 1]
        check_out(got[a:b], lse[a:b], ref, ref_lse, mag, d, f"request {r}")
    assert (got[c.cu[-1]:] == 7.0).all()


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("i", range(12))
def test_evict(i, kv):
    ctx, keep, sink, recent, bs, kind = [
        ([100, 64, 33, 0], 64, 4, 8, 16, "plain"), ([1], 1, 0, 0, 16, "plain"), ([300], 299, 0, 299, 32, "plain"),
        ([1000, 999, 200], 128, 0, 0, 64, "ties"), ([513, 700], 65, 1, 64, 128, "plain"), ([2000], 1000, 4, 100, 16, "nan"),
        ([40000], 3000, 4, 32, 128, "plain"), ([3000, 100], 7, 7, 0, 16, "zeros"),
        ([60000], 2500, 3, 60, 64, "ties"),
        ([45000] + [3, 70] * 80, 61, 2, 3, 128, "ties"),              # many units: one CTA each
        ([340000, 20], 1500, 4, 64, 128, "plain"),                    # runs longer than shared memory holds
        ([9000, 33, 8193, 4097], 4000, 3990, 5, 16, "zeros")][i]   # runs without a token to choose from
    hq, hk, d = HEADS[i % len(HEADS)] if i < 10 else HEADS[0]
    if i in (9, 10):
        hq, hk, d = 2, 1, 64
    need = [-(-min(n, keep) // bs) for n in ctx]
    c = PoolCase(900 + i, ctx, [0] * len(ctx), hq, hk, d, bs, kv, spare=sum(need)).cuda()
    w = c.rng.exponential(1.0, (len(ctx), hk, c.max_ctx)).astype(np.float32)
    if kind == "ties":
        w = np.round(w * 2) / 2 * np.where(c.rng.random(w.shape) < 0.5, -1, 1).astype(np.float32)
    elif kind == "nan":
        w[c.rng.random(w.shape) < 0.6] = np.nan
        w[c.rng.random(w.shape) < 0.02] = -np.inf
        w[c.rng.random(w.shape) < 0.02] = np.inf
    elif kind == "zeros":
        w[:] = 0.0
    dst = np.full((len(ctx), c.nb), -1, np.int32)
    free = c.rng.permutation(np.arange(c.n_slots - sum(need), c.n_slots))
    at = 0
    for r, n in enumerate(need):
        dst[r, :n] = free[at:at + n]
        at += n
    before = c.dk.clone()
    kept = torch.full((len(ctx), hk, keep), -5, dtype=torch.int32, device="cuda")
    n_kept = torch.full((len(ctx),), -5, dtype=torch.int32, device="cuda")
    w_out = torch.full((len(ctx), hk, c.max_ctx), -5.0, device="cuda")
    c.pool.evict(0, torch.from_numpy(w).cuda(), c.d_ctx, c.d_table, keep, sink, recent, torch.from_numpy(dst).cuda(), kept, n_kept, w_out)
    torch.cuda.synchronize()
    assert c.pool.poll_error() == 0
    kept, n_kept, w_out = kept.cpu().numpy(), n_kept.cpu().numpy(), w_out.cpu().numpy()
    bits = (lambda x: x.cpu().view(torch.int16).numpy()) if kv == "bf16" else (lambda x: x.cpu().numpy())
    for pool, old in ((bits(c.dk), bits(c.k)), (bits(c.dv), bits(c.v))):
        for r, n in enumerate(ctx):
            m = min(n, keep)
            assert n_kept[r] == m
            for h in range(hk):
                want = pool_kept(w[r, h], n, keep, sink, recent)
                assert np.array_equal(kept[r, h, :m], want), (r, h)
                assert (kept[r, h, m:] == -5).all()
                assert np.array_equal(w_out[r, h, :m], w[r, h, want], equal_nan=True) and (w_out[r, h, m:] == -5).all()
                j = np.arange(m)
                a = pool[0, dst[r, j // bs], h, j % bs]
                assert np.array_equal(a, old[0, c.table[r, want // bs], h, want % bs])
        assert np.array_equal(pool[0, :c.n_used + 2], old[0, :c.n_used + 2])       # sources untouched
    assert torch.equal(before.view(torch.uint8)[:, :c.n_used], c.dk.view(torch.uint8)[:, :c.n_used])


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("heads", HEADS[:4])
def test_append(heads, kv):
    hq, hk, d = heads
    ctx, m = [40, 1, 17, 0, 64], [5, 1, 17, 0, 1]
    c = PoolCase(hq, ctx, m, hq, hk, d, 16, kv, n_layer=2, layer=1, pad_tokens=2).cuda()
    wide = torch.randn((c.n_tok, 2 * hk + 1, d), generator=torch.Generator().manual_seed(5)).to(torch.bfloat16).cuda()
    k_new, v_new = wide[:, :hk], wide[:, hk:2 * hk]                  # slices of one projection
    ref_k, ref_v = c.dk.clone(), c.dv.clone()
    for x, new, scale in ((ref_k, k_new, c.scales[0]), (ref_v, v_new, c.scales[1])):
        if kv == "bf16":
            codes = new.contiguous()
        else:
            codes = torch.empty(new.shape, dtype=torch.uint8, device="cuda")
            K.quantize_e4m3(new.contiguous(), codes, scale)
        for r in range(len(ctx)):
            for i in range(m[r]):
                p = ctx[r] - m[r] + i
                x[1, c.table[r, p // 16], :, p % 16] = codes[c.cu[r] + i]
    c.pool.append(1, k_new, v_new, c.d_cu, c.d_ctx, c.d_table)
    torch.cuda.synchronize()
    assert c.pool.poll_error() == 0
    assert torch.equal(c.dk.view(torch.uint8), ref_k.view(torch.uint8)) and torch.equal(c.dv.view(torch.uint8), ref_v.view(torch.uint8))

"""Device-resident pools as a serving loop uses them: calls refused on the host, bad lengths and slots reported by the
device, captured and replayed calls, other streams, several layers, and a run of all the operators together."""
import ctypes

import numpy as np
import pytest
import torch

import sparse_kv_cache_decode_gb300 as K
from oracle import pool_attend, pool_kept
from pool_harness import PoolCase, check_out

pytestmark = pytest.mark.gpu
INVALID_ARG, BAD_INDEX = 1, 7


def dev(a, t=np.int32):
    return torch.from_numpy(np.ascontiguousarray(np.array(a, t))).cuda()


def attend(c, window=0, sink=0, **kw):
    out, lse = c.out()
    c.pool.attn(c.layer, c.d_q, c.d_cu, c.d_ctx, c.d_table, out, window=window, n_sink=sink, lse=lse, **kw)
    return out, lse


def check(c, out, lse, window=0, sink=0, only=None):
    got, lse = out.double().cpu().numpy(), lse.cpu().numpy()
    for r in range(len(c.ctx)):
        if only is None or r in only:
            ref, ref_lse, mag, _ = pool_attend(c.query(r), *c.rows[r], c.softmax_scale, window, sink)
            a, b = c.cu[r], c.cu[r + 1]
            check_out(got[a:b], lse[a:b], ref, ref_lse, mag, c.d, f"request {r}")


def small(**kw):
    return PoolCase(1, [70, 33], [2, 3], 8, 2, 64, 16, prefixes=[20], pad_tokens=1, **kw).cuda()


# ------------------------------------------------------------------ refusals
def evict_args(c, keep=8):
    n, hk = len(c.ctx), c.hk
    return [torch.zeros((n, hk, c.max_ctx), device="cuda"), c.d_ctx, c.d_table, keep, 1, 2, c.d_table.clone(),
            torch.zeros((n, hk, keep), dtype=torch.int32, device="cuda"), torch.zeros(n, dtype=torch.int32, device="cuda"),
            torch.zeros((n, hk, c.max_ctx), device="cuda")]


def test_host_refusals():
    c = small()
    p, out, lse = c.pool, *c.out()
    base = [0, c.d_q, c.d_cu, c.d_ctx, c.d_table, out]
    before = p.launch_count()

    def refused(kind, call, *a, **kw):
        with pytest.raises(kind):
            call(*a, **kw)

    for i, bad in [(0, 1), (0, -1)]:
        refused(K.KvsError, p.attn, *(base[:i] + [bad] + base[i + 1:]))
    refused(K.KvsError, p.attn, *base, window=-1)
    refused(K.KvsError, p.attn, *base, n_sink=-1)
    refused(K.KvsError, p.attn, *(base[:5] + [c.d_q]))                               # out is q
    for i, bad in [(1, c.d_q.float()), (1, c.d_q[:, :4]), (1, c.d_q[:, :, :32]), (1, c.d_q.cpu()), (1, c.d_q.transpose(0, 1)),
                   (2, c.d_cu.long()), (2, c.d_cu[:2]), (3, c.d_ctx.float()), (4, c.d_table[:, :1]), (4, c.d_table[:1]),
                   (4, c.d_table.cpu()), (5, out[:3]), (5, out.float()), (5, out.transpose(1, 2))]:
        refused(ValueError, p.attn, *(base[:i] + [bad] + base[i + 1:]))
    refused(ValueError, p.attn, *base, lse=lse.double())
    refused(ValueError, p.attn, *base, lse=lse[:2])
    refused(ValueError, p.attn, *base, weight=torch.zeros((2, 2, 3), device="cuda"))
    # q: tokens that are no multiple of 16 bytes apart, a start that is not 16-byte aligned
    wide = torch.zeros((c.n_tok, 8 * 64 + 4), dtype=torch.bfloat16, device="cuda")
    refused(K.KvsError, p.attn, *(base[:1] + [wide[:, :512].unflatten(1, (8, 64))] + base[2:]))
    flat = torch.zeros(c.n_tok * 512 + 4, dtype=torch.bfloat16, device="cuda")
    refused(K.KvsError, p.attn, *(base[:1] + [flat[4:].view(c.n_tok, 8, 64)] + base[2:]))
    # more tokens or requests than configured
    refused(K.KvsError, p.attn, 0, torch.zeros((c.n_tok + 1, 8, 64), dtype=torch.bfloat16, device="cuda"), c.d_cu, c.d_ctx, c.d_table,
            torch.zeros((c.n_tok + 1, 8, 64), dtype=torch.bfloat16, device="cuda"))
    refused(K.KvsError, p.attn, 0, c.d_q, dev([0, 1, 2, 3]), dev([1, 1, 1]), dev(np.zeros((3, c.nb))), out)
    # append
    new = torch.zeros((c.n_tok, 2, 64), dtype=torch.bfloat16, device="cuda")
    refused(ValueError, p.append, 0, new, new[:2], c.d_cu, c.d_ctx, c.d_table)
    refused(ValueError, p.append, 0, new.float(), new, c.d_cu, c.d_ctx, c.d_table)
    refused(K.KvsError, p.append, 3, new, new.clone(), c.d_cu, c.d_ctx, c.d_table)
    # prefixes
    pre = [0, c.d_q, c.d_cu, c.d_ctx, c.d_table, dev([0, 2]), dev([20]), dev(c.prefix_table)]
    refused(ValueError, p.prefix_attn, *(pre[:5] + [dev([0, 1, 2])] + pre[6:]), out)
    refused(ValueError, p.prefix_attn, *(pre[:7] + [c.d_table]), out)
    refused(K.KvsError, p.prefix_attn, *pre, c.d_q)
    refused(K.KvsError, p.prefix_attn, *(pre[:5] + [dev([0, 1, 1, 2]), dev([1, 1, 1]), dev(np.zeros((3, c.nb)))]), out)
    # eviction
    e = evict_args(c)
    for i, bad in [(4, -1), (5, -1), (4, 9), (5, 8), (9, e[0]), (8, c.d_ctx), (6, c.d_table)]:
        refused(K.KvsError, p.evict, 0, *(e[:i] + [bad] + e[i + 1:]))
    for i, bad in [(0, e[0].double()), (7, e[7][:, :, :4]), (8, e[8][:1]), (9, e[9][:1])]:
        refused(ValueError, p.evict, 0, *(e[:i] + [bad] + e[i + 1:]))
    refused(K.KvsError, p.evict, 0, *(e[:3] + [c.max_ctx + 1] + e[4:7] + [torch.zeros((2, 2, c.max_ctx + 1), dtype=torch.int32, device="cuda")] + e[8:]))
    refused(K.KvsError, p.evict, 0, *(e[:3] + [0, 0, 0] + e[6:7] + [torch.zeros((2, 2, 0), dtype=torch.int32, device="cuda")] + e[8:]))
    assert p.launch_count() == before and p.poll_error() == 0
    assert (out == 7).all()
    p.close()
    refused(ValueError, p.attn, *base)


def test_create_refuses_memory_it_cannot_use():
    c = small()
    L, cfg, h = K.lib(), c.pool.cfg, ctypes.c_void_p()
    n = L.kvs_pool_workspace_bytes(ctypes.byref(cfg))
    ws = torch.empty(n + 512, dtype=torch.uint8, device="cuda")
    at = (ws.data_ptr() + 255) // 256 * 256
    host = torch.empty(1 << 16, dtype=torch.uint8).pin_memory()
    k, v = c.dk.data_ptr(), c.dv.data_ptr()
    for a in [(k + 16, v, at, n), (k, v + 16, at, n), (k, v, at + 16, n), (k, v, at, n - 1), (host.data_ptr() // 256 * 256, v, at, n),
              (k, k, at, n), (k, v, k, n)]:
        assert L.kvs_pool_create(ctypes.byref(cfg), *a, ctypes.byref(h)) == INVALID_ARG and not h, a


@pytest.mark.parametrize("m", [2, 200])          # the kernels for few and for many rows
@pytest.mark.parametrize("bad", ["slot", "unset", "length", "negative", "offset"])
def test_bad_indices_are_reported_and_stay_with_their_request(bad, m):
    c = PoolCase(3, [300, 411, 250], [m, m, m], 8, 2, 128, 16, pad_tokens=3).cuda()
    table, ctx, cu = c.table.copy(), np.array(c.ctx, np.int32), c.cu.copy()
    if bad == "slot":
        table[1, 2] = c.n_slots
    elif bad == "unset":
        table[1, 3] = -1
    elif bad == "length":
        ctx[1] = c.max_ctx + 1
    elif bad == "negative":
        ctx[1] = -4
    else:
        cu[1:3] = cu[2], cu[1]              # requests 0 and 1 swap an offset: 0 and 2 get other rows, 1 none
    c.d_table, c.d_ctx, c.d_cu = dev(table), dev(ctx), dev(cu)
    w = torch.zeros((3, 2, c.max_ctx), device="cuda")
    for weight in (None, w):
        out, lse = attend(c, weight=weight)
        assert c.pool.poll_error() == BAD_INDEX
        assert c.pool.poll_error() == 0             # read and cleared
        if bad != "offset":
            check(c, out, lse, only=(0, 2))
        assert (out[c.cu[-1]:] == 7).all()


def test_eviction_and_append_report_bad_slots():
    c = PoolCase(4, [100, 64], [1, 1], 8, 2, 64, 16, spare=8).cuda()
    e = evict_args(c, keep=32)
    dst = np.full((2, c.nb), -1, np.int32)
    dst[0, :2] = c.n_slots - 8, c.n_slots - 7       # the second request has nowhere to go
    e[6] = dev(dst)
    before = c.dk.clone()
    c.pool.evict(0, *e)
    assert c.pool.poll_error() == BAD_INDEX
    used = before.view(torch.int16)[:, :c.n_used + 2]
    assert torch.equal(c.dk.view(torch.int16)[:, :c.n_used + 2], used) and (e[8].cpu() == 32).all()
    new = torch.ones((2, 2, 64), dtype=torch.bfloat16, device="cuda")
    bad = c.table.copy()
    bad[1, 3] = c.n_slots
    c.pool.append(0, new, new.clone(), c.d_cu, c.d_ctx, dev(bad))
    assert c.pool.poll_error() == BAD_INDEX
    assert (c.dk[0, c.table[0, 99 // 16], :, 99 % 16] == 1).all() and not (c.dk[0, c.table[1, 3], :, 15] == 1).all()


# ------------------------------------------------------------------ empty calls, layouts, layers
def test_calls_without_requests_or_tokens():
    c = small()
    n0 = c.pool.launch_count()
    e = torch.empty
    z = dict(dtype=torch.int32, device="cuda")
    q0 = e((0, 8, 64), dtype=torch.bfloat16, device="cuda")
    c.pool.attn(0, q0, torch.zeros(1, **z), e((0,), **z), e((0, c.nb), **z), q0.clone())
    c.pool.attn(0, q0, torch.zeros(3, **z), c.d_ctx, c.d_table, q0.clone())
    c.pool.append(0, q0[:, :2], q0[:, :2], torch.zeros(3, **z), c.d_ctx, c.d_table)
    c.pool.prefix_attn(0, q0, torch.zeros(3, **z), c.d_ctx, c.d_table, dev([0, 2]), dev([20]), dev(c.prefix_table), q0.clone())
    assert c.pool.launch_count() == n0
    out, lse = c.out()
    c.pool.attn(0, c.d_q, torch.zeros(3, **z), c.d_ctx, c.d_table, out, lse=lse)           # tokens of no request
    assert c.pool.poll_error() == 0 and (out == 7).all() and (lse == 7).all()
    c.pool.prefix_attn(0, c.d_q, c.d_cu, c.d_ctx, c.d_table, dev([0]), e((0,), **z), e((0, c.nb), **z), out, lse=lse)   # no prefix
    assert c.pool.poll_error() == 0
    check(c, out, lse)
    out, lse = c.out()
    L = K.lib()
    args = [t.data_ptr() for t in (c.d_cu, c.d_ctx, c.d_table)]
    assert L.kvs_pool_prefix_attn(c.pool.h, 0, c.d_q.data_ptr(), 8 * 64, *args, 2, c.n_tok, None, None, None, 0, out.data_ptr(),
                                  lse.data_ptr(), torch.cuda.current_stream().cuda_stream) == 0
    assert c.pool.poll_error() == 0
    check(c, out, lse)


@pytest.mark.parametrize("m", [1, 90])
def test_layers_and_a_fused_projection(m):
    c = PoolCase(6, [500, 120], [m, m], 12, 3, 64, 32, n_layer=3, layer=2).cuda()
    wide = torch.full((c.n_tok, 20, 64), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:, 4:16] = c.d_q
    c.d_q = wide[:, 4:16]
    check(c, *attend(c, 77, 3), 77, 3)
    assert c.pool.poll_error() == 0


def test_pool_past_32_bit_offsets():
    """K and V of 2^32 elements and more each; the request's blocks are at both ends."""
    hk, bs, d, n = 8, 128, 128, 1000
    n_slots = (1 << 32) // (hk * bs * d) + 40
    r = np.random.default_rng(11)
    k = torch.empty((1, n_slots, hk, bs, d), dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    pool = K.Pool(K.make_pool_config(1, n_slots, 16, hk, d, bs, 2048, 1, 512), k, v)
    table = np.full((1, 16), -1, np.int32)
    table[0, :8] = [n_slots - 1, 0, n_slots - 2, n_slots // 2 + 1, 1, n_slots - 30, n_slots - 17, 2]
    new = [torch.from_numpy(r.standard_normal((n, hk, d)).astype(np.float32)).to(torch.bfloat16) for _ in range(2)]
    for a in range(0, n, 500):
        pool.append(0, new[0][a:a + 500].cuda(), new[1][a:a + 500].cuda(), dev([0, 500]), dev([a + 500]), dev(table))
    kv = [x.double().numpy() for x in new]
    for m in (1, 300):
        q = torch.from_numpy(r.standard_normal((m, 16, d)).astype(np.float32)).to(torch.bfloat16)
        out, lse = torch.empty((m, 16, d), dtype=torch.bfloat16, device="cuda"), torch.empty((m, 16), device="cuda")
        pool.attn(0, q.cuda(), dev([0, m]), dev([n]), dev(table), out, lse=lse)
        ref, ref_lse, mag, _ = pool_attend(q.double().numpy(), *kv, float(np.float32(1 / np.sqrt(d))))
        check_out(out.double().cpu().numpy(), lse.cpu().numpy(), ref, ref_lse, mag, d)
    w = r.random((1, hk, 2048)).astype(np.float32)
    dst = np.full((1, 16), -1, np.int32)
    dst[0, :3] = [n_slots - 5, 7, n_slots - 9]
    kept, n_kept = torch.zeros((1, hk, 300), dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    pool.evict(0, torch.from_numpy(w).cuda(), dev([n]), dev(table), 300, 4, 10, dev(dst), kept, n_kept, torch.zeros((1, hk, 2048), device="cuda"))
    assert pool.poll_error() == 0
    for h in range(hk):
        want = pool_kept(w[0, h], n, 300, 4, 10)
        j = np.arange(300)
        for x, src in ((k, new[0]), (v, new[1])):
            got = x[0, torch.from_numpy(dst[0, j // bs]).long().cuda(), h, torch.from_numpy(j % bs).cuda()]
            assert torch.equal(got.cpu(), src[want, h])


# ------------------------------------------------------------------ streams and graphs
@pytest.mark.parametrize("m", [1, 70])
def test_another_stream_and_two_pools_at_once(m):
    c = PoolCase(7, [3000, 2000], [m, m], 8, 2, 128, 64).cuda()
    twin = K.Pool(c.pool.cfg, c.dk, c.dv)               # the same memory, a workspace of its own
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    ref, _ = attend(c)
    torch.cuda.synchronize()
    outs = [[], []]
    for _ in range(8):
        for i, (p, s) in enumerate(((c.pool, s1), (twin, s2))):
            out, lse = c.out()
            s.wait_stream(torch.cuda.current_stream())
            p.attn(0, c.d_q, c.d_cu, c.d_ctx, c.d_table, out, lse=lse, stream=s)
            outs[i].append((out, lse))
    torch.cuda.synchronize()
    for out, lse in outs[0] + outs[1]:
        assert torch.equal(out, ref)                    # the same split, so the same roundings
    check(c, *outs[1][3])
    assert c.pool.poll_error() == 0 and twin.poll_error() == 0


def test_captured_calls_replay_with_new_lengths():
    """append, attention with weights and eviction captured once; replayed with other lengths, offsets, tables and inputs."""
    a = PoolCase(8, [600, 200, 5], [1, 40, 5], 8, 2, 64, 16, spare=40, max_ctx=700, pad_tokens=10)
    b = PoolCase(9, [33, 700, 0], [20, 30, 0], 8, 2, 64, 16, spare=40, max_ctx=700, pad_tokens=6)
    assert a.n_tok == b.n_tok
    n_slots = max(a.n_slots, b.n_slots)
    kp = torch.zeros((1, n_slots, 2, 16, 64), dtype=torch.bfloat16, device="cuda")
    vp = torch.zeros_like(kp)
    pool = K.Pool(K.make_pool_config(**(a.cfg | dict(n_slots=n_slots))), kp, vp)
    nb, keep = a.nb, 24
    q, cu, ctx, table, dst = a.q.cuda(), dev(a.cu), dev(a.ctx), dev(a.table), dev(np.full((3, nb), -1))
    kn, vn = torch.zeros((a.n_tok, 2, 64), dtype=torch.bfloat16, device="cuda"), torch.zeros((a.n_tok, 2, 64), dtype=torch.bfloat16, device="cuda")
    w, w2 = torch.zeros((3, 2, 700), device="cuda"), torch.zeros((3, 2, 700), device="cuda")
    kept, n_kept = torch.zeros((3, 2, keep), dtype=torch.int32, device="cuda"), torch.zeros(3, dtype=torch.int32, device="cuda")
    out, lse = torch.empty_like(q), torch.empty((a.n_tok, 8), device="cuda")
    graph, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=s):
        pool.append(0, kn, vn, cu, ctx, table, stream=s)
        pool.attn(0, q, cu, ctx, table, out, lse=lse, weight=w, stream=s)
        pool.evict(0, w, ctx, table, keep, 2, 8, dst, kept, n_kept, w2, stream=s)
    for c in (a, b, a):
        kp[:, :c.n_slots].copy_(c.k)
        vp[:, :c.n_slots].copy_(c.v)
        for r, n in enumerate(c.ctx):                   # the last tokens arrive by the call
            m = c.q_len[r]
            for x, dst_new, i in ((kp, kn, 0), (vp, vn, 1)):
                rows = torch.from_numpy(c.rows[r][i][n - m:]).to(torch.bfloat16)
                dst_new[c.cu[r]:c.cu[r + 1]].copy_(rows)
                for j in range(n - m, n):
                    x[0, c.table[r, j // 16], :, j % 16] = float("nan")
        d2 = np.full((3, nb), -1, np.int32)
        d2[:, :2] = (n_slots - 6 + np.arange(6)).reshape(3, 2)
        q.copy_(c.q), cu.copy_(torch.from_numpy(c.cu)), ctx.copy_(torch.tensor(c.ctx, dtype=torch.int32))
        table.copy_(torch.from_numpy(c.table)), dst.copy_(torch.from_numpy(d2))
        w.zero_(), out.fill_(7.0), lse.fill_(7.0)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert pool.poll_error() == 0
        check(c, out, lse)
        assert (out[c.cu[-1]:] == 7).all()
        wh, kh = w.cpu().numpy(), kept.cpu().numpy()
        for r, n in enumerate(c.ctx):
            assert int(n_kept[r]) == min(n, keep)
            total = wh[r].sum()                         # each row's weights sum to 1, over 4 heads per kv head
            rows = sum(1 for i in range(c.q_len[r]) if n - c.q_len[r] + i >= 0)
            assert abs(total - rows * 8) <= 2e-3 * rows * 8 + 1e-5
            for h in range(2):
                want = pool_kept(wh[r, h], n, keep, 2, 8)
                assert np.array_equal(kh[r, h, :len(want)], want)


def test_results_do_not_change_from_run_to_run():
    for m, kv in ((1, "bf16"), (3, "fp8"), (150, "bf16"), (150, "fp8")):
        c = PoolCase(10 + m, [5000, 777, 2222], [m] * 3, 8, 2, 128, 32, kv).cuda()
        w = [torch.zeros((3, 2, c.max_ctx), device="cuda") for _ in range(2)]
        (o1, l1), (o2, l2) = attend(c, weight=w[0]), attend(c, weight=w[1])
        torch.cuda.synchronize()
        assert torch.equal(o1, o2) and torch.equal(l1, l2) and torch.equal(w[0], w[1])


# ------------------------------------------------------------------ the operators together
@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_serving_run(kv):
    """A prompt in chunks with weights, eviction to a budget, decode steps over what was kept, all beside a shared prefix."""
    hq, hk, d, bs, NL, keep = 8, 2, 128, 16, 2, 96
    r = np.random.default_rng(21)
    prompts, n_dec, max_ctx = [230, 150, 60], 5, 256
    nb = max_ctx // bs
    n_req, n_slots = 3, 3 * nb * 2 + 8
    ks, vs = (0.05, 0.03) if kv == "fp8" else (1.0, 1.0)
    pools = [torch.zeros((NL, n_slots, hk, bs, d), dtype=torch.uint8 if kv == "fp8" else torch.bfloat16, device="cuda") for _ in range(2)]
    pool = K.Pool(K.make_pool_config(NL, n_slots, hq, hk, d, bs, max_ctx, n_req, 512, 16, kv_dtype=kv, k_scale=ks, v_scale=vs), *pools)
    order = r.permutation(n_slots).astype(np.int32)
    table, table2, pre_table = order[:3 * nb].reshape(3, nb), order[3 * nb:6 * nb].reshape(3, nb), np.full((1, nb), -1, np.int32)
    pre_table[0, :4] = order[6 * nb:6 * nb + 4]
    scale = float(np.float32(1 / np.sqrt(d)))

    def rows(n, heads):
        return torch.from_numpy(r.standard_normal((n, heads, d)).astype(np.float32)).to(torch.bfloat16)

    def held(t, s):                     # what the pool holds of new rows
        return t.double().numpy() if kv == "bf16" else (t.float() / s).clamp(-448, 448).to(torch.float8_e4m3fn).double().numpy() * np.float32(s)

    hist = [[[np.zeros((0, hk, d))] * 2 for _ in range(n_req)] for _ in range(NL)]
    weight = torch.zeros((NL, n_req, hk, max_ctx), device="cuda")
    want_w = np.zeros((NL, n_req, hk, max_ctx))

    def step(layer, lens, q_len, tab, w, ref_w):
        cu = np.concatenate([[0], np.cumsum(q_len)])
        q, kn, vn = rows(cu[-1], hq), rows(cu[-1], hk), rows(cu[-1], hk)
        out, lse = torch.empty((cu[-1], hq, d), dtype=torch.bfloat16, device="cuda"), torch.empty((cu[-1], hq), device="cuda")
        pool.append(layer, kn.cuda(), vn.cuda(), dev(cu), dev(lens), dev(tab))
        pool.attn(layer, q.cuda(), dev(cu), dev(lens), dev(tab), out, lse=lse, weight=w)
        for i in range(n_req):
            a, b = cu[i], cu[i + 1]
            hist[layer][i] = [np.concatenate([hist[layer][i][0], held(kn[a:b], ks)]), np.concatenate([hist[layer][i][1], held(vn[a:b], vs)])]
            assert len(hist[layer][i][0]) == lens[i]
            ref, ref_lse, mag, wt = pool_attend(q[a:b].double().numpy(), *hist[layer][i], scale)
            check_out(out[a:b].double().cpu().numpy(), lse[a:b].cpu().numpy(), ref, ref_lse, mag, d, f"layer {layer} request {i}")
            p0 = lens[i] - q_len[i]
            ref_w[i, :, :p0] += wt[:p0].T
            ref_w[i, :, p0:lens[i]] = wt[p0:].T

    for chunk in (0, 1):
        q_len = [p // 2 if chunk == 0 else p - p // 2 for p in prompts]
        lens = [p // 2 if chunk == 0 else p for p in prompts]
        for layer in range(NL):
            step(layer, lens, q_len, table, weight[layer], want_w[layer])
    tol = 2 * 2.0 ** -23 * (d + 4) * 80
    assert (np.abs(weight.cpu().numpy() - want_w) <= tol * np.abs(want_w) + 2e-6).all()
    # to the budget; the old blocks are free after it
    kept, n_kept = torch.zeros((n_req, hk, keep), dtype=torch.int32, device="cuda"), torch.zeros(n_req, dtype=torch.int32, device="cuda")
    weight2 = torch.zeros_like(weight)
    for layer in range(NL):
        pool.evict(layer, weight[layer], dev(prompts), dev(table), keep, 4, 16, dev(table2), kept, n_kept, weight2[layer])
        k, n, w = kept.cpu().numpy(), n_kept.cpu().tolist(), weight[layer].cpu().numpy()
        for i in range(n_req):
            assert n[i] == min(keep, prompts[i])
            for h in range(hk):
                assert np.array_equal(k[i, h, :n[i]], pool_kept(w[i, h], prompts[i], keep, 4, 16))
            hist[layer][i] = [np.stack([x[k[i, h, :n[i]], h] for h in range(hk)], 1) for x in hist[layer][i]]
    want_w = weight2.double().cpu().numpy().copy()
    for t in range(1, n_dec + 1):
        for layer in range(NL):
            step(layer, [x + t for x in n], [1] * n_req, table2, weight2[layer], want_w[layer])
    assert (np.abs(weight2.cpu().numpy() - want_w) <= tol * np.abs(want_w) + 2e-6).all()
    # a shared prefix of 4 blocks in layer 0, and drafts of each request behind it
    pk, pv = rows(64, hk), rows(64, hk)
    pool.append(0, pk.cuda(), pv.cuda(), dev([0, 64]), dev([64]), dev(pre_table))
    lens, cu = [x + n_dec for x in n], [0, 3, 6, 9]
    q = rows(9, hq)
    out, lse = torch.empty((9, hq, d), dtype=torch.bfloat16, device="cuda"), torch.empty((9, hq), device="cuda")
    pool.prefix_attn(0, q.cuda(), dev(cu), dev(lens), dev(table2), dev([0, 2]), dev([64]), dev(pre_table), out, lse=lse)
    for i in range(n_req):
        p = dict(prefix_k=held(pk, ks), prefix_v=held(pv, vs)) if i < 2 else {}
        ref, ref_lse, mag, _ = pool_attend(q[cu[i]:cu[i + 1]].double().numpy(), *hist[0][i], scale, **p)
        check_out(out[cu[i]:cu[i + 1]].double().cpu().numpy(), lse[cu[i]:cu[i + 1]].cpu().numpy(), ref, ref_lse, mag, d, f"behind a prefix: {i}")
    assert pool.poll_error() == 0

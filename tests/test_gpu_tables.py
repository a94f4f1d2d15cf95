"""Block tables, slot maps and positions built on the device, against lists and loops; whole numbers are equal.  And a serving run of
the operators between a projection and a pool together: tables, rotation, append, attention, drafts taken back, eviction, new positions."""
import numpy as np
import pytest
import torch

import sparse_kv_cache_decode_gb300 as K
from oracle import TableOracle, pool_attend, rope_freqs, rope_rows
from pool_harness import check_out

pytestmark = pytest.mark.gpu
CAPACITY, BAD_INDEX = 3, 7


def i32(x):
    return torch.tensor(np.asarray(x, np.int64), dtype=torch.int64).to(torch.int32).cuda()


class Tables:
    """A BlockTables beside the oracle; the ring starts somewhere in the middle, in random order."""
    def __init__(self, seed, n_req, n_slots, bs, max_ctx, max_tokens=4096, ring=None):
        r = self.rng = np.random.default_rng(seed)
        k = torch.zeros((1, n_slots, 1, bs, 64), dtype=torch.bfloat16, device="cuda")
        self.pool = K.Pool(K.make_pool_config(1, n_slots, 1, 1, 64, bs, max_ctx, n_req, max_tokens), k, torch.zeros_like(k))
        order, head = r.permutation(n_slots), int(r.integers(n_slots))
        self.t = K.BlockTables(self.pool, torch.full((n_req, self.pool.nb_max), -1, dtype=torch.int32, device="cuda"), i32([0] * n_req),
                               i32(np.roll(order, head)), i32([head, n_slots, 0]))
        self.o = TableOracle(n_slots, n_req, bs, free=order.tolist())
        self.n_req, self.n_slots, self.bs, self.max_ctx = n_req, n_slots, bs, max_ctx

    def check(self):
        held, table = self.t.n_held.cpu().numpy(), self.t.block2slot.cpu().numpy()
        ring, (head, n, short) = self.t.ring.cpu().numpy(), self.t.ring_state.tolist()
        assert held.tolist() == [len(r) for r in self.o.rows]
        for r, row in enumerate(self.o.rows):
            assert table[r, :len(row)].tolist() == row, r
        assert n == len(self.o.free) and short == self.o.short and 0 <= head < self.n_slots
        assert ring[(head + np.arange(n)) % self.n_slots].tolist() == list(self.o.free)

    def step(self, ctx, q=None, delta=None, pad=0, places=False):
        """One call, checked.  q: new tokens of each request."""
        ok = self.o.reserve(ctx)
        if q is None:
            self.t.reserve(i32(ctx))
        else:
            cu = np.concatenate([[0], np.cumsum(q)])
            n = int(cu[-1]) + pad
            place = torch.full((n,), 99, dtype=torch.int64, device="cuda")
            pos = torch.full((n,), 99, dtype=torch.int32, device="cuda")
            self.t.reserve(i32(ctx), i32(cu), place, pos, None if delta is None else i32(delta))
            want = self.o.places(ctx, cu.tolist(), n, delta)
            assert place.tolist() == want[0] and pos.tolist() == want[1]
            if places and ok:
                place.fill_(99), pos.fill_(99)
                self.pool.places(i32(cu), i32(ctx), self.t.block2slot, place, pos, None if delta is None else i32(delta))
                assert place.tolist() == want[0] and pos.tolist() == want[1]
        assert self.pool.poll_error() == (0 if ok else CAPACITY)
        self.check()
        return ok


@pytest.mark.parametrize("n_req,bs,max_ctx", [(1, 16, 1), (1, 128, 5000), (3, 16, 50), (33, 32, 700), (513, 16, 300), (2048, 64, 2000)])
def test_growing_and_shrinking(n_req, bs, max_ctx):
    nb = -(-max_ctx // bs)
    t = Tables(n_req, n_req, max(2, n_req * nb * 2 // 3) + 1, bs, max_ctx, max_tokens=1 << 16)
    r = t.rng
    ctx = np.zeros(n_req, int)
    served = 0
    for step in range(8):
        new = ctx.copy()
        done = r.random(n_req) < 0.25
        new[done] = 0
        more = r.random(n_req) < 0.5
        new[more] = r.integers(0, max_ctx + 1, int(more.sum()))
        q = np.minimum(np.minimum(np.maximum(new - ctx, 0), r.integers(0, 40, n_req)) + (r.random(n_req) < 0.2), 30)
        if t.step(new.tolist(), q.tolist() if step % 3 else None, r.integers(-5, 5, n_req).tolist() if step % 2 else None, pad=step, places=True):
            ctx = new
            served += 1
    t.step([0] * n_req)
    assert sorted(t.o.free) == list(range(t.n_slots)) and served


def test_blocks_given_back_are_taken_in_the_same_call():
    t = Tables(1, 4, 10, 16, 160)
    t.step([160, 0, 0, 0])                                   # everything
    t.step([0, 70, 0, 90], [0, 70, 0, 3])                    # handed over
    t.step([33, 16, 64, 17], [33, 0, 64, 17], pad=3)
    t.step([16, 80, 64, 0], [1, 70, 1, 1])


def test_a_ring_that_runs_short_changes_nothing():
    t = Tables(2, 3, 8, 16, 200)
    assert t.step([60, 17, 0], [60, 17, 0])
    assert not t.step([60, 18, 50], [1, 1, 50], pad=2)       # two lacking; the others' places are there
    assert t.o.short == 2
    assert not t.step([200, 200, 200])
    assert t.step([60, 18, 32], [0, 1, 32])


def test_whole_prompts_at_once():
    """Many CTAs: every block of the pool in one call, one row of them all, and all back."""
    t = Tables(3, 40, 20000, 16, 16000, max_tokens=1 << 19)
    lens = t.rng.integers(0, 16000, 40).tolist()
    while sum(-(-n // 16) for n in lens) > 20000:
        lens[int(np.argmax(lens))] //= 2
    t.step(lens, lens, pad=5, places=True)
    back = [0 if i % 3 else n // 2 for i, n in enumerate(lens)]
    t.step(back)
    t.step([n + 100 for n in back], [100] * 40)
    t.step([0] * 40)
    t2 = Tables(4, 1, 1000, 16, 16000, max_tokens=1 << 14)
    t2.step([16000], [16000])
    t2.step([1], [1])


@pytest.mark.parametrize("bad", ["length", "negative", "held", "held negative"])
def test_a_bad_request_keeps_its_blocks(bad):
    t = Tables(5, 3, 12, 16, 64)
    t.step([20, 30, 40])
    before = t.t.block2slot.clone()
    if bad.startswith("held"):
        t.t.n_held[1] = -1 if "negative" in bad else 5
    ctx = [40, 31, 0] if bad.startswith("held") else [40, 65 if bad == "length" else -1, 0]
    place, pos = torch.zeros(3, dtype=torch.int64, device="cuda"), i32([9, 9, 9])
    t.t.reserve(i32(ctx), i32([0, 1, 2, 3]), place, pos)
    assert t.pool.poll_error() == BAD_INDEX and t.pool.poll_error() == 0
    assert t.t.n_held.tolist()[0] == 3 and t.t.n_held.tolist()[2] == 0
    assert torch.equal(t.t.block2slot[1], before[1])
    assert place[1:].tolist() == [-1, -1] and place[0] >= 0 and pos.tolist() == [39, 0, -1]


@pytest.mark.parametrize("state", [[-1, 5, 0], [12, 5, 0], [0, -1, 0], [0, 13, 0], [0, 9, 0]])
def test_a_ring_that_cannot_be_is_reported(state):
    """The last: more free slots than there can be beside those a request gives back."""
    t = Tables(6, 2, 12, 16, 96)
    t.step([70, 0])
    t.t.ring_state.copy_(i32(state))
    kept = [x.clone() for x in (t.t.block2slot, t.t.n_held, t.t.ring, t.t.ring_state)]
    t.t.reserve(i32([0, 33]))
    assert t.pool.poll_error() == BAD_INDEX
    assert all(torch.equal(a, b) for a, b in zip(kept, (t.t.block2slot, t.t.n_held, t.t.ring, t.t.ring_state)))


def test_bad_offsets_and_slots():
    t = Tables(7, 3, 12, 16, 64)
    t.step([20, 30, 40])
    place, pos = torch.full((6,), 99, dtype=torch.int64, device="cuda"), i32([99] * 6)
    for cu in ([0, 4, 2, 6], [0, 2, 4, 7], [-1, 2, 4, 6]):
        t.pool.places(i32(cu), i32([20, 30, 40]), t.t.block2slot, place, pos)
        assert t.pool.poll_error() == BAD_INDEX and ((place >= -1) & (place < 12 * 16)).all()
    table = t.t.block2slot.clone()
    table[1, 1], table[2, 2] = 12, -1
    t.pool.places(i32([0, 2, 4, 6]), i32([20, 30, 40]), table, place, pos)
    assert t.pool.poll_error() == BAD_INDEX
    want = t.o.places([20, 30, 40], [0, 2, 4, 6], 6)
    assert place.tolist() == want[0][:2] + [-1] * 4 and pos.tolist() == want[1]
    place.fill_(99)
    t.pool.places(i32([2, 2, 4, 4]), i32([0, 2, 40]), t.t.block2slot, place)             # tokens of nobody, a place without a context
    assert place.tolist() == [-1, -1] + [int(t.t.block2slot[1, 0]) * 16 + i for i in range(2)] + [-1, -1] and t.pool.poll_error() == 0


def test_tokens_of_no_batch():
    """No requests at all: every token is nobody's."""
    t = Tables(12, 2, 4, 16, 32, max_tokens=8)
    none = torch.zeros(0, dtype=torch.int32, device="cuda")
    place, pos = torch.full((7,), 99, dtype=torch.int64, device="cuda"), i32([99] * 7)
    t.pool.places(i32([0]), none, t.t.block2slot[:0], place, pos)
    assert place.tolist() == [-1] * 7 and pos.tolist() == [0] * 7
    empty = K.BlockTables(t.pool, t.t.block2slot[:0], none, t.t.ring, t.t.ring_state)
    place.fill_(99)
    empty.reserve(none, i32([0]), place, pos)
    empty.reserve(none)
    assert place.tolist() == [-1] * 7 and t.pool.poll_error() == 0
    t.check()


def test_refusals():
    t = Tables(8, 2, 4, 16, 32, max_tokens=4)
    place = torch.zeros(5, dtype=torch.int64, device="cuda")
    with pytest.raises(K.KvsError):
        t.t.reserve(i32([1, 1]), i32([0, 1, 2]), place)                                     # more tokens than configured
    with pytest.raises(K.KvsError):
        t.pool.places(i32([0, 1, 2]), i32([1, 1]), t.t.block2slot, place)
    with pytest.raises(K.KvsError):
        t.t.reserve(t.t.n_held)                                                             # what it reads and what it writes
    with pytest.raises(ValueError):
        t.t.reserve(i32([1, 1]).cpu())
    t.t.reserve(i32([1, 1]), i32([0, 0, 0]), place[:0])
    assert t.pool.poll_error() == 0 and t.t.n_held.tolist() == [1, 1]
    t.pool.close()
    with pytest.raises(ValueError):
        t.t.reserve(i32([1, 1]))


def test_captured_and_replayed():
    """A graph of one step; lengths change between its replays, on another stream than the one of the capture."""
    t = Tables(9, 5, 64, 16, 200)
    ctx, cu = i32([0] * 5), i32([0, 1, 2, 3, 4, 5])
    place, pos = torch.zeros(6, dtype=torch.int64, device="cuda"), i32([0] * 6)
    t.t.reserve(ctx, cu, place, pos)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ctx.add_(1)
        t.t.reserve(ctx, cu, place, pos)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    n = [0] * 5
    with torch.cuda.stream(s):
        for i in range(40):
            if i == 20:
                ctx[2] = 0
                n[2] = 0
            g.replay()
            n = [x + 1 for x in n]
            assert t.o.reserve(n)
            assert place.tolist() == t.o.places(n, [0, 1, 2, 3, 4, 5], 6)[0]
    torch.cuda.synchronize()
    t.check()
    assert t.pool.poll_error() == 0


def test_two_pools_at_once():
    """Large calls of two pools (many CTAs, each pool's own workspace) on two streams, in graphs replayed beside each other."""
    sets = [Tables(60 + i, 300, 40000, 16, 4000, max_tokens=1 << 19) for i in range(2)]
    r = np.random.default_rng(3)
    lens = [r.integers(0, 2000, 300).tolist() for _ in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    bufs, graphs = [], []
    for t, n in zip(sets, lens):
        cu = i32(np.concatenate([[0], np.cumsum(n)]))
        bufs.append((i32(n), cu, torch.zeros(sum(n), dtype=torch.int64, device="cuda"), i32([0] * sum(n)), i32([0] * 300)))
    torch.cuda.synchronize()
    for t, b, s in zip(sets, bufs, streams):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            t.t.reserve(b[0], b[1], b[2], b[3])
            t.t.reserve(b[4])
            t.t.reserve(b[0], b[1], b[2], b[3])
        graphs.append(g)
    for _ in range(3):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for t, n, b in zip(sets, lens, bufs):
            assert t.o.reserve(n) and t.o.reserve([0] * 300) and t.o.reserve(n)
            t.check()
            assert b[2].tolist() == t.o.places(n, b[1].tolist(), sum(n))[0] and t.pool.poll_error() == 0
            t.o.reserve([0] * 300)
            t.t.reserve(b[4])
            t.check()


# ------------------------------------------------------------------ together
@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_serving_run(kv):
    """Prompts, tokens, drafts of which some are refused, a request that ends and one that starts, an eviction and tokens after it."""
    r = np.random.default_rng(11)
    hq, hk, d, bs, n_req, keep, theta = 8, 2, 64, 16, 3, 48, 1e4
    scales = (0.03, 0.02) if kv == "fp8" else (1.0, 1.0)
    n_slots, max_ctx = 40, 320
    kind = torch.float8_e4m3fn if kv == "fp8" else torch.bfloat16
    kp, vp = (torch.full((1, n_slots, hk, bs, d), float("nan"), device="cuda").to(kind) for _ in range(2))
    pool = K.Pool(K.make_pool_config(1, n_slots, hq, hk, d, bs, max_ctx, n_req, 512, kv_dtype=kv, k_scale=scales[0], v_scale=scales[1]), kp, vp)
    rope = K.Rope(K.make_rope_config(d, theta=theta))
    freqs = rope_freqs(d, theta)
    tables, spare = K.BlockTables.empty(pool, n_req), None
    weight = torch.zeros((n_req, hk, max_ctx), device="cuda")
    wq, wk = (torch.from_numpy((1 + 0.2 * r.standard_normal(d)).astype(np.float32)).cuda() for _ in range(2))
    rows = [[] for _ in range(n_req)]               # fp64 (k before rotation, v) of every token, and the position it was rotated for

    def cached(side, req, n, scale):
        slots = tables.block2slot[req, :-(-n // bs)].long()
        x = side[0][slots].float().double().transpose(1, 2).reshape(-1, hk, d)[:n]
        return (x * scale).cpu().numpy()

    def step(ctx, q_len):
        cu = np.concatenate([[0], np.cumsum(q_len)])
        n = int(cu[-1])
        x = torch.from_numpy(r.standard_normal((n, hq + 2 * hk, d)).astype(np.float32)).to(torch.bfloat16).cuda()
        place, pos = torch.empty(n, dtype=torch.int64, device="cuda"), torch.empty(n, dtype=torch.int32, device="cuda")
        d_ctx, d_cu, out = i32(ctx), i32(cu), torch.zeros((n, hq, d), dtype=torch.bfloat16, device="cuda")
        lse = torch.zeros((n, hq), device="cuda")
        k_in = x[:, hq:hq + hk].clone()
        tables.reserve(d_ctx, d_cu, place, pos)
        pool.rotate_append(0, rope, x[:, :hq], x[:, hq:hq + hk], x[:, hq + hk:], pos, place, x[:, :hq], q_norm=wq, k_norm=wk)
        pool.attn(0, x[:, :hq], d_cu, d_ctx, tables.block2slot, out, lse=lse, weight=weight)
        assert pool.poll_error() == 0
        want = np.concatenate([np.arange(c - m, c) for c, m in zip(ctx, q_len)])
        assert pos.tolist() == want.tolist()
        normed, _ = rope_rows(k_in.double().cpu().numpy(), want[None], freqs * 0, weight=wk.double().cpu().numpy(), eps=1e-6)
        for i in range(n_req):
            a, b = cu[i], cu[i + 1]
            rows[i] = rows[i][:ctx[i] - q_len[i]] + [normed[t] for t in range(a, b)]
            k, v = cached(kp, i, ctx[i], scales[0]), cached(vp, i, ctx[i], scales[1])
            ref, ref_lse, mag, _ = pool_attend(x[a:b, :hq].double().cpu().numpy(), k, v, float(np.float32(1 / np.sqrt(d))))
            check_out(out[a:b].double().cpu().numpy(), lse[a:b].cpu().numpy(), ref, ref_lse, mag, d, f"request {i}")
            for h in range(hk if ctx[i] else 0):    # the keys in the pool: normed, at their positions
                y, m = rope_rows(np.array(history(i, h))[:, None], np.arange(ctx[i])[None], freqs)
                # One rounding, and a second where the key was moved.  A rounding is off by half a step of each element, so a pair is off by
                # half a step of its length (below m) before it turns, and by as much of its new elements after it, which are longer by
                # 1 + 2^-4 at most.  Below E4M3's normal range both elements are off by 2^-10 (turned: sqrt(2) of it), then once more.
                half = 2.0 ** -4 if kv == "fp8" else 2.0 ** -8
                tol = 2.1 * half * m[:, 0] + 3 * 2.0 ** -10 * scales[0] if moved[i] else half * np.abs(y[:, 0]) + 2.0 ** -10 * scales[0]
                tol = tol + 2.0 ** -17 * m[:, 0]
                assert (np.abs(k[:, h] - y[:, 0]) <= tol).all(), (i, h)
        return ctx

    moved = [None] * n_req
    kept_rows = [None] * n_req

    def history(i, h):
        if not moved[i]:
            return [x[h] for x in rows[i]]
        return [kept_rows[i][t][h] for t in moved[i][h]] + [x[h] for x in rows[i][len(moved[i][h]):]]

    ctx = step([100, 37, 0], [100, 37, 0])                  # prompts
    ctx = step([c + 1 for c in ctx[:2]] + [1], [1, 1, 1])
    ctx = step([c + 5 for c in ctx], [5, 5, 5])             # a token and four drafts
    ctx = [ctx[0] - 3, ctx[1] - 4, ctx[2]]                  # some of which are refused
    tables.reserve(i32(ctx))
    rows[:] = [x[:n] for x, n in zip(rows, ctx)]
    ctx = step([ctx[0] + 2, 60, ctx[2] + 2], [2, 60, 2])    # request 1 gives way to a new prompt
    assert tables.n_held.tolist() == [-(-n // bs) for n in ctx]
    # request 0's cache is cut down to `keep` tokens, in blocks of its own
    spare = K.BlockTables.empty(pool, n_req, like=tables)
    spare.reserve(i32([keep, min(keep, ctx[1]), min(keep, ctx[2])]))
    kept, n_kept = torch.full((n_req, hk, keep), -1, dtype=torch.int32, device="cuda"), i32([0] * n_req)
    weight_out = torch.zeros_like(weight)
    pool.evict(0, weight, i32(ctx), tables.block2slot, keep, 4, 8, spare.block2slot, kept, n_kept, weight_out)
    pool.reposition(0, rope, kept, n_kept, spare.block2slot)
    tables.reserve(i32([0] * n_req))
    assert pool.poll_error() == 0
    tables, weight = spare, weight_out
    ctx = n_kept.tolist()
    assert ctx == [keep, keep, min(keep, 8)]
    for i in range(n_req):
        moved[i] = [kept[i, h, :ctx[i]].tolist() for h in range(hk)]
        kept_rows[i] = rows[i]
        rows[i] = [None] * ctx[i]
    ctx = step([c + 3 for c in ctx], [3, 3, 3])             # goes on behind the kept tokens
    free = set((tables.ring.cpu().numpy()[(tables.ring_state[0].item() + np.arange(tables.ring_state[1].item())) % n_slots]).tolist())
    owned = [s for i in range(n_req) for s in tables.block2slot[i, :tables.n_held[i]].tolist()]
    assert len(free) + len(owned) == n_slots and free.isdisjoint(owned) and len(set(owned)) == len(owned)

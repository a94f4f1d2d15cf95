"""What becomes of a cache that is cut back again and again: keys that keep their old positions (later tokens' positions run on through
pos_delta) stay as they were stored, keys that are moved each time are rounded each time."""
import numpy as np
import pytest
import torch

import sparse_kv_cache_decode_gb300 as K
from oracle import pool_attend, rope_freqs, rope_rows
from pool_harness import check_out

pytestmark = pytest.mark.gpu
KIND = {"bf16": torch.bfloat16, "fp8": torch.float8_e4m3fn}


def i32(x):
    return torch.tensor(np.asarray(x, np.int64), dtype=torch.int64).to(torch.int32).cuda()


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("axes", [1, 3])
def test_old_positions_go_on(kv, axes):
    """Prompts and six rounds of new tokens, each followed by an eviction to `keep`.  A token's position is its number since the start, for
    good; a key's bits are those of its append."""
    r = np.random.default_rng(3)
    hq, hk, d, bs, keep, n_req, theta = 8, 2, 64, 16, 40, 2, 1e4
    scales = (0.03, 0.02) if kv == "fp8" else (1.0, 1.0)
    n_slots, max_ctx = 40, 160
    kp, vp = (torch.zeros((1, n_slots, hk, bs, d), device="cuda").to(KIND[kv]) for _ in range(2))
    pool = K.Pool(K.make_pool_config(1, n_slots, hq, hk, d, bs, max_ctx, n_req, 256, kv_dtype=kv, k_scale=scales[0], v_scale=scales[1]), kp, vp)
    pair_axes = None if axes == 1 else K.rope_axes([12, 10, 10])
    rope, freqs = K.Rope(K.make_rope_config(d, theta=theta, axes=pair_axes)), rope_freqs(d, theta)
    tables = K.BlockTables.empty(pool, n_req)
    weight = torch.zeros((n_req, hk, max_ctx), device="cuda")
    delta = torch.zeros(n_req, dtype=torch.int32, device="cuda")
    ctx = [0] * n_req
    seen = [0] * n_req                                   # tokens since the start
    stored = [[] for _ in range(n_req)]                  # per token: [hk][d] patterns of its key
    cached = [[[] for _ in range(hk)] for _ in range(n_req)]      # which tokens stand in the cache

    def rows(side, i, n):
        x = side[0][tables.block2slot[i, :-(-n // bs)].long()]
        return x.view(torch.uint8 if kv == "fp8" else torch.int16).transpose(1, 2).reshape(-1, hk, d)[:n]

    def values(x, scale):
        return x.view(KIND[kv]).double().cpu().numpy() * scale

    for q_len in ([97, 60], [16, 1], [5, 33], [16, 16], [1, 1], [16, 40], [30, 2]):
        ctx = [c + m for c, m in zip(ctx, q_len)]
        cu, n = np.concatenate([[0], np.cumsum(q_len)]), sum(q_len)
        x = torch.from_numpy(r.standard_normal((n, hq + 2 * hk, d)).astype(np.float32)).to(torch.bfloat16).cuda()
        raw_k = x[:, hq:hq + hk].double().cpu().numpy()
        place, pos = torch.empty(n, dtype=torch.int64, device="cuda"), torch.empty(n, dtype=torch.int32, device="cuda")
        d_ctx, d_cu, out, lse = i32(ctx), i32(cu), torch.zeros((n, hq, d), dtype=torch.bfloat16, device="cuda"), torch.zeros((n, hq), device="cuda")
        tables.reserve(d_ctx, d_cu, place, pos, pos_delta=delta)
        want = np.concatenate([np.arange(s, s + m) for s, m in zip(seen, q_len)])
        assert pos.tolist() == want.tolist()
        pool.rotate_append(0, rope, x[:, :hq], x[:, hq:hq + hk], x[:, hq + hk:], pos, place, x[:, :hq])
        pool.attn(0, x[:, :hq], d_cu, d_ctx, tables.block2slot, out, lse=lse, weight=weight)
        assert pool.poll_error() == 0
        y, mag = rope_rows(raw_k, np.broadcast_to(want, (axes, n)), freqs, pair_axes)
        for i in range(n_req):
            a, b, old = cu[i], cu[i + 1], ctx[i] - q_len[i]
            k = rows(kp, i, ctx[i])
            for j in range(old):                         # the cached ones: as they were appended
                for h in range(hk):
                    assert torch.equal(k[j, h], stored[i][cached[i][h][j]][h]), (i, j, h)
            # the new ones: one rounding of the exact values, half a step (2^-4 and 2^-10 of a code's unit, or 2^-8), and the angle's 2^-18
            tol = (2.0 ** -4 * np.abs(y[a:b]) + 2.0 ** -10 * scales[0] if kv == "fp8" else 2.0 ** -8 * np.abs(y[a:b])) + 2.0 ** -18 * mag[a:b]
            assert (np.abs(values(k[old:], scales[0]) - y[a:b]) <= tol).all()
            stored[i] += list(k[old:].clone())
            for h in range(hk):
                cached[i][h] += range(seen[i], seen[i] + q_len[i])
            seen[i] += q_len[i]
            ref = pool_attend(x[a:b, :hq].double().cpu().numpy(), values(k, scales[0]), values(rows(vp, i, ctx[i]), scales[1]), float(np.float32(1 / np.sqrt(d))))
            check_out(out[a:b].double().cpu().numpy(), lse[a:b].cpu().numpy(), *ref[:3], d, f"request {i}")
        spare = K.BlockTables.empty(pool, n_req, like=tables)
        spare.reserve(i32([min(keep, c) for c in ctx]))
        kept, n_kept, w_out = torch.full((n_req, hk, keep), -1, dtype=torch.int32, device="cuda"), i32([0] * n_req), torch.zeros_like(weight)
        pool.evict(0, weight, d_ctx, tables.block2slot, keep, 4, 8, spare.block2slot, kept, n_kept, w_out)
        tables.reserve(i32([0] * n_req))
        delta += d_ctx - n_kept                          # positions run on
        tables, weight, ctx = spare, w_out, n_kept.tolist()
        for i in range(n_req):
            for h in range(hk):
                cached[i][h] = [cached[i][h][j] for j in kept[i, h, :ctx[i]].tolist()]
        assert pool.poll_error() == 0 and ctx == [min(keep, s) for s in seen]


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("moves,by", [(1, 64), (5, 64), (12, 17)])
def test_each_move_rounds_once_more(kv, moves, by):
    """An error e of a pair of length z keeps its length when the pair turns.  A move then rounds both elements by half a step h of each at
    most, h (z + e) of the pair, or by sqrt(2) * u below the type's normal range (bf16's: none here), and turns it with an error of 2^-18 of |a| + |b|, 2^-17 of its length.
    So e + z grows by 1 + h + 2^-17 a move."""
    r = np.random.default_rng(moves)
    hk, d, bs, n = 2, 128, 16, 300
    nb = -(-n // bs)
    kp = torch.from_numpy(r.standard_normal((1, nb, hk, bs, d)).astype(np.float32)).cuda().mul(30.0 if kv == "fp8" else 1.0).clamp(-300, 300).to(KIND[kv])
    pool = K.Pool(K.make_pool_config(1, nb, hk, hk, d, bs, nb * bs, 1, 8, kv_dtype=kv), kp, torch.zeros((), device="cuda").to(KIND[kv]).expand(kp.shape).contiguous())
    table, n_kept = torch.arange(nb, dtype=torch.int32, device="cuda").view(1, -1), i32([n])
    kept = (torch.arange(n, dtype=torch.int32, device="cuda") + by).expand(1, hk, n).contiguous()
    rows = lambda: kp[0].float().double().transpose(1, 2).reshape(-1, hk, d)[:n].cpu().numpy()  # noqa: E731
    before = rows()
    rope, freqs = K.Rope(K.make_rope_config(d, theta=5e5)), rope_freqs(d, 5e5)
    for _ in range(moves):
        pool.reposition(0, rope, kept, n_kept, table)
    assert pool.poll_error() == 0
    y, _ = rope_rows(before, np.full((1, n), -by * moves), freqs)
    pairs = lambda x: np.hypot(x[..., :d // 2], x[..., d // 2:])  # noqa: E731
    h, u = (2.0 ** -4, 2.0 ** -10) if kv == "fp8" else (2.0 ** -8, 0.0)
    grow = (1 + h + 2.0 ** -17) ** moves
    bound = pairs(before) * (grow - 1) + moves * np.sqrt(2) * u * grow
    bound = np.where(pairs(before) * grow < 440, bound, np.inf)      # (past the largest code they saturate)
    assert (pairs(rows() - y) <= bound + 1e-12).all()

"""Batches with free places: a request without a context, or with more query tokens than its context holds, goes through
append and attention like any other.  Its tokens at positions below 0 have no place and no keys, and that is no error."""
import pytest
import torch

import sparse_kv_cache_decode_gb300 as K
from oracle import pool_attend
from pool_harness import PoolCase, check_out

pytestmark = pytest.mark.gpu

BATCHES = [  # contexts, query tokens
    ([0], [1]), ([40, 0, 17], [1, 1, 1]), ([0, 33, 0, 200], [1, 1, 2, 1]), ([5, 64, 0], [9, 30, 40]), ([0, 300], [1, 150]),
]


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("i", range(len(BATCHES)))
def test_append_and_attention_with_free_places(i, kv):
    ctx, m = BATCHES[i]
    hq, hk, d, bs = 8, 2, 128, 16
    c = PoolCase(20 + i, ctx, m, hq, hk, d, bs, kv, pad_tokens=1).cuda()
    g = torch.Generator().manual_seed(i)
    new = [torch.randn((c.n_tok, hk, d), generator=g).to(torch.bfloat16) for _ in range(2)]
    want = [c.dk.clone(), c.dv.clone()]
    for x in range(2):
        if kv == "bf16":
            codes, held = new[x].cuda(), new[x].double().numpy()
        else:
            codes = torch.empty(new[x].shape, dtype=torch.uint8, device="cuda")
            K.quantize_e4m3(new[x].cuda(), codes, c.scales[x])
            held = codes.cpu().view(torch.float8_e4m3fn).double().numpy() * c.scales[x]
        for r, n in enumerate(ctx):
            for j in range(m[r]):
                p = n - m[r] + j
                if p >= 0:
                    want[x][0, c.table[r, p // bs], :, p % bs] = codes[c.cu[r] + j]
                    c.rows[r][x][p] = held[c.cu[r] + j]
    c.pool.append(0, new[0].cuda(), new[1].cuda(), c.d_cu, c.d_ctx, c.d_table)
    assert c.pool.poll_error() == 0
    for got, ref in zip((c.dk, c.dv), want):
        assert torch.equal(got.view(torch.uint8), ref.view(torch.uint8))
    out, lse = c.out()
    c.pool.attn(0, c.d_q, c.d_cu, c.d_ctx, c.d_table, out, lse=lse)
    assert c.pool.poll_error() == 0
    got, lse = out.double().cpu().numpy(), lse.cpu().numpy()
    for r in range(len(ctx)):
        ref, ref_lse, mag, _ = pool_attend(c.query(r), *c.rows[r], c.softmax_scale)
        a, b = c.cu[r], c.cu[r + 1]
        check_out(got[a:b], lse[a:b], ref, ref_lse, mag, d, f"request {r}")
    assert (got[c.cu[-1]:] == 7.0).all()


def test_append_still_reports_bad_slots_and_lengths():
    c = PoolCase(30, [40, 0], [2, 1], 8, 2, 64, 16).cuda()
    new = torch.ones((c.n_tok, 2, 64), dtype=torch.bfloat16, device="cuda")
    table = c.d_table.clone()
    table[0, 2] = -1
    c.pool.append(0, new, new.clone(), c.d_cu, c.d_ctx, table)
    assert c.pool.poll_error() == 7
    ctx = c.d_ctx.clone()
    ctx[1] = -1
    c.pool.append(0, new, new.clone(), c.d_cu, ctx, c.d_table)
    assert c.pool.poll_error() == 7

"""Rows of kvs_rotate as the sparse step's queries, drafts and appended keys: the two calls on one stream, layer after layer.  The rotated rows
are held against fp64, and the step on them against the oracle on the same rows (near-tied blocks may be ordered otherwise,
as in the step's own tests)."""
import numpy as np
import pytest

import workload as W
from kvs_harness import GpuCase, compare_step
from oracle import rope_freqs, rope_rows

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
import sparse_kv_cache_decode_gb300 as K  # noqa: E402

CASES = [
    (W.TINY_APPEND.with_(name="rope_append", n_req=2, n_layer=2), [4096, 1001], dict(), True),
    (W.TINY_APPEND.with_(name="rope_append_fp8", n_req=2, kv_dtype="fp8", v_scale=0.5), [4096, 700], dict(rot=96, adjacent=True), True),
    (W.TINY_LOOKAHEAD.with_(name="rope_lookahead", n_req=2), [4096, 2050], dict(adjacent=True), False),
    (W.TINY_MLA.with_(name="rope_latent", n_layer=2), [4096], dict(part=64, adjacent=True), False),      # the last 64 dims of rows of 576
]


@pytest.mark.parametrize("w,lens,opt,norm", CASES, ids=[c[0].name for c in CASES])
@pytest.mark.parametrize("copy_stream", [False, True])
def test_rotated_rows_in_the_step(w, lens, opt, norm, copy_stream):
    g = GpuCase(w, lens, copy_stream=copy_stream)
    o = g.oracle()
    d, first = opt.get("part", w.d_k), w.d_k - opt.get("part", w.d_k)
    rot, adjacent = opt.get("rot", d), opt.get("adjacent", False)
    rope, freqs = K.Rope(K.make_rope_config(d, rot, theta=5e5, adjacent=adjacent)), rope_freqs(rot, 5e5)
    r = np.random.default_rng(7)
    wq, wk = ((1 + 0.2 * r.standard_normal(d)).astype(np.float32) if norm else None for _ in range(2))
    wq_d, wk_d = (None if x is None else torch.from_numpy(x).cuda() for x in (wq, wk))
    up = lambda x: torch.from_numpy(x.view(np.int16).copy()).cuda().view(torch.bfloat16)  # noqa: E731
    down = lambda t: t.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)  # noqa: E731

    def check(before, after, pos, weight):
        """[n][heads][d_k] each.  Tolerance: one rounding to bf16 (2^-8 of the value), and 2^-18 of a pair's |a| + |b| (angles, cosines, norm)."""
        x = before.double().cpu().numpy()
        y, mag = rope_rows(x[..., first:], pos[None], freqs, adjacent=adjacent, weight=weight, eps=1e-6)
        got = after.double().cpu().numpy()
        assert np.array_equal(got[..., :first], x[..., :first])
        assert (np.abs(got[..., first:] - y) <= 2.0 ** -8 * np.abs(y) + 2.0 ** -18 * mag).all()

    frozen = set()
    for t in range(min(w.steps, 8)):
        q, dr, nk, nv = g.step_inputs(t)
        qs, ds, ks, vs = (None if x is None else [up(x[l]) for l in range(w.n_layer)] for x in (q, dr, nk, nv))
        ks = ks or [None] * w.n_layer
        raw = [[x.clone() for x in qs], None if ds is None else [x.clone() for x in ds], [None if x is None else x.clone() for x in ks]]
        if w.append:
            g.ctx.advance_ctx(g.ctx_len)
        pos = (g.ctx_len - 1).to(torch.int32)
        for l in range(w.n_layer):
            x, k = qs[l][..., first:], None if ks[l] is None else ks[l][..., first:]
            rope.rotate(x, pos, x, k, k, q_norm=wq_d, k_norm=None if k is None else wk_d)      # in place, within longer rows
            if ds is not None:
                y = ds[l].view(-1, w.n_q_head, w.d_k)[..., first:]
                rope.rotate(y, pos.repeat_interleave(w.n_draft), y, q_norm=wq_d)
            g.ctx.decode_step(l, qs[l], None if ds is None else ds[l], w.n_score_q if ds is not None else 1, g.index, g.ctx_len, g.out[l], g.stats,
                              ks[l], None if vs is None else vs[l], g.sel[l], g.nsel[l], copy_stream=g.copy_stream)
        g.ctx.join()
        torch.cuda.synchronize()
        g.t += 1
        p = pos.cpu().numpy()
        for l in range(w.n_layer):
            check(raw[0][l], qs[l], p, wq)
            if ks[l] is not None:
                check(raw[2][l], ks[l], p, wk)
            if ds is not None:
                check(raw[1][l].view(-1, w.n_q_head, w.d_k), ds[l].view(-1, w.n_q_head, w.d_k), p.repeat(w.n_draft), wq)
        q = np.stack([down(x) for x in qs])
        dr = None if ds is None else np.stack([down(x) for x in ds])
        nk = None if nk is None else np.stack([down(x) for x in ks])
        out_ref, recs = o.step(q, dr, nk, nv)
        compare_step(g, o, out_ref, recs, None, exact=False, frozen=frozen)
    assert len(frozen) <= max(1, w.n_layer * w.n_req * w.n_kv_head // 2)
    assert g.ctx.poll_error() == 0

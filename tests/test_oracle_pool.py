"""The pool oracle against closed forms, torch's attention in 64 bits and brute force."""
import numpy as np
import pytest
import torch

from oracle import pool_attend, pool_kept


def _rand(seed, m, n, hq, hk, d):
    r = np.random.default_rng(seed)
    return r.standard_normal((m, hq, d)), r.standard_normal((n, hk, d)), r.standard_normal((n, hk, d))


@pytest.mark.parametrize("m,n,window,sink,n0", [(1, 7, 0, 0, 0), (5, 9, 3, 0, 0), (9, 9, 4, 2, 0), (3, 11, 1, 1, 0), (4, 6, 0, 0, 5)])
def test_attend_equals_masked_sdpa(m, n, window, sink, n0):
    q, k, v = _rand(m * n, m, n, 6, 2, 8)
    _, k0, v0 = _rand(5, 1, n0, 1, 2, 8) if n0 else (None, None, None)
    out, lse, mag, weight = pool_attend(q, k, v, 0.3, window, sink, k0, v0)
    mask = torch.zeros((m, n0 + n), dtype=torch.bool)
    for i in range(m):
        p = n - m + i
        for t in range(n):
            mask[i, n0 + t] = t <= p and (not window or p - t < window or t < sink)
    mask[:, :n0] = True
    kk, vv = (torch.from_numpy(np.concatenate([b, a]) if n0 else a).repeat_interleave(3, 1).transpose(0, 1) for a, b in ((k, k0), (v, v0)))
    qq = torch.from_numpy(q).transpose(0, 1)
    ref = torch.nn.functional.scaled_dot_product_attention(qq, kk, vv, attn_mask=mask, scale=0.3).transpose(0, 1).numpy()
    assert np.abs(out - ref).max() < 1e-12
    s = (qq @ kk.transpose(1, 2) * 0.3).masked_fill(~mask, -np.inf)
    assert np.abs(lse.T - torch.logsumexp(s, -1).numpy()).max() < 1e-12
    w = torch.softmax(s, -1).sum(1)[:, n0:].view(2, 3, n).sum(1).T.numpy()
    assert np.abs(weight - w).max() < 1e-12
    assert (mag + 1e-12 >= np.abs(out)).all()


def test_attend_closed_forms():
    q, k, v = _rand(1, 3, 5, 2, 1, 4)
    out, lse, _, weight = pool_attend(q, k, v, 0.5, window=1)      # each row sees its own key only
    assert np.allclose(out, v[2:])
    assert np.allclose(weight[:, 0], [0, 0, 2, 2, 2])
    out, lse, _, _ = pool_attend(q, np.zeros_like(k), v, 0.5)      # equal logits: the mean
    assert np.allclose(out[2, 0], v[:, 0].mean(0)) and np.isclose(lse[2, 0], np.log(5))
    out, lse, _, weight = pool_attend(q, k[:1], v[:1], 0.5)        # two of three rows before the first key
    assert (out[:2] == 0).all() and np.isneginf(lse[:2]).all() and np.allclose(out[2], v[0]) and weight[0, 0] == 2


def test_kept_brute_force():
    r = np.random.default_rng(3)
    for _ in range(200):
        n = int(r.integers(1, 30))
        keep = int(r.integers(1, 30))
        sink = int(r.integers(0, keep + 1))
        recent = int(r.integers(0, keep - sink + 1))
        w = r.integers(0, 4, n).astype(np.float64)
        w[r.random(n) < 0.1] = np.nan
        w[r.random(n) < 0.1] = -0.0
        got = pool_kept(w, n, keep, sink, recent)
        assert got.size == min(n, keep) and (np.diff(got) > 0).all()
        if n <= keep:
            continue
        forced = {t for t in range(n) if t < sink or t >= n - recent}
        assert forced <= set(got.tolist())
        val = np.where(np.isnan(w), -np.inf, w)
        for t in range(n):
            if t not in forced:
                better = sum(1 for o in range(n) if o not in forced and (val[o] > val[t] or (val[o] == val[t] and o < t)))
                assert (t in got) == (better < keep - sink - recent)

"""Device-resident pools: attention over one request's cached tokens and the eviction rule (fp64).

Positions: the m query tokens of a request with n cached tokens stand at n - m .. n - 1.
"""
from __future__ import annotations

import numpy as np

__all__ = ["pool_attend", "pool_kept"]


def pool_attend(q, k, v, scale, window=0, n_sink=0, prefix_k=None, prefix_v=None):
    """q [m][H_q][d], k / v [n][H_kv][d] (fp64), prefix_k / prefix_v [n0][H_kv][d] seen by every row.

    Returns out [m][H_q][d], lse [m][H_q], mag [m][H_q][d] = sum_t p_t |v_t| (what a relative error of the
    weights p can move an output by) and weight [n][H_kv] (the request's own keys' summed weights)."""
    m, hq, d = q.shape
    n, hk = k.shape[:2]
    g = hq // hk
    n0 = 0 if prefix_k is None else prefix_k.shape[0]
    kk = k if n0 == 0 else np.concatenate([prefix_k, k])
    vv = v if n0 == 0 else np.concatenate([prefix_v, v])
    pos = np.arange(n - m, n)[:, None]
    t = np.arange(n)[None, :]
    seen = t <= pos
    if window:
        seen &= (pos - t < window) | (t < n_sink)
    seen = np.concatenate([np.ones((m, n0), bool), seen], axis=1)
    out = np.zeros((m, hq, d))
    mag = np.zeros((m, hq, d))
    lse = np.full((m, hq), -np.inf)
    weight = np.zeros((n, hk))
    for h in range(hq):
        s = np.where(seen, scale * (q[:, h] @ kk[:, h // g].T), -np.inf)
        top = np.max(s, axis=1, initial=-np.inf, keepdims=True)
        p = np.exp(s - np.where(np.isinf(top), 0.0, top))
        total = p.sum(axis=1, keepdims=True)
        some = total[:, 0] > 0
        p /= np.where(total > 0, total, 1.0)
        lse[some, h] = top[some, 0] + np.log(total[some, 0])
        out[:, h] = p @ vv[:, h // g]
        mag[:, h] = p @ np.abs(vv[:, h // g])
        weight[:, h // g] += p[:, n0:].sum(axis=0)
    return out, lse, mag, weight


def pool_kept(weight, n, keep, n_sink, n_recent):
    """Ascending indices of the min(keep, n) tokens of weight[:n] that are kept: the first n_sink, the last
    n_recent and of the others the largest (ties: the earlier; NaN below -inf; -0.0 == +0.0)."""
    if n <= keep:
        return np.arange(n)
    mid = np.arange(n_sink, n - n_recent)
    w = weight[mid].astype(np.float64)
    order = sorted(range(mid.size), key=lambda i: (np.isnan(w[i]), -w[i] if not np.isnan(w[i]) else 0.0, i))
    best = mid[order[:keep - n_sink - n_recent]]
    return np.sort(np.concatenate([np.arange(n_sink), best, np.arange(n - n_recent, n)]).astype(np.int64))

"""Steps of single tokens in which long requests end and others begin: many blocks change hands in a call with few tokens."""
import numpy as np
import pytest

from test_gpu_tables import Tables

import torch  # noqa: F401  (CUDA)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n_req,bs,max_ctx,n_slots", [(64, 16, 20000, 45000), (3, 128, 120000, 2000), (300, 16, 2000, 20000)])
def test_requests_that_end(n_req, bs, max_ctx, n_slots):
    t = Tables(n_req, n_req, n_slots, bs, max_ctx)
    r = t.rng
    ctx = r.integers(0, max_ctx // 2, n_req)
    while int(np.sum(-(-ctx // bs))) > n_slots * 2 // 3:
        ctx[np.argmax(ctx)] //= 2
    assert t.step(ctx.tolist())
    for i in range(6):
        new = np.minimum(ctx + 1, max_ctx)
        ends = r.random(n_req) < (0.2, 1.0, 0.5)[i % 3]
        new[ends] = 0
        if i % 2:                                       # others take the place of those that end, with their blocks
            at = np.flatnonzero(ends)
            new[at] = np.roll(ctx[at], 1)
        q = np.where(new > 0, 1, 0)
        if t.step(new.tolist(), q.tolist(), pad=i % 3, places=True):
            ctx = new
    t.step([0] * n_req, [0] * n_req, pad=2)
    assert sorted(t.o.free) == list(range(n_slots))

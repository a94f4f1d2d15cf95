"""Rows that lie between others, for any number of tokens: the same bits as rows of their own, and nothing else is written."""
import numpy as np
import pytest
import torch

import sparse_kv_cache_decode_gb300 as K

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n", [1, 2, 41, 3000])
@pytest.mark.parametrize("d", [64, 128])
def test_heads_between_others(n, d):
    r = np.random.default_rng(n + d)
    rope = K.Rope(K.make_rope_config(d))
    x = torch.from_numpy(r.standard_normal((n, 8, 3, d)).astype(np.float32)).to(torch.bfloat16).cuda()
    pos = torch.from_numpy(r.integers(0, 1 << 20, n).astype(np.int32)).cuda()
    w = [torch.from_numpy(r.standard_normal(d).astype(np.float32)).cuda() for _ in range(2)]
    q, k = x[:, :, 0].contiguous(), x[:, :, 1].contiguous()
    want_q, want_k = torch.empty_like(q), torch.empty_like(k)
    rope.rotate(q, pos, want_q, k, want_k, q_norm=w[0], k_norm=w[1])

    def check(y, **parts):
        """y: the buffer after the call; parts: what its slices are now, the others as before."""
        want = x.clone()
        for i, t in parts.items():
            want[:, :, int(i[1])] = t
        assert torch.equal(y, want)

    y = x.clone()                                       # in place
    rope.rotate(y[:, :, 0], pos, y[:, :, 0], y[:, :, 1], y[:, :, 1], q_norm=w[0], k_norm=w[1])
    check(y, p0=want_q, p1=want_k)
    y = x.clone()                                       # into the columns of v
    rope.rotate(y[:, :, 0], pos, y[:, :, 2], q_norm=w[0])
    check(y, p2=want_q)
    z = x.view(n, 24, d).clone()                        # every second head into the others
    even = z[:, ::2].contiguous()
    want = torch.empty_like(even)
    rope.rotate(even, pos, want, q_norm=w[0])
    rope.rotate(z[:, ::2], pos, z[:, 1::2], q_norm=w[0])
    assert torch.equal(z[:, ::2], even) and torch.equal(z[:, 1::2], want)
    t = torch.zeros((8, 2, n, d), dtype=torch.bfloat16, device="cuda")      # a head's tokens together, the output's behind the input's
    t[:, 0] = q.transpose(0, 1)
    rope.rotate(t[:, 0].transpose(0, 1), pos, t[:, 1].transpose(0, 1), q_norm=w[0])
    assert torch.equal(t[:, 0].transpose(0, 1), q) and torch.equal(t[:, 1].transpose(0, 1), want_q)
    for a, b in ((x[:, :, 0], x.view(n, 24, d)[:, :8]), (t[:, 0].transpose(0, 1), t.view(16, n, d)[:8].transpose(0, 1))):
        with pytest.raises(K.KvsError):
            rope.rotate(a, pos, b)

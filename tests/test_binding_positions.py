"""Position tensors that the compiled calls look at: those they do not take are left to the checks that say why (no GPU)."""
import pytest

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def K():
    from sparse_kv_cache_decode_gb300 import build as B
    B.build()
    import sparse_kv_cache_decode_gb300 as K
    return K


def test_shapes_are_no_errors(K):
    """Tensors of the CPU: the calls never get as far as the library."""
    fast = K.binding()
    rope = K.Rope(K.make_rope_config(64, axes=[0, 1] * 16))
    q, kv = torch.zeros((3, 8, 64), dtype=torch.bfloat16), torch.zeros((3, 2, 64), dtype=torch.bfloat16)
    place = torch.zeros(3, dtype=torch.int64)
    for pos in (torch.tensor(5), torch.zeros(3), torch.zeros((2, 3)), torch.zeros((2, 5))[:, 1:4], torch.zeros((3, 2)).T, torch.zeros((1, 2, 3)), torch.zeros(0),
                torch.zeros((2, 0)), torch.zeros((3, 3)), torch.zeros(4)):
        pos = pos.to(torch.int32)
        assert fast.rotate(rope.address, 64, 2, q, pos, q, None, None, None, None, 0) is None
        assert fast.rotate_append(4096, rope.address, -1, 8, 2, 64, 2, 0, q, kv, kv, pos, place, q, None, None, 0) is None


@pytest.mark.gpu
def test_rows_of_longer_rows_take_the_short_way(K):
    fast = K.binding()
    rope = K.Rope(K.make_rope_config(64, axes=[0, 1] * 16))
    q = torch.randn((3, 8, 64), device="cuda").to(torch.bfloat16)
    wide = torch.arange(20, dtype=torch.int32, device="cuda").view(2, 10)
    want, out = torch.empty_like(q), torch.empty_like(q)
    rope.rotate(q, wide[:, 4:7].contiguous(), want)
    s = torch.cuda.current_stream().cuda_stream
    assert fast.rotate(rope.address, 64, 2, q, wide[:, 4:7], out, None, None, None, None, s) == 0
    assert torch.equal(out, want)
    rope.rotate(q, wide[:1, 4:7].expand(2, 3).contiguous(), want)
    assert fast.rotate(rope.address, 64, 2, q, wide[:1, 4:7].expand(2, 3), out, None, None, None, None, s) == 0      # one row for both axes
    assert torch.equal(out, want)
    one = wide.T[4:5].T                                    # a token: any strides
    rope.rotate(q[:1], one.contiguous(), want[:1])
    rope.rotate(q[:1], one, out[:1])
    assert torch.equal(out[:1], want[:1])
    for bad in (torch.tensor(5, dtype=torch.int32, device="cuda"), wide[:, :6:2], wide[:, 4:8], wide[0, :4]):
        assert fast.rotate(rope.address, 64, 2, q, bad, out, None, None, None, None, s) is None
        with pytest.raises(ValueError, match="pos"):
            rope.rotate(q, bad, out)

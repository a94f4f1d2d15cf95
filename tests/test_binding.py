"""The compiled part of the Python binding: what it says about tensors, what it refuses to pass on (no GPU)."""
import ctypes

import pytest

torch = pytest.importorskip("torch")

BF, F32, I32 = (torch.bfloat16, torch.int16), (torch.float32,), (torch.int32,)


@pytest.fixture(scope="module")
def fast():
    from sparse_kv_cache_decode_gb300 import build as B
    B.build()
    import sparse_kv_cache_decode_gb300 as K
    return K.binding()


def test_whole(fast):
    x = torch.zeros((3, 4), dtype=torch.int16)
    assert fast.whole(x, BF, (3, 4), -1) == x.data_ptr()
    assert fast.whole(x[1:], BF, (2, 4), -1) == x.data_ptr() + 8
    assert fast.whole(torch.zeros((0, 4)), F32, (0, 4), -1) == 0
    for a in ((x, F32, (3, 4), -1), (x, BF, (3, 5), -1), (x, BF, (12,), -1), (x, BF, (3, 4, 1), -1), (x, BF, (3, 4), 0), (x.T, BF, (4, 3), -1),
              (x[:, :2], BF, (3, 2), -1), (None, BF, (3, 4), -1), ([1, 2], BF, (2,), -1), (x, list(BF), (3, 4), -1)):
        assert fast.whole(*a) is None, a
    for a in ((x, BF, (3, 4)), (x, BF, (3, 4), -1, 0)):
        with pytest.raises(TypeError):
            fast.whole(*a)
    with pytest.raises(OverflowError):
        fast.whole(x, BF, (1 << 70, 4), -1)


def test_rows(fast):
    x = torch.zeros((5, 6, 64), dtype=torch.bfloat16)
    p = x.data_ptr()
    assert fast.rows(x, BF, 6, 64, -1) == (p, 384, 64, 5, 6)
    assert fast.rows(x[:, 1:3], BF, -1, 64, -1) == (p + 128, 384, 64, 5, 2)
    assert fast.rows(x[::2, ::3, :], BF, 2, 64, -1) == (p, 768, 192, 3, 2)
    assert fast.rows(x[:, :, 32:], BF, 6, 32, -1) == (p + 64, 384, 64, 5, 6)
    assert fast.rows(x[2:3], BF, 6, 64, -1)[1:] == (384, 64, 1, 6) and fast.rows(x[:, 2:3], BF, 1, 64, -1)[1:] == (384, 64, 5, 1)
    assert fast.rows(x[:0], BF, 6, 64, -1)[1:] == (384, 64, 0, 6)
    none = torch.zeros((5, 0, 64), dtype=torch.bfloat16)            # no rows: their strides may be anything
    assert fast.rows(none, BF, 0, 64, -1)[3:] == fast.rows(none.as_strided((5, 0, 64), (7, 7, 7)), BF, -1, 64, -1)[3:] == (5, 0)
    for a in ((x.float(), BF, 6, 64, -1), (x, BF, 5, 64, -1), (x, BF, 6, 32, -1), (x, BF, 6, 64, 0), (x[0], BF, 6, 64, -1), (x[:, :, ::2], BF, 6, 32, -1),
              (x.transpose(1, 2), BF, 64, 6, -1), ("x", BF, 6, 64, -1)):
        assert fast.rows(*a) is None, a


def test_tensors_without_memory_are_no_crash(fast):
    for t in (torch.zeros((3, 4), device="meta"), torch.zeros((3, 4)).to_sparse(), torch.zeros(3, 4).to_sparse_csr()):
        for check in (lambda: fast.whole(t, F32, (3, 4), -1), lambda: fast.rows(t, F32, 3, 4, -1)):
            try:
                assert check() is None or t.device.type == "meta"
            except RuntimeError:
                pass


def test_calls_pass_numbers_on_as_they_are(fast):
    """Refused calls (no handle): as through ctypes, but integers are never cut to their low bits."""
    h = ctypes.c_void_p()
    ok = [h, 256, 256, 256, 256, 256, 1, 256, None, 1, 256, None, None]
    assert fast.kvs_pool_reserve(*ok) == 1 and fast.kvs_pool_reserve(*([None] + ok[1:])) == 1
    for i in (6, 9):
        for big in (1 << 32, -(1 << 31) - 1, 1 << 80):
            with pytest.raises(OverflowError):
                fast.kvs_pool_reserve(*(ok[:i] + [big] + ok[i + 1:]))
    with pytest.raises(TypeError):
        fast.kvs_pool_reserve(*ok[:-1])
    with pytest.raises(TypeError):
        fast.kvs_pool_reserve(*(ok[:6] + ["1"] + ok[7:]))
    with pytest.raises(AttributeError):
        fast.kvs_pool_reserve(*(["x"] + ok[1:]))
    from sparse_kv_cache_decode_gb300 import _SIGS
    names = [n for n in dir(fast) if n.startswith("kvs_")]
    assert len(names) >= 9 and all(n in _SIGS for n in names)

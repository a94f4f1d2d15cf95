"""What the rotation and the block tables refuse before anything touches a GPU (no GPU)."""
import ctypes

import pytest

torch = pytest.importorskip("torch")

INVALID_ARG = 1
A, B, C, D = 1 << 20, 1 << 21, 1 << 22, 1 << 23           # addresses that are never followed


@pytest.fixture(scope="module")
def K():
    from sparse_kv_cache_decode_gb300 import build as B
    B.build()
    import sparse_kv_cache_decode_gb300 as K
    return K


@pytest.mark.parametrize("over", [
    dict(), dict(head_dim=64), dict(head_dim=256), dict(rot_dim=0), dict(rot_dim=16), dict(rot_dim=112), dict(adjacent=True),
    dict(axes=[0, 1, 2, 3] * 16), dict(axes=[7] * 64), dict(inv_freq=[0.5] * 64, theta=-1.0), dict(inv_freq=[-3.0] * 64), dict(rot_scale=0.0),
    dict(norm_eps=0.0), dict(rot_dim=0, theta=0.0), dict(axes=[0] * 64)])
def test_supported(K, over):
    K.Rope(K.make_rope_config(**(dict(head_dim=128) | over))).close()


@pytest.mark.parametrize("over", [
    dict(head_dim=96), dict(head_dim=512), dict(head_dim=0), dict(rot_dim=8), dict(rot_dim=24), dict(rot_dim=144), dict(theta=0.0),
    dict(theta=float("inf")), dict(theta=float("nan")), dict(inv_freq=[float("nan")] * 64), dict(inv_freq=[float("inf")] * 64),
    dict(axes=[8] * 64), dict(rot_scale=-1.0), dict(rot_scale=float("nan")), dict(norm_eps=-1e-6), dict(norm_eps=float("inf"))])
def test_other_configurations_are_refused(K, over):
    with pytest.raises(K.KvsError):
        K.Rope(K.make_rope_config(**(dict(head_dim=128) | over)))


def test_configurations_that_do_not_fit_together(K):
    for over in (dict(axes=[0] * 63), dict(axes=[-1] + [0] * 63), dict(axes=[256] * 64), dict(inv_freq=[1.0] * 32), dict(rot_dim=-16),
                 dict(head_dim=(1 << 32) + 128), dict(rot_dim=(1 << 32))):
        with pytest.raises(ValueError):
            K.make_rope_config(**(dict(head_dim=128) | over))
    cfg = K.make_rope_config(128)
    cfg.n_axis = 2                                         # several axes without a map
    h = ctypes.c_void_p()
    L = K.lib()
    assert L.kvs_rope_create(ctypes.byref(cfg), ctypes.byref(h)) == INVALID_ARG and not h
    cfg.n_axis, cfg.adjacent = 1, 2
    assert L.kvs_rope_create(ctypes.byref(cfg), ctypes.byref(h)) == INVALID_ARG and not h
    assert L.kvs_rope_create(None, ctypes.byref(h)) == INVALID_ARG and L.kvs_rope_destroy(None) == INVALID_ARG
    assert L.kvs_rope_create(ctypes.byref(K.make_rope_config(128)), None) == INVALID_ARG


def test_axes_of_sections(K):
    assert K.rope_axes([2, 3, 1]) == [0, 0, 1, 1, 1, 2]
    assert K.rope_axes([2, 3, 1], cycle=True) == [0, 1, 2, 0, 1, 1]
    assert K.rope_axes([]) == [] and K.rope_axes([0, 2], cycle=True) == [1, 1]


def _rotate(K, rope, **over):
    a = dict(q=A, qs=256, qh=128, hq=2, qn=None, qo=B, qos=256, qoh=128, k=C, ks=128, kh=128, hk=1, kn=None, ko=D, kos=128, koh=128,
             pos=4096, ps=0, n=4) | over
    return K.lib().kvs_rotate(rope.h, *a.values(), None)


def test_rows_that_are_refused(K):
    r = K.Rope(K.make_rope_config(128))
    bad = [dict(q=0), dict(qo=0), dict(k=0), dict(ko=0), dict(pos=0), dict(n=-1), dict(hq=-1), dict(hk=-1), dict(hq=1025), dict(ps=-1),
           dict(q=A + 8), dict(ko=D + 2), dict(qs=260), dict(qoh=132), dict(qh=64), dict(qs=200), dict(kos=120), dict(qn=8), dict(kn=4),
           dict(qs=128, qh=384), dict(qs=128, qh=504), dict(qs=64, qh=4096), dict(qs=1 << 62), dict(qh=1 << 62), dict(qs=1 << 39, n=1 << 30),
           # outputs over inputs or each other: shifted by a token or a head, of other strides, over the other's rows
           dict(qo=A + 512), dict(qo=A + 256), dict(qo=A, qos=512), dict(qo=C), dict(ko=A), dict(ko=B), dict(ko=B + 256), dict(ko=C + 256),
           dict(qs=768, qh=384, qo=A + 128, qos=768, qoh=384),          # half a head further
           dict(qs=256, qo=A + 256, qos=256, hq=1, n=2, qoh=128, k=A + 128)]
    for over in bad:
        assert _rotate(K, r, **over) == INVALID_ARG, over
    # nothing to do is no error, and launches nothing
    assert _rotate(K, r, n=0, pos=0, q=0) == 0 and _rotate(K, r, hq=0, hk=0) == 0
    assert K.lib().kvs_rotate(None, *([0] * 19), None) == INVALID_ARG


@pytest.mark.skipif(torch.cuda.is_available(), reason="the addresses are not real")
def test_rows_that_may_lie_beside_each_other(K):
    """Calls that pass every check and end at the launch, which fails without a device."""
    r = K.Rope(K.make_rope_config(128))
    ok = [dict(), dict(qo=A, ko=C), dict(q=A, qs=640, k=A + 512, ks=640, qo=A, qos=640, ko=A + 512, kos=640),      # in place in a fused row
          dict(q=A, qs=640, qo=A + 512, qos=640),                                                               # other columns
          dict(qs=768, qh=384, qo=A + 256, qos=768, qoh=384),                                                   # heads in between
          dict(qs=128, qh=512), dict(hk=0, k=0, ko=0, kn=8), dict(hq=0, q=0), dict(n=1, qs=8, ks=0)]
    for over in ok:
        assert _rotate(K, r, **over) == 2, over


def test_null_pools(K):
    r = K.Rope(K.make_rope_config(128))
    L = K.lib()
    assert L.kvs_pool_reserve(None, A, B, C, D, 4096, 1, A, None, 1, B, None, None) == INVALID_ARG
    assert L.kvs_pool_places(None, A, B, C, 1, 1, None, D, None, None) == INVALID_ARG
    assert L.kvs_pool_rotate_append(None, r.h, 0, A, 1024, B, C, 256, None, None, D, 0, 4096, 1, A, 1024, None) == INVALID_ARG
    assert L.kvs_pool_reposition(None, r.h, 0, A, B, C, 1, 8, None) == INVALID_ARG


def test_tensors(K):
    r = K.Rope(K.make_rope_config(128))
    q = torch.zeros((2, 4, 128), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        r.rotate(q, torch.zeros(2, dtype=torch.int32), q)
    r.close()
    with pytest.raises(ValueError, match="closed"):
        r.rotate(q, torch.zeros(2, dtype=torch.int32), q)


class Calls:
    """Stands in for the library: keeps each call's arguments and returns success."""
    def __init__(self):
        self.args = None

    def __getattr__(self, name):
        def call(*a):
            self.args = a
            return 0
        return call


@pytest.fixture
def pool(K, monkeypatch):
    p = object.__new__(K.Pool)
    p.cfg = K.make_pool_config(n_layer=2, n_slots=8, n_q_head=8, n_kv_head=2, head_dim=128, block_size=16, max_ctx=100, max_req=4, max_tokens=64)
    p.L, p.h, p.index, p.device, p.nb_max = Calls(), 1, -1, torch.device("cpu"), 7
    monkeypatch.setattr(torch.cuda, "current_device", lambda: -1)
    yield p
    p.h = None


def test_pool_tensors(K, pool):
    r = K.Rope(K.make_rope_config(128, axes=[0, 1] * 32))
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)  # noqa: E731
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    base = dict(layer=0, rope=r, q=bf(3, 8, 128), k=bf(3, 2, 128), v=bf(3, 2, 128), pos=i32(2, 3), place=torch.zeros(3, dtype=torch.int64),
                q_out=bf(3, 8, 128), q_norm=torch.ones(128), k_norm=torch.ones(128), stream=0)
    pool.rotate_append(**base)
    assert pool.L.args[11] == 3                                             # the axes' stride
    pool.rotate_append(**(base | dict(pos=i32(3))))
    assert pool.L.args[11] == 0                                             # one row for all axes
    for over in (dict(q=bf(3, 4, 128)), dict(q=bf(2, 8, 128)), dict(k=bf(3, 8, 128)), dict(v=bf(2, 2, 128)), dict(v=bf(3, 4, 128)[:, ::2]),
                 dict(v=bf(3, 3, 128)[:, :2]), dict(q_out=bf(3, 8, 128).float()), dict(q_out=bf(4, 8, 128)), dict(pos=i32(3, 3)),
                 dict(pos=i32(2, 4)), dict(pos=i32(4)), dict(pos=torch.zeros(2, 3)), dict(pos=i32(3, 2).T), dict(pos=i32(2, 2, 3)), dict(place=i32(3)),
                 dict(place=torch.zeros(4, dtype=torch.int64)), dict(q_norm=torch.ones(64)), dict(k_norm=torch.ones(128, dtype=torch.bfloat16)),
                 dict(k_norm=torch.ones(256)[::2]), dict(rope=None), dict(layer=1 << 32)):
        with pytest.raises(ValueError):
            pool.rotate_append(**(base | over))
    kept, n, tab = i32(2, 2, 5), i32(2), i32(2, 7)
    pool.reposition(0, r, kept, n, tab, stream=0)
    for bad in ((kept[:, :1], n, tab), (kept, n[:1], tab), (kept, n, tab[:, :3]), (kept.long(), n, tab)):
        with pytest.raises(ValueError):
            pool.reposition(0, r, *bad, stream=0)
    r.close()
    with pytest.raises(ValueError, match="rope"):
        pool.rotate_append(**base)


def test_table_tensors(K, pool):
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    base = [i32(3, 7), i32(3), i32(8), i32(3)]
    t = K.BlockTables(pool, *base)
    for i, bad in [(0, i32(3, 6)), (0, i32(3, 7).long()), (1, i32(2)), (2, i32(7)), (3, i32(2)), (2, i32(16)[::2])]:
        with pytest.raises(ValueError):
            K.BlockTables(pool, *(base[:i] + [bad] + base[i + 1:]))
    place = torch.zeros(5, dtype=torch.int64)
    t.reserve(i32(3), stream=0)
    t.reserve(i32(3), i32(4), place, i32(5), i32(3), stream=0)
    for a in ((i32(2),), (i32(3), i32(3), place), (i32(3), i32(4)), (i32(3), None, place), (i32(3), i32(4), i32(5)),
              (i32(3), i32(4), place, i32(4)), (i32(3), i32(4), place, i32(5), i32(5)), (i32(3), None, None, i32(5))):
        with pytest.raises(ValueError):
            t.reserve(*a, stream=0)
    pool.places(i32(4), i32(3), i32(3, 7), place, stream=0)
    for a in ((i32(3), i32(3), i32(3, 7), place), (i32(4), i32(3), i32(3, 6), place), (i32(4), i32(3), i32(3, 7), i32(5))):
        with pytest.raises(ValueError):
            pool.places(*a, stream=0)

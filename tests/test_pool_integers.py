"""Integers that do not fit the C ABI's 32 bits: ctypes would cut them to their low bits (no GPU)."""
import pytest

torch = pytest.importorskip("torch")

BIG = 1 << 32
OK = dict(n_layer=2, n_slots=8, n_q_head=8, n_kv_head=2, head_dim=128, block_size=16, max_ctx=100, max_req=4, max_tokens=64,
          max_prefix_tokens=16)


@pytest.fixture(scope="module")
def K():
    from sparse_kv_cache_decode_gb300 import build as B
    B.build()
    import sparse_kv_cache_decode_gb300 as K
    return K


@pytest.mark.parametrize("name", list(OK) + ["wait_timeout_us"])
@pytest.mark.parametrize("sign", [1, -1])
def test_configuration(K, name, sign):
    with pytest.raises(ValueError, match=name):
        K.make_pool_config(**(OK | {name: sign * BIG + OK.get(name, 1000)}))
    if name == "wait_timeout_us":
        assert K.make_pool_config(**OK, wait_timeout_us=BIG - 1).wait_timeout_us == BIG - 1
        with pytest.raises(ValueError, match=name):
            K.make_pool_config(**OK, wait_timeout_us=-1)


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
    p.cfg, p.L, p.h, p.index, p.device, p.nb_max = K.make_pool_config(**OK), Calls(), 1, -1, torch.device("cpu"), 7
    monkeypatch.setattr(torch.cuda, "current_device", lambda: -1)
    yield p
    p.h = None


def _batch():
    z = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    return z(2), z(1), z(1, 7)


@pytest.mark.parametrize("layer", [BIG, BIG + 1, -BIG, 1 << 31])
def test_layers(pool, layer):
    cu, ctx, tab = _batch()
    q, new = torch.zeros((1, 8, 128), dtype=torch.bfloat16), torch.zeros((1, 2, 128), dtype=torch.bfloat16)
    w = torch.zeros((1, 2, 100))
    calls = [lambda: pool.attn(layer, q, cu, ctx, tab, q.clone(), stream=0), lambda: pool.append(layer, new, new, cu, ctx, tab, stream=0),
             lambda: pool.prefix_attn(layer, q, cu, ctx, tab, cu, ctx, tab, q.clone(), stream=0),
             lambda: pool.evict(layer, w, ctx, tab, 5, 1, 1, tab, torch.zeros((1, 2, 5), dtype=torch.int32), ctx, w, stream=0)]
    for call in calls:
        with pytest.raises(ValueError, match="layer"):
            call()
    assert pool.L.args is None


@pytest.mark.parametrize("n_sink,n_recent", [(BIG + 1, 1), (1, BIG + 1), (-BIG, 1), (1, -BIG)])
def test_evicted_runs(pool, n_sink, n_recent):
    _, ctx, tab = _batch()
    w = torch.zeros((1, 2, 100))
    with pytest.raises(ValueError, match="n_sink|n_recent"):
        pool.evict(0, w, ctx, tab, 5, n_sink, n_recent, tab, torch.zeros((1, 2, 5), dtype=torch.int32), ctx, w, stream=0)
    assert pool.L.args is None


@pytest.mark.parametrize("n", [99, 100, 5000, BIG + 3, 1 << 40, (1 << 63) - 1])
def test_a_window_longer_than_any_context_is_none(pool, n):
    """A window or a run of first tokens of any size is meaningful: beyond the longest context it is the longest context."""
    cu, ctx, tab = _batch()
    q = torch.zeros((1, 8, 128), dtype=torch.bfloat16)
    pool.attn(0, q, cu, ctx, tab, q.clone(), window=n, n_sink=n, stream=0)
    window, n_sink = pool.L.args[9:11]
    assert (window, n_sink) == (min(n, 100), min(n, 100))
    pool.attn(0, q, cu, ctx, tab, q.clone(), window=-1, n_sink=-1, stream=0)
    assert pool.L.args[9:11] == (-1, -1)                     # left to the library, which refuses them
    with pytest.raises(ValueError, match="window"):
        pool.attn(0, q, cu, ctx, tab, q.clone(), window=-BIG + 3, stream=0)

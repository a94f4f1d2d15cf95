"""What a device-resident pool refuses before anything touches a GPU (no GPU)."""
import ctypes

import pytest

torch = pytest.importorskip("torch")

INVALID_ARG = 1
OK = dict(n_layer=2, n_slots=8, n_q_head=8, n_kv_head=2, head_dim=128, block_size=16, max_ctx=100, max_req=4, max_tokens=64,
          max_prefix_tokens=16)


@pytest.fixture(scope="module")
def K():
    from sparse_kv_cache_decode_gb300 import build as B
    B.build()
    import sparse_kv_cache_decode_gb300 as K
    return K


def _bytes(K, **over):
    return K.lib().kvs_pool_workspace_bytes(ctypes.byref(K.make_pool_config(**(OK | over))))


@pytest.mark.parametrize("over", [
    dict(), dict(head_dim=64), dict(block_size=128), dict(n_q_head=128, n_kv_head=1), dict(n_q_head=2), dict(n_q_head=6),
    dict(max_ctx=1), dict(max_ctx=1 << 30), dict(max_req=2048), dict(max_req=1, n_kv_head=1024, n_q_head=1024),
    dict(max_prefix_tokens=0), dict(max_prefix_tokens=64), dict(kv_dtype="fp8", k_scale=0.0), dict(max_tokens=1 << 23, max_prefix_tokens=0),
    dict(max_req=2048, n_kv_head=8, n_q_head=64, max_tokens=1 << 20)])
def test_supported_configurations_size_a_workspace(K, over):
    n = _bytes(K, **over)
    c = OK | over
    # the rows of shared prefixes are held in fp32 between the two parts of their attention
    assert n >= c["max_prefix_tokens"] * c["n_q_head"] * (c["head_dim"] + 1) * 4 + c["max_tokens"] * c["n_q_head"] * 4


@pytest.mark.parametrize("over", [
    dict(n_layer=0), dict(n_slots=0), dict(n_q_head=7), dict(n_kv_head=0), dict(n_q_head=0), dict(n_q_head=258), dict(head_dim=96),
    dict(head_dim=0), dict(block_size=8), dict(block_size=48), dict(block_size=256), dict(max_ctx=0), dict(max_ctx=(1 << 30) + 1),
    dict(max_req=0), dict(max_req=2049), dict(max_req=2048, n_kv_head=32, n_q_head=32), dict(max_tokens=0), dict(max_tokens=-5),
    dict(max_tokens=1 << 24, n_q_head=8), dict(max_prefix_tokens=65), dict(max_prefix_tokens=-1), dict(k_scale=-1.0),
    dict(v_scale=float("inf")), dict(k_scale=float("nan")), dict(softmax_scale=-1.0), dict(softmax_scale=float("nan")),
    dict(n_slots=(1 << 31) - 1), dict(max_req=2048, n_kv_head=16, n_q_head=128, max_tokens=1 << 20)])
def test_other_configurations_are_refused(K, over):
    assert _bytes(K, **over) == 0
    cfg = K.make_pool_config(**(OK | over))
    h = ctypes.c_void_p()
    assert K.lib().kvs_pool_create(ctypes.byref(cfg), 4096, 8192, 4096, 1 << 40, ctypes.byref(h)) == INVALID_ARG and not h
    with pytest.raises(K.KvsError):
        K.Pool(cfg, torch.empty(1), torch.empty(1))


def test_unknown_dtype(K):
    cfg = K.make_pool_config(**OK)
    cfg.kv_dtype = 7
    assert K.lib().kvs_pool_workspace_bytes(ctypes.byref(cfg)) == 0
    with pytest.raises(KeyError):
        K.make_pool_config(**(OK | dict(kv_dtype="fp16")))


def test_null_handles_and_pointers(K):
    L = K.lib()
    cfg = K.make_pool_config(**OK)
    h = ctypes.c_void_p()
    n = L.kvs_pool_workspace_bytes(ctypes.byref(cfg))
    assert L.kvs_pool_workspace_bytes(None) == 0
    assert L.kvs_pool_create(None, 256, 256, 256, n, ctypes.byref(h)) == INVALID_ARG
    assert L.kvs_pool_create(ctypes.byref(cfg), None, 256, 256, n, ctypes.byref(h)) == INVALID_ARG
    assert L.kvs_pool_create(ctypes.byref(cfg), 256, 256, 256, n - 1, ctypes.byref(h)) == INVALID_ARG      # too small
    assert L.kvs_pool_create(ctypes.byref(cfg), 256, 256, 256, n, None) == INVALID_ARG
    st = ctypes.c_int()
    assert L.kvs_pool_destroy(None) == INVALID_ARG and L.kvs_pool_poll_error(None, ctypes.byref(st)) == INVALID_ARG
    assert L.kvs_pool_launch_count(None) == 0
    assert L.kvs_pool_append(None, 0, 256, 256, 256, 256, 256, 256, 1, 1, None) == INVALID_ARG
    assert L.kvs_pool_attn(None, 0, 256, 1024, 256, 256, 256, 1, 1, 0, 0, 256, None, None, None) == INVALID_ARG
    assert L.kvs_pool_prefix_attn(None, 0, 256, 1024, 256, 256, 256, 1, 1, 256, 256, 256, 1, 256, None, None) == INVALID_ARG
    assert L.kvs_pool_evict(None, 0, 256, 256, 256, 1, 1, 0, 0, 256, 256, 256, 512, None) == INVALID_ARG


def test_pool_tensors(K):
    cfg = K.make_pool_config(**OK)
    shape = (2, 8, 2, 16, 128)
    k = torch.empty(shape, dtype=torch.bfloat16)
    for bad in (k[:, :, :, :, :64], k.float(), k.transpose(2, 3), k[:1], torch.empty(shape, dtype=torch.uint8)):
        with pytest.raises(ValueError, match="k:"):
            K.Pool(cfg, bad, k)
        with pytest.raises(ValueError, match="v:"):
            K.Pool(cfg, k, bad)
    with pytest.raises(ValueError, match="CUDA"):
        K.Pool(cfg, k, k.clone())

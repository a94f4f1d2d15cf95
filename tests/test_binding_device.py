"""What the binding takes for the current device (no GPU)."""
import pytest

torch = pytest.importorskip("torch")


@pytest.mark.skipif(torch.cuda.is_available(), reason="a machine without a GPU")
def test_no_device():
    from sparse_kv_cache_decode_gb300 import build as B
    B.build()
    import sparse_kv_cache_decode_gb300 as K
    assert K.binding().device() == -1


@pytest.mark.gpu
def test_device():
    import sparse_kv_cache_decode_gb300 as K
    assert K.binding().device() == torch.cuda.current_device()

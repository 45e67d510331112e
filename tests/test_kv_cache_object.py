"""The cache object of the Python binding (no GPU needed)."""
import pytest

torch = pytest.importorskip("torch")

from block_quantized_int8_q8_gb300 import _build, api


@pytest.fixture(scope="module", autouse=True)
def built():
    _build.build()


def test_a_cache_keeps_its_tensors():
    """The calls use the tensors that a cache was made of, so another one cannot be put in their place."""
    cache = object.__new__(api.KVCache)
    for name in ("k", "v", "k_scale", "v_scale", "pages", "kv_heads", "page_size", "head_dim", "block"):
        with pytest.raises(AttributeError):
            setattr(cache, name, torch.zeros(1))
        with pytest.raises(AttributeError):
            delattr(cache, name)

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


@pytest.mark.parametrize("page_size,block", [(64, 24), (64, 48), (40, 16), (16, 32), (64, 0), (64, -16)])
def test_blocks_that_do_not_fill_a_page_are_refused(page_size, block):
    """64 tokens in blocks of 24 would otherwise come out as blocks of 32."""
    with pytest.raises(api.MMQError, match="block"):
        api.KVCache.empty(4, 2, 64, page_size, block, device="cpu")

"""The cache's Python objects without a GPU."""
import pytest

from precision_attention_fa4fp4_gb300 import api, build


def test_cache_that_was_never_initialised():
    build.build()
    cache = api.KVCache.__new__(api.KVCache)
    for name in ("k", "v", "ks", "vs", "kb", "device"):
        with pytest.raises(AttributeError):
            getattr(cache, name)
    assert cache.num_pages == cache.Hkv == cache.page == cache.d == 0
    with pytest.raises(ValueError, match="KVCache"):
        api.cache_append(cache, None, None, None, None)

"""The binding's own checks, as far as they need no GPU."""
import pytest


def test_missing_tensors_are_named():
    from kv_cache_vector_compress_b200 import tq
    with pytest.raises(TypeError, match="lens must be given"):
        tq._arg(None, "lens", None, 3, 0)
    with pytest.raises(TypeError, match="own keys and values must be given"):
        tq._cache_args(None, None, None, 3, "own", 0)
    with pytest.raises(TypeError, match="lens must be given"):
        tq.tq_evict(None, None, None, None, None, 1, 8, 4, 1, 4)

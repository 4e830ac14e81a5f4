"""The compiled module behind the paged and windowed calls."""

import pytest


@pytest.fixture(scope="module")
def ub():
    from kv_cache_reuse_falcon_b200 import build
    build.build()
    from kv_cache_reuse_falcon_b200 import binding
    return binding


@pytest.mark.parametrize("name,count", [("pool_write", 14), ("decode", 19), ("evict", 14), ("prefill", 14),
                                        ("prefill_bwd", 19)])
def test_calls_check_the_number_of_their_arguments(ub, name, count):
    f = getattr(ub._calls, name)
    for n in (0, 1, count - 1, count + 1):
        with pytest.raises(TypeError, match="%d arguments by position, got %d" % (count, n)):
            f(*[None] * n)
    with pytest.raises(ValueError):          # the right number, of no tensors
        f(*[None] * count)

"""Sizes that the paged calls refuse without a device."""

import ctypes

import pytest


@pytest.fixture(scope="module")
def ub():
    from kv_cache_reuse_falcon_b200 import build
    build.build()
    from kv_cache_reuse_falcon_b200 import binding
    return binding


INVALID = -1
A = 0x10000   # an aligned address that is never read


@pytest.mark.parametrize("budget", [(1 << 30) + 1, 2 ** 31 - 1000, 2 ** 31 - 1])
def test_evict_refuses_budgets_beyond_its_row_numbers(ub, budget):
    """The kernels step through `budget` places with 32-bit numbers; no request has more than 2^30 rows."""
    pool = ub.KVPool(A, A, 2, 4, 2, 16, 64, 0, 1.0, 1.0)
    assert ub.LIB.unipin_paged_evict(ctypes.byref(pool), 0, A, A, 4, A, 2, 32, budget, 0, 0, A, A + 64, None,
                                     None) == INVALID

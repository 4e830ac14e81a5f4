"""Paged calls at the largest numbers that they take."""

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ub():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from kv_cache_reuse_falcon_b200 import binding
    return binding


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def test_evict_checks_the_pages_of_the_longest_request(ub):
    """2^30 rows in a page of 2^30 + 1: their sum passes 31 bits.  The page id does not exist, so nothing moves."""
    page = (1 << 30) + 1
    free, _ = torch.cuda.mem_get_info()
    if free < 80 << 30:
        pytest.skip("needs 80 GB")
    pk = torch.empty((1, 1, 1, page, 32), dtype=torch.uint8, device="cuda")
    pv, w = torch.empty_like(pk), torch.empty((1, 1, 1, page), device="cuda")
    w[..., :64] = torch.arange(64.0, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    kept, fewer = ub.paged_evict(pk, pv, w, 0, _i32([[1]]), _i32([1 << 30]), 1 << 30, 40, dev_status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == -4 and fewer.tolist() == [-1] and (kept == -1).all()
    # a request of the same pool whose page is there
    status.zero_()
    kept, fewer = ub.paged_evict(pk, pv, w, 0, _i32([[0]]), _i32([64]), 1 << 30, 40, dev_status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0 and fewer.tolist() == [40] and kept[0, 0].tolist() == list(range(24, 64))


def test_write_refuses_a_segment_that_ends_far_before_its_start(ub):
    """The difference of the two ends passes 31 bits and must not come out as a long segment."""
    g = torch.Generator().manual_seed(2)
    k = torch.randn(16, 1, 32, generator=g).to(torch.bfloat16).cuda()
    pk = torch.zeros((1, 2, 1, 8, 32), dtype=torch.bfloat16, device="cuda")
    pv, status = torch.zeros_like(pk), torch.zeros(1, dtype=torch.int32, device="cuda")
    ub.paged_pool_write(pk, pv, 0, k, k, _i32([4, -2 ** 31]), _i32([2]), _i32([[0]]), _i32([0]), 2, dev_status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == -4 and (pk == 0).all() and (pv == 0).all()

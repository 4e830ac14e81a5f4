"""A recorded timeout (the bounded waits' status word) makes later blocks and calls skip their work."""

import glob
import os
import re

import pytest
import torch

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "kv_cache_reuse_falcon_b200", "csrc")
TIMEOUT = -6


def test_a_block_takes_one_decision():
    """Every kernel with bounded waits asks through block_timed_out, whose answer is the same in all warps of a
    block; none compares the status word by itself, where two warps could see different values."""
    asks = 0
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu*"))):
        src = re.sub(r"//[^\n]*", "", open(path).read())
        assert not re.search(r"[=!]=\s*\(int\)\s*UNIPIN_ERR_DEVICE_TIMEOUT", src), path
        asks += len(re.findall(r"if \([^;]*block_timed_out\(\w+(?:\(p\.status\))?, \(int\)UNIPIN_ERR_DEVICE_TIMEOUT\)\)", src))
        # a block takes its decision before the first barrier or tensor-memory set-up
        for kernel in re.split(r"__global__", src)[1:]:
            if "block_timed_out" in kernel and "tmem_alloc" in kernel:
                assert kernel.index("block_timed_out") < min(kernel.index("mbar_init"), kernel.index("tmem_alloc"))
    assert asks == 5


@pytest.mark.gpu
def test_calls_behind_a_timeout_leave_their_outputs():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from kv_cache_reuse_falcon_b200 import binding as ub
    dev = torch.device("cuda")
    g = torch.Generator().manual_seed(1)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)
    q, k, v = (torch.randn(400, h, 64, generator=g).to(torch.bfloat16).to(dev) for h in (4, 2, 2))
    cu, past = i32([0, 250, 400]), i32([200, 150])
    lse = torch.empty(400, 4, device=dev)
    o = ub.windowed_prefill_attn(q, k, v, cu, past, 250, 40, 2, out_fp32=False, lse=lse)
    status = torch.full((1,), TIMEOUT, dtype=torch.int32, device=dev)
    a, b, dq = (torch.full((400, 4, 64), 7.0, device=dev) for _ in range(3))
    ub.masked_prefill_attn(q, k, v, cu, past, 250, out=a, dev_status=status)
    ub.windowed_prefill_attn(q, k, v, cu, past, 250, 40, 2, out=b, dev_status=status)
    ub.windowed_prefill_bwd(q, k, v, o, q, lse, cu, past, 250, 40, 2, dq=dq, dev_status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == TIMEOUT
    assert all((x == 7).all() for x in (a, b, dq))
    status.zero_()
    ub.windowed_prefill_attn(q, k, v, cu, past, 250, 40, 2, out=b, dev_status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0 and (b - o.float()).abs().max() <= o.float().abs().max() * 2.0 ** -8

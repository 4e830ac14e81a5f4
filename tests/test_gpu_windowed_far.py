"""Windowed prefill and gradients of segments that lie behind 2^32 bytes of their tensors."""

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("H,Hkv", [(8, 8), (8, 2)])
def test_segments_behind_four_gigabytes(H, Hkv):
    """The same bits as the same segments at the tensors' beginning."""
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from kv_cache_reuse_falcon_b200 import binding as ub
    free, _ = torch.cuda.mem_get_info()
    if free < 60 << 30:
        pytest.skip("needs 60 GB")
    D, front, lens, past = 128, 2200000, [300, 1, 130], [270, 0, 130]
    T = sum(lens)
    g = torch.Generator().manual_seed(31)
    near = [torch.randn(T, h, D, generator=g).to(torch.bfloat16).cuda() for h in (H, Hkv, Hkv, H)]
    far = []
    for x in near:
        y = torch.empty((front + T,) + x.shape[1:], dtype=x.dtype, device="cuda")
        y[front:] = x
        far.append(y)

    def step(x, at):
        cu = torch.tensor([at, at + 300, at + 301, at + 431], dtype=torch.int32, device="cuda")
        n = torch.tensor(past, dtype=torch.int32, device="cuda")
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        lse = torch.empty(x[0].shape[:2], device="cuda")
        out = ub.windowed_prefill_attn(x[0], x[1], x[2], cu, n, 300, 100, 3, out_fp32=False, lse=lse, dev_status=status)
        grads = ub.windowed_prefill_bwd(x[0], x[1], x[2], out, x[3], lse, cu, n, 300, 100, 3, grad_fp32=False,
                                        dev_status=status)
        assert int(status.item()) == 0
        return [y[at:].clone() for y in (out, lse) + tuple(grads)]

    for a, b in zip(step(near, 0), step(far, front)):
        assert torch.equal(a, b)

"""The windowed gradients' workspace: room for the partial sums of the key tiles whose sweeps are cut, and of no
others, and nothing behind it is written."""

import pytest
import torch

SLOT = 2 * 128 * 4          # dV and dK of 128 keys, per head dim


@pytest.fixture(scope="module")
def ub():
    from kv_cache_reuse_falcon_b200 import build
    build.build()
    from kv_cache_reuse_falcon_b200 import binding
    return binding


@pytest.mark.parametrize("B,H,Hkv,D,rows,window,sinks,cut", [
    (8, 8, 2, 128, 1630, 300, 4, 32),         # the first key tile of 16 (segment, head) in two pieces
    (8, 8, 1, 128, 8192, 300, 16, 40),        # .. of 8 in five
])
def test_sums_of_cut_tiles_only(ub, B, H, Hkv, D, rows, window, sinks, cut):
    size = lambda n: ub.windowed_prefill_bwd_workspace_size(B, H, Hkv, D, rows, B * rows, window, n)
    counters = B * Hkv * ((rows + 127) // 128) * 2 * 4
    assert size(sinks) - size(0) <= cut * SLOT * D + counters + 512


@pytest.mark.gpu
@pytest.mark.parametrize("lens,past,H,Hkv,D,window,sinks", [
    ([700, 300, 1500, 90], [650, 300, 1400, 60], 8, 1, 64, 100, 4),      # tiles with sinks in pieces
    ([700, 300, 900, 90], [650, 300, 800, 60], 16, 1, 32, 90, 0),        # the others
    ([700, 300, 900, 90], [650, 300, 800, 60], 16, 1, 32, 300, 200),     # both
])
def test_nothing_behind_the_workspace_is_written(ub, lens, past, H, Hkv, D, window, sinks):
    """A workspace of exactly the size asked for, among bytes that stay as they were; the bits of another one."""
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    g = torch.Generator().manual_seed(9)
    T = sum(lens)
    cu = torch.tensor([0] + lens).cumsum(0).to(torch.int32).cuda()
    n = torch.tensor(past, dtype=torch.int32, device="cuda")
    q, k, v, dout = (torch.randn(T, h, D, generator=g).to(torch.bfloat16).cuda() for h in (H, Hkv, Hkv, H))
    lse = torch.empty(T, H, device="cuda")
    out = ub.windowed_prefill_attn(q, k, v, cu, n, max(lens), window, sinks, out_fp32=False, lse=lse)
    need = ub.windowed_prefill_bwd_workspace_size(len(lens), H, Hkv, D, max(lens), T, window, sinks)
    space = torch.full((need + 8192,), 0x5A, dtype=torch.uint8, device="cuda")
    args = (q, k, v, out, dout, lse, cu, n, max(lens), window, sinks)
    got = ub.windowed_prefill_bwd(*args, workspace=space[4096:4096 + need])
    want = ub.windowed_prefill_bwd(*args)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert (space[:4096] == 0x5A).all() and (space[4096 + need:] == 0x5A).all()

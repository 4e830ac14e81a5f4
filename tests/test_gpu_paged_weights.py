"""The one-token decode over rows whose weights lie far apart: four rows of weight 1, all others of weight 2^-x.

Tolerance.  Weights are rounded for the product with V by at most 2^-8 relative in bfloat16.  In float16 (E4M3
pools with power-of-two scales) they are held so that the largest is at least 2^14: by at most 2^-11
relative, or by 2^-25 / 2^14 = 2^-39 of the largest where they fall below float16's normal range.  A score is
one exact product times a float32 factor: off by 2^-23 relative, x 2^-22 absolute as a weight's relative error,
below 2^-16; exp2 the same: 2^-15 in all.  The row's sums are float32: a lane adds N / 32 weights where one
block takes the whole row (four warps, eight lanes to a head), each addition off by at most 2^-24 of the sum,
and the products' sums at most N / 4 / 16 additions of 16 rows each: N / 32 * 2^-24 + N / 64 * 2^-24 < N 2^-28."""

import pytest
import torch

pytestmark = pytest.mark.gpu

N, D, PAGE = 1 << 18, 32, 4096
ONE = {torch.uint8: 0x38, torch.bfloat16: 1.0}
ROUND = {"bf16": 2.0 ** -8, "e4m3pow2": 2.0 ** -11, "e4m3": 2.0 ** -8}


@pytest.mark.parametrize("below", [8.3, 20.3, 22.7, 25.5, 30.2])
@pytest.mark.parametrize("kind", ["bf16", "e4m3pow2", "e4m3"])
@pytest.mark.parametrize("one_block", [True, False])
def test_small_weights_count_in_the_output(kind, below, one_block):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from kv_cache_reuse_falcon_b200 import binding as ub
    dtype = torch.bfloat16 if kind == "bf16" else torch.uint8
    scales = {"bf16": None, "e4m3pow2": (1.0, 1.0), "e4m3": (0.75, 0.75)}[kind]
    unit = 0.75 if kind == "e4m3" else 1.0
    pk = torch.zeros((1, N // PAGE, 1, PAGE, D), dtype=dtype, device="cuda")
    pv = torch.full((1, N // PAGE, 1, PAGE, D), ONE[dtype], dtype=dtype, device="cuda")
    tops = [5, 37, 69, 101]                                   # one in each warp's rows
    pk[0, 0, 0, tops, 0] = ONE[dtype]
    pv[0, 0, 0, tops] = 0
    q = torch.zeros((1, 1, D), dtype=torch.bfloat16, device="cuda")
    q[0, 0, 0] = 1.0
    scale = below * 0.6931471805599453 / unit                 # score of a top row: `below` in log2 units, others 0
    table = torch.arange(N // PAGE, dtype=torch.int32, device="cuda")[None]
    lens = torch.tensor([N], dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = ub.paged_decode_attn(q, table, lens, pk, pv, 0, N, scale=scale, workspace=None if one_block else "auto",
                               dev_status=status, pool_scales=scales)
    assert int(status.item()) == 0
    w = 2.0 ** -below * (N - 4)
    want = unit * w / (4 + w)
    tol = want * (ROUND[kind] + 2.0 ** -15 + N * 2.0 ** -28)
    if kind == "e4m3pow2":
        tol += N * 2.0 ** -39
    assert ((out.cpu().double() - want).abs() <= tol).all(), (want, out.flatten()[0].item())

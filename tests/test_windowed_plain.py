"""The windowed prefill's float64 plain forms that the GPU tests compare with: the mask against its
definition, the gradients' formula against differences of the output."""

import pytest
import torch

from tests.windowed_helpers import allowed, grads64, prefill64


@pytest.mark.parametrize("length,n,window,sinks", [(1, 0, 1, 0), (9, 9, 3, 2), (12, 7, 4, 1), (12, 7, None, 0), (6, 0, 2, 5)])
def test_mask_is_the_definition(length, n, window, sinks):
    ok = allowed(length, n, window, sinks)
    for i in range(length):
        for j in range(length):
            pos = min(i, n)
            want = j < n and j <= i and (window is None or pos - j < window or j < sinks)
            assert bool(ok[i, j]) == (want or i == j)


def test_formula_gradients_are_the_differences():
    g = torch.Generator().manual_seed(0)
    cu, past, window, sinks = [0, 7, 8, 19], [4, 0, 11], 3, 1
    q = torch.randn(19, 4, 8, generator=g, dtype=torch.float64)
    k, v = (torch.randn(19, 2, 8, generator=g, dtype=torch.float64) for _ in range(2))
    dout = torch.randn(19, 4, 8, generator=g, dtype=torch.float64)
    grads = grads64(q, k, v, dout, cu, past, window, sinks)
    for name, x in (("dq", q), ("dk", k), ("dv", v)):
        step = torch.randn(x.shape, generator=g, dtype=torch.float64)
        h = 1e-5
        x += h * step
        up = (prefill64(q, k, v, cu, past, window, sinks)[0] * dout).sum()
        x -= 2 * h * step
        down = (prefill64(q, k, v, cu, past, window, sinks)[0] * dout).sum()
        x += h * step
        want = (grads[name][0] * step).sum()
        # central differences: O(h^2) plus 1e-16 / h of rounding in sums around 1e2
        assert abs((up - down) / (2 * h) - want) < 1e-6 * (1 + abs(want))

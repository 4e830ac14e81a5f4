"""How exact the windowed gradients are, in the L2 norm: the kernels' roundings and no others.

The forward's output and row statistic are taken from float64 (the output rounded to bfloat16, as a training
step stores it), so what is left is the backward's own: Dvec = dO . O of that rounded output (of rows that see
eight keys or fewer the sum over those keys instead, which rounds nothing), dS as the sum of two bfloat16, P
as one.  A plain form in float64 with these roundings planted says what they cost on the test's inputs.  Beyond
them a weight is off by the float32 score (sums of D products of numbers around 1, 2^-13 at the very most, in the
weight and in its normaliser) and dP, Dvec and the sums by float32: each well below 2^-12 of a gradient's norm.
The same form with dS rounded once, and with Dvec of every row from the rounded output, lies above the bound: the
test would see either."""

import math

import pytest
import torch

from tests.windowed_helpers import allowed, grads64, prefill64

FEW = 8


def bf16(x):
    return x.to(torch.bfloat16).double()


def two(x):
    """The upper eight bits of the significand, and the rest rounded to as many."""
    f = x.float()
    up = (f.view(torch.int32) & -65536).view(torch.float32)
    return up.double() + bf16(f - up)


def planted(q, k, v, dout, o, cu, past, window, sinks, cut, few):
    """The gradients with `cut` in place of dS's rounding and Dvec from `o` where a row sees more than `few` keys."""
    T, H, D = q.shape
    G = H // k.shape[1]
    scale = 1.0 / math.sqrt(D)
    q, k, v, dout, o = (x.double() for x in (q, k, v, dout, o))
    g = [torch.zeros_like(x) for x in (q, k, v)]
    for b, n in enumerate(past):
        t = slice(cu[b], cu[b + 1])
        ok = allowed(cu[b + 1] - cu[b], n, window, sinks)
        for h in range(H):
            hk = h // G
            p = torch.softmax((q[t, h] @ k[t, hk].T * scale).masked_fill(~ok, -math.inf), -1)
            dP = dout[t, h] @ v[t, hk].T
            dvec = torch.where(ok.sum(-1) <= few, (p * dP).sum(-1), (dout[t, h] * o[t, h]).sum(-1))
            dS, own = p * (dP - dvec[:, None]), torch.eye(len(ok), dtype=torch.bool)
            own &= torch.arange(len(ok))[:, None] >= n            # a candidate's own key stays in float32
            dS, p = torch.where(own, dS, cut(dS)), torch.where(own, p, bf16(p))
            g[0][t, h] = scale * dS @ k[t, hk]
            g[1][t, hk] += scale * dS.T @ q[t, h]
            g[2][t, hk] += p.T @ dout[t, h]
    return g


CASES = [
    # lens, past, H, Hkv, window, sinks
    ([200, 150], [200, 120], 2, 1, 2, 0),
    ([300, 60], [250, 60], 2, 2, 6, 2),
    ([420, 300], [400, 250], 2, 2, 128, 0),
    ([500, 200], [430, 200], 4, 1, 64, 4),
]


def bounds(case, D):
    """Inputs, the exact gradients and, for each, the bound and the errors of the two coarser forms."""
    lens, past, H, Hkv, window, sinks = CASES[case]
    g = torch.Generator().manual_seed(50 + case)
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    q, k, v, dout = (torch.randn(cu[-1], h, D, generator=g).to(torch.bfloat16) for h in (H, Hkv, Hkv, H))
    o, _, lse = prefill64(q, k, v, cu, past, window, sinks)
    o = o.to(torch.bfloat16)
    exact = [x[0] for x in grads64(q, k, v, dout, cu, past, window, sinks).values()]
    form = lambda cut, few: planted(q, k, v, dout, o, cu, past, window, sinks, cut, few)
    err = lambda got: [float((a - b).norm() / b.norm()) for a, b in zip(got, exact)]
    kernel, once, rounded = err(form(two, FEW)), err(form(bf16, FEW)), err(form(two, 0))
    return (q, k, v, dout, o, lse.float(), cu, past, max(lens), window, sinks), exact, [x + 2.0 ** -12 for x in kernel], \
        once, rounded


@pytest.mark.parametrize("D", [32, 128])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_the_bound_tells_the_coarser_forms(case, D):
    _, _, bound, once, rounded = bounds(case, D)
    for i in (0, 1):                                      # dq, dk
        assert once[i] > 1.2 * bound[i], (bound, once)
        if CASES[case][4] + CASES[case][5] <= FEW:        # every row sees few keys
            assert rounded[i] > 1.2 * bound[i], (bound, rounded)


@pytest.mark.gpu
@pytest.mark.parametrize("D", [32, 64, 128])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_gradients_have_no_other_roundings(case, D):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from kv_cache_reuse_falcon_b200 import binding as ub
    (q, k, v, dout, o, lse, cu, past, rows, window, sinks), exact, bound, _, _ = bounds(case, D)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    got = ub.windowed_prefill_bwd(q.cuda(), k.cuda(), v.cuda(), o.cuda(), dout.cuda(), lse.cuda(), i32(cu), i32(past),
                                  rows, window, sinks)
    for name, a, b, most in zip(("dq", "dk", "dv"), got, exact, bound):
        err = float((a.cpu().double() - b).norm() / b.norm())
        assert err <= most, "%s: %.3e above %.3e" % (name, err, most)

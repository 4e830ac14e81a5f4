"""The windowed prefill and its gradients against their plain forms in float64.

Tolerances.  A weight comes from a float32 score (off by less than 2^-13 absolute: 128 products of numbers
around 1, as in the paged decode's tests) through exp2, of which one pair in four is a polynomial with a
relative error of 1.02e-4; the normaliser is a sum of such weights, and the backward's lse its logarithm.
So a weight is off by at most 2 (2^-13 + 1.02e-4) < 2^-11 relative (WEIGHT), and by one bfloat16 rounding,
2^-8 (ROUND), as an operand of the product with V or dO: |out - ref| <= sum p |v| (2^-8 + 2^-11).  lse is
off by log2(e) (2^-13 + 1.02e-4) < 2^-11.  dS takes one rounding and the weight's error, and the error of
Dvec = dO . out, where out was rounded to bfloat16 and has the forward's error (windowed_helpers.grads64
sums these).  A bfloat16 output adds 2^-8 of its value."""

import pytest
import torch

from tests.windowed_helpers import ROUND, WEIGHT, grads64, prefill64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ub():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from kv_cache_reuse_falcon_b200 import binding
    return binding


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _ok(ub, status):
    torch.cuda.synchronize()
    assert int(status.item()) == 0, ub.status_string(int(status.item()))


def _inputs(seed, lens, H, Hkv, D, front=0, back=0):
    """q, k, v, dout with `front` rows of NaN before the first segment and `back` behind the last, and cu."""
    g = torch.Generator().manual_seed(seed)
    cu = [front]
    for n in lens:
        cu.append(cu[-1] + n)
    T = cu[-1] + back
    out = []
    for heads in (H, Hkv, Hkv, H):
        x = torch.randn(T, heads, D, generator=g).to(torch.bfloat16)
        x[:front] = float("nan")
        x[cu[-1]:] = float("nan")
        out.append(x)
    return out, cu


def _forward(ub, q, k, v, cu, past, window, sinks, out_fp32):
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    T, H, D = q.shape
    out = torch.full((T, H, D), 7.0, dtype=torch.float32 if out_fp32 else torch.bfloat16, device="cuda")
    lse = torch.full((T, H), 7.0, dtype=torch.float32, device="cuda")
    ub.windowed_prefill_attn(q.cuda(), k.cuda(), v.cuda(), _i32(cu), _i32(past),
                             max(b - a for a, b in zip(cu, cu[1:])), window, sinks, out=out, out_fp32=out_fp32, lse=lse,
                             dev_status=status)
    _ok(ub, status)
    return out, lse


def _within(got, ref, tol, rows):
    got = got.cpu().double()
    over = ((got - ref).abs() - tol)[rows]
    assert torch.isfinite(got[rows]).all()
    assert over.numel() == 0 or over.max() <= 0, "over by %.3e" % over.max()


def _check_forward(out, lse, ref, mag, lse_ref, rows):
    tol = mag * (ROUND + WEIGHT) + 1e-6
    if out.dtype == torch.bfloat16:
        tol = tol + ref.abs() * ROUND
    _within(out, ref, tol, rows)
    _within(lse, lse_ref, torch.full_like(lse_ref, 2.0 ** -11), rows)


CASES = [
    # lens, past, H, Hkv, window, sinks
    ([1, 2, 63, 64, 65, 1], [1, 0, 40, 64, 1, 0], 2, 2, 5, 0),
    ([300, 129, 40, 257], [300, 100, 0, 256], 2, 1, 1, 0),
    ([300, 129, 40, 257], [250, 129, 40, 200], 4, 2, 64, 4),
    ([700, 1, 513], [600, 0, 512], 3, 1, 100, 1),
    ([700, 130, 513], [690, 30, 129], 2, 2, 130, 70),
    ([640, 128, 256], [500, 64, 128], 2, 2, 127, 200),
    ([420, 90], [128, 77], 16, 1, 300, 16),
    ([420, 90], [400, 77], 2, 2, None, 0),
    ([530, 200], [520, 190], 2, 1, 2 ** 31 - 1, 2 ** 31 - 1),
]


@pytest.mark.parametrize("D", [32, 64, 128])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_forward_and_gradients_match_plain(ub, D, case):
    lens, past, H, Hkv, window, sinks = CASES[case]
    front, back = (5, 9) if case % 2 else (0, 130)
    (q, k, v, dout), cu = _inputs(10 * case + D, lens, H, Hkv, D, front, back)
    rows = slice(cu[0], cu[-1])
    ref, mag, lse_ref = prefill64(q, k, v, cu, past, window, sinks)
    out32, lse = _forward(ub, q, k, v, cu, past, window, sinks, True)
    _check_forward(out32, lse, ref, mag, lse_ref, rows)
    out, lse = _forward(ub, q, k, v, cu, past, window, sinks, False)
    _check_forward(out, lse, ref, mag, lse_ref, rows)
    for x in (out32, out, lse):                            # rows of no segment are left as they were
        assert (x[: cu[0]] == 7).all() and (x[cu[-1]:] == 7).all()
    want = grads64(q, k, v, dout, cu, past, window, sinks)
    args = [x.cuda() for x in (q, k, v)] + [out, dout.cuda(), lse, _i32(cu), _i32(past), max(lens), window, sinks]
    for fp32 in (True, False):
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        kind = torch.float32 if fp32 else torch.bfloat16
        g = [torch.full(x.shape, 7.0, dtype=kind, device="cuda") for x in (q, k, v)]
        ub.windowed_prefill_bwd(*args, grad_fp32=fp32, dq=g[0], dk=g[1], dv=g[2], dev_status=status)
        _ok(ub, status)
        for name, got in zip(("dq", "dk", "dv"), g):
            r, tol = want[name]
            tol = tol + 1e-6 + (0 if fp32 else r.abs() * ROUND)
            _within(got, r, tol, rows)
            assert (got[: cu[0]] == 7).all() and (got[cu[-1]:] == 7).all()
        again = ub.windowed_prefill_bwd(*args, grad_fp32=fp32)
        for a, b in zip(g, again):                         # no atomics: the same bits
            assert torch.equal(a[rows], b[rows])


@pytest.mark.parametrize("D", [32, 64, 128])
def test_segments_are_apart(ub, D):
    """A segment full of NaN and infinities changes no bit of its neighbours, shorter than a tile or longer."""
    lens, past, window, sinks = [70, 33, 10, 300, 5], [60, 30, 10, 280, 0], 40, 2
    (q, k, v, dout), cu = _inputs(77, lens, 2, 1, D)

    def run(q, k, v, dout):
        out, lse = _forward(ub, q, k, v, cu, past, window, sinks, False)
        return [out, lse] + list(ub.windowed_prefill_bwd(q.cuda(), k.cuda(), v.cuda(), out, dout.cuda(), lse, _i32(cu),
                                                         _i32(past), max(lens), window, sinks))

    clean = run(q, k, v, dout)
    for bad in (0, 1, 3):
        x = [t.clone() for t in (q, k, v, dout)]
        for t in x:
            t[cu[bad]:cu[bad + 1]] = float("nan")
            t[cu[bad] + 1] = float("inf")
        got = run(*x)
        for a, b in zip(clean, got):
            for s in range(len(lens)):
                if s != bad:
                    assert torch.equal(a[cu[s]:cu[s + 1]], b[cu[s]:cu[s + 1]]), (bad, s)


def test_masked_scores_and_odd_values(ub):
    """NaN and infinite keys that the mask hides change nothing; seen, they make their rows NaN; a key whose
    score is -inf has no weight."""
    lens, past, window, sinks = [200], [200], 16, 1
    (q, k, v, _), cu = _inputs(5, lens, 1, 1, 64)
    ref, _ = _forward(ub, q, k, v, cu, past, window, sinks, True)
    for val in (float("nan"), float("inf")):
        k2 = k.clone()
        k2[100] = val
        out, lse = _forward(ub, q, k2, v, cu, past, window, sinks, True)
        seen = torch.zeros(200, dtype=torch.bool)
        seen[100:116] = True
        assert torch.equal(out.cpu()[~seen], ref.cpu()[~seen])
        if val != val:
            assert torch.isnan(out.cpu()[seen]).all() and torch.isnan(lse.cpu()[seen]).all()
    q2, k2 = torch.ones_like(q), k.clone()
    k2[100] = float("-inf")
    out, _ = _forward(ub, q2, k2, v, cu, past, window, sinks, True)
    K, V = k2.double()[:, 0], v.double()[:, 0]
    for i in (100, 105, 115, 116):
        idx = [j for j in range(i + 1) if (i - j < 16 or j < 1) and j != 100]
        p = torch.softmax(K[idx].sum(-1) / 8, 0)
        # scores of |k| sums up to 64 terms around 1: the weight bound of the notes above holds
        assert ((out[i, 0].cpu().double() - p @ V[idx]).abs() <= (p @ V[idx].abs()) * (ROUND + WEIGHT) + 1e-6).all()


def test_no_window_is_the_masked_prefill(ub):
    """Without a window the pairs are the masked prefill's: each of two results is within the bounds of the
    notes above of the exact one, so they are within twice those of each other."""
    lens, past = [300, 77, 520], [250, 77, 400]
    (q, k, v, dout), cu = _inputs(6, lens, 4, 2, 128)
    out, lse = _forward(ub, q, k, v, cu, past, None, 0, False)
    ref_lse = torch.empty_like(lse)
    ref = ub.masked_prefill_attn(q.cuda(), k.cuda(), v.cuda(), _i32(cu), _i32(past), 520, out_fp32=False, lse=ref_lse)
    exact, mag, _ = prefill64(q, k, v, cu, past, None, 0)
    tol = 2 * (mag * (ROUND + WEIGHT) + 1e-6 + exact.abs() * ROUND)
    assert ((out - ref).abs().cpu().double() <= tol).all() and ((lse - ref_lse).abs() <= 2.0 ** -10).all()
    a = ub.masked_prefill_bwd(q.cuda(), k.cuda(), v.cuda(), out, dout.cuda(), lse, _i32(cu), _i32(past), 520)
    b = ub.windowed_prefill_bwd(q.cuda(), k.cuda(), v.cuda(), out, dout.cuda(), lse, _i32(cu), _i32(past), 520, None)
    want = grads64(q, k, v, dout, cu, past, None, 0)
    for name, x, y in zip(("dq", "dk", "dv"), a, b):
        assert ((x - y).abs().cpu().double() <= 2 * want[name][1] + 1e-6).all()


def test_device_rejections(ub):
    """A history longer than its segment, or a segment longer than max_seqlen: a status, zeros where the rows
    are known, the other segments untouched by it."""
    lens, past, window, sinks = [40, 70, 50], [30, 60, 50], 9, 2
    (q, k, v, dout), cu = _inputs(8, lens, 2, 2, 32)
    good, lse = _forward(ub, q, k, v, cu, past, window, sinks, False)
    gg = ub.windowed_prefill_bwd(q.cuda(), k.cuda(), v.cuda(), good, dout.cuda(), lse, _i32(cu), _i32(past), 70, window,
                                 sinks)
    for bad_past, max_len in (([30, 71, 50], 70), ([30, -1, 50], 70), (past, 60)):
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        out = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
        ub.windowed_prefill_attn(q.cuda(), k.cuda(), v.cuda(), _i32(cu), _i32(bad_past), max_len, window, sinks, out=out,
                                 out_fp32=False, dev_status=status)
        torch.cuda.synchronize()
        assert int(status.item()) == -4
        status.zero_()
        g = [torch.full(x.shape, 7.0, dtype=torch.float32, device="cuda") for x in (q, k, v)]
        ub.windowed_prefill_bwd(q.cuda(), k.cuda(), v.cuda(), good, dout.cuda(), lse, _i32(cu), _i32(bad_past), max_len,
                                window, sinks, dq=g[0], dk=g[1], dv=g[2], dev_status=status)
        torch.cuda.synchronize()
        assert int(status.item()) == -4
        for s in (0, 2):
            r = slice(cu[s], cu[s + 1])
            assert torch.equal(out[r], good[r])
            assert all(torch.equal(a[r], b[r]) for a, b in zip(g, gg))
        if max_len == 70:
            assert (out[cu[1]:cu[2]] == 0).all() and all((x[cu[1]:cu[2]] == 0).all() for x in g)

"""The paged pool's operators against their plain forms in float64: the write, the one-token decode
and the eviction, alone and one after another.

Tolerances.  Softmax weights are rounded once for the product with V, by at most half a step: 2^-8
relative in bfloat16, 2^-11 in float16 (E4M3 pools with power-of-two scales), where a weight below
float16's normal range is off by at most 2^-25 of the largest one.  With o = sum p v that is an error of at
most 2^-8 sum p |v| (2^-11 sum p |v| + n 2^-25 max |v|).  Scores are float32 sums of D <= 128 exact products
of numbers around 1: off by less than 2^-13 (128 * 2^-24 * sum |q k| scale, sum |q k| scale below 16), so
each weight by as much relative, twice with the normaliser: 2^-12.  A bfloat16 output adds 2^-8 |o|.
Collected weights have only the 2^-12, and the float32 rounding of the sum they are added to."""

import pytest
import torch

from tests.paged_helpers import PagedCase, decode64, evict64, visible

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ub():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from kv_cache_reuse_falcon_b200 import binding
    return binding


def _status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def _ok(ub, status):
    torch.cuda.synchronize()
    assert int(status.item()) == 0, ub.status_string(int(status.item()))


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _pow2(scales):
    return scales is not None and all(float(torch.frexp(torch.tensor(s))[0]) == 0.5 for s in scales)


def _check_out(out, ref, mag, case, half_p):
    tol = mag * ((2.0 ** -11 if half_p else 2.0 ** -8) + 2.0 ** -12) + 1e-6
    if half_p:
        tol = tol + max(case.lens + [1]) * 2.0 ** -25 * 16
    if out.dtype == torch.bfloat16:
        tol = tol + ref.abs() * 2.0 ** -8
    err = (out.cpu().double() - ref).abs()
    assert torch.isfinite(out).all()
    worst = (err - tol).max()
    assert worst <= 0, "over by %.3e (error %.3e)" % (worst, err.max())


def _decode(ub, case, q, k_self=None, v_self=None, window=None, sinks=0, weights=False, out_fp32=True, max_len=None,
            workspace="auto"):
    status = _status()
    w = case.weights.cuda() if weights else None
    out = ub.paged_decode_attn(q.cuda(), case.table.cuda(), _i32(case.lens), case.k.cuda(), case.v.cuda(), case.layer,
                               max(case.lens) if max_len is None else max_len,
                               k_self=None if k_self is None else k_self.cuda(),
                               v_self=None if v_self is None else v_self.cuda(), window=window, n_sinks=sinks,
                               key_weights=w, out_fp32=out_fp32, dev_status=status, pool_scales=case.scales,
                               workspace=workspace)
    _ok(ub, status)
    return out, w


def _inputs(case, H, own):
    R = len(case.lens)
    q = torch.randn(R, H, case.D, generator=case.g).to(torch.bfloat16)
    if not own:
        return q, None, None
    return (q, torch.randn(R, case.Hkv, case.D, generator=case.g).to(torch.bfloat16),
            torch.randn(R, case.Hkv, case.D, generator=case.g).to(torch.bfloat16))


POW2, ANY = (2.0 ** -6, 2.0 ** -5), (0.0171, 0.0233)


@pytest.mark.parametrize("D", [32, 64, 128])
@pytest.mark.parametrize("scales", [None, POW2, ANY], ids=["bf16", "e4m3pow2", "e4m3"])
@pytest.mark.parametrize("H,Hkv,page,window,sinks,own,weights", [
    (2, 2, 16, None, 0, True, False),
    (8, 2, 7, None, 0, False, True),
    (6, 3, 1, 5, 2, True, True),
    (16, 1, 64, 40, 4, False, True),     # 16 query heads: all rows of the MMA
    (40, 2, 48, 70, 100, True, True),    # 20 per key/value head: two column groups; more sinks than window
    (9, 1, 128, 1, 0, True, False),      # a window of the token itself
    (3, 3, 33, 1, 0, False, True),       # the last row alone
], ids=["mha", "gqa", "page1", "g16", "g20", "own", "last"])
def test_decode_matches_plain(ub, D, scales, H, Hkv, page, window, sinks, own, weights):
    lens = [0, 1, 130, 16, 17, 63, 300]
    case = PagedCase(100 + D + H, lens, Hkv, D, page, scales=scales)
    case.poison_unseen([set(visible(n, window, sinks, own)) for n in lens])
    q, ks, vs = _inputs(case, H, own)
    ref, mag, wref = decode64(case, q, ks, vs, window, sinks)
    for out_fp32 in (True, False):
        out, w = _decode(ub, case, q, ks, vs, window, sinks, weights, out_fp32)
        _check_out(out, ref, mag, case, _pow2(scales))
        if lens[0] == 0 and not own:
            assert (out[0] == 0).all()
        if not weights:
            continue
        want = case.weights.double().clone()
        size = torch.zeros_like(want)
        for r, (idx, p) in wref.items():
            for i, j in enumerate(idx):
                pg, off = case.row(r, j)
                want[case.layer, pg, :, off] += p[i]
                size[case.layer, pg, :, off] = p[i]
        got = w.cpu().double()
        assert torch.equal(torch.isnan(got), torch.isnan(want))
        fine = ~torch.isnan(want)
        assert ((got - want).abs()[fine] <= (size * 2.0 ** -12 + want.abs() * 2.0 ** -23)[fine]).all()


@pytest.mark.parametrize("scales", [None, POW2], ids=["bf16", "e4m3pow2"])
def test_decode_split_and_unsplit_agree_with_plain_on_long_caches(ub, scales):
    """Several chunks per request, the joins over ragged counts of them, and the one-block form."""
    lens = [5000, 1, 2049, 0]
    case = PagedCase(7, lens, 1, 64, 96, scales=scales)
    q, ks, vs = _inputs(case, 2, True)
    ref, mag, _ = decode64(case, q, ks, vs, None, 0)
    nbytes = ub.paged_decode_workspace_size(case.k.cuda(), case.v.cuda(), 4, 2, 5000, pool_scales=scales)
    assert nbytes > 0
    for ws in ("auto", None, torch.empty(16, dtype=torch.uint8, device="cuda")):
        out, _ = _decode(ub, case, q, ks, vs, workspace=ws)
        _check_out(out, ref, mag, case, _pow2(scales))
    # a bound on the lengths above them all changes the split, not the result
    wide = PagedCase(7, lens, 1, 64, 96, scales=scales, width=200)
    out, _ = _decode(ub, wide, q, ks, vs, max_len=200 * 96)
    _check_out(out, ref, mag, case, _pow2(scales))


def test_decode_large_scores_and_infinite_inputs(ub):
    """Scores far apart (the running maximum moves), and non-finite inputs reach only their own rows."""
    lens = [200, 200, 200]
    case = PagedCase(11, lens, 1, 64, 16)
    q, _, _ = _inputs(case, 1, False)
    q = (q.float() * 40).to(torch.bfloat16)
    ref, mag, _ = decode64(case, q, None, None, None, 0)
    # |q k| sums up to 40 times larger here: scores are off by 2^-13 * 40, the weights by that relative
    out, _ = _decode(ub, case, q)
    err = (out.cpu().double() - ref).abs()
    assert (err <= mag * (2.0 ** -8 + 40 * 2.0 ** -12) + 1e-6).all()
    pg, off = case.row(1, 150)
    case.k[case.layer, pg, :, off] = float("nan")
    pg, off = case.row(2, 3)
    case.v[case.layer, pg, :, off] = float("inf")
    again, _ = _decode(ub, case, q)
    assert torch.equal(again[0], out[0])
    assert torch.isnan(again[1]).all()
    assert not torch.isfinite(again[2]).any()


def test_decode_minus_infinity_scores_are_no_weight(ub):
    """A key whose score is -inf carries no weight; where every score is, the row is zeros."""
    lens = [40, 40]
    case = PagedCase(12, lens, 1, 32, 8)
    q = torch.ones(2, 1, 32).to(torch.bfloat16)
    for j in range(40):
        for r in ((0, 1) if j % 2 else (1,)):
            pg, off = case.row(r, j)
            case.k[case.layer, pg, :, off] = float("-inf")
    out, w = _decode(ub, case, q, weights=True)
    keep = [j for j in range(40) if j % 2 == 0]
    K = case.rows64(case.k, None, 0, keep)[:, 0]
    V = case.rows64(case.v, None, 0, keep)[:, 0]
    p = torch.softmax(K.sum(-1) / 32 ** 0.5, 0)
    assert ((out[0, 0].cpu().double() - p @ V).abs() <= (p @ V.abs()) * (2.0 ** -8 + 2.0 ** -12) + 1e-6).all()
    assert (out[1] == 0).all()
    pg, off = case.row(0, 1)
    assert w[case.layer, pg, 0, off].item() == case.weights[case.layer, pg, 0, off].item()


def test_decode_e4m3_reads_every_code(ub):
    """A window of one row makes the output that row: every finite code, exactly, for both kinds of scales."""
    for scales in (POW2, ANY, (2.0 ** 20, 2.0 ** -40)):
        codes = [c for c in range(256) if c & 0x7F != 0x7F]
        lens = [1] * 8
        case = PagedCase(13, lens, 1, 32, 4, scales=scales)
        for r in range(8):
            pg, off = case.row(r, 0)
            part = codes[32 * r: 32 * r + 32]
            case.v[case.layer, pg, 0, off] = torch.tensor(part + [0] * (32 - len(part)), dtype=torch.uint8)
        q = torch.randn(8, 1, 32, generator=case.g).to(torch.bfloat16)
        out, _ = _decode(ub, case, q)
        want = torch.stack([case.rows64(case.v, scales[1], r, [0])[0] for r in range(8)])
        assert torch.equal(out.cpu().double(), want)
    # a NaN code reads as NaN
    pg, off = case.row(3, 0)
    case.v[case.layer, pg, 0, off, 5] = 0xFF
    out, _ = _decode(ub, case, q)
    assert torch.isnan(out[3, 0, 5])


def test_decode_e4m3_query_range(ub):
    """Queries of very different magnitudes over an E4M3 pool with power-of-two scales (float16 operands)."""
    lens = [64] * 5
    case = PagedCase(14, lens, 1, 64, 16, scales=POW2)
    q = torch.randn(5, 1, 64, generator=case.g)
    q = q * torch.tensor([1e-38, 1e-6, 1.0, 1e5, 0.0])[:, None, None]
    q[3] *= 1e-5 * 8   # and a row with one element far above the others
    q[3, 0, 0] = 30.0
    q = q.to(torch.bfloat16)
    ref, mag, _ = decode64(case, q, None, None, None, 0)
    out, _ = _decode(ub, case, q)
    _check_out(out, ref, mag, case, True)


def test_decode_rejects_bad_lengths_and_pages(ub):
    """A request with a length or a page out of range is zeros and a status; the others are untouched by it,
    and weights are collected for the others only."""
    lens = [40, 40, 40]
    case = PagedCase(15, lens, 2, 32, 8)
    q, ks, vs = _inputs(case, 4, True)
    good, wgood = _decode(ub, case, q, ks, vs, weights=True)
    for what in ("page", "negative", "long"):
        table, n = case.table.clone(), list(lens)
        if what == "page":
            table[1, 3] = case.k.shape[1]
        else:
            n[1] = -1 if what == "negative" else 41
        status = _status()
        w = case.weights.cuda()
        out = ub.paged_decode_attn(q.cuda(), table.cuda(), _i32(n), case.k.cuda(), case.v.cuda(), case.layer, 40,
                                   k_self=ks.cuda(), v_self=vs.cuda(), key_weights=w, dev_status=status)
        torch.cuda.synchronize()
        assert int(status.item()) == -4
        assert (out[1] == 0).all()
        assert torch.equal(out[0], good[0]) and torch.equal(out[2], good[2])
        for r in range(3):
            for j in range(40):
                pg, off = case.row(r, j)
                want = case.weights if r == 1 else wgood.cpu()
                assert torch.equal(w.cpu()[case.layer, pg, :, off], want[case.layer, pg, :, off])


# --------------------------------------------------------------------- write

@pytest.mark.parametrize("D,Hkv,page", [(32, 1, 1), (64, 3, 7), (128, 2, 64)])
@pytest.mark.parametrize("scales", [None, POW2, ANY], ids=["bf16", "e4m3pow2", "e4m3"])
def test_write_puts_rows_into_pages(ub, D, Hkv, page, scales):
    new, extra, first = [5, 0, 70, 1], [2, 3, 0, 0], [0, 4, 9, 64]
    lens = [f + n for f, n in zip(first, new)]
    case = PagedCase(20, lens, Hkv, D, page, scales=scales)
    segs = [n + e for n, e in zip(new, extra)]
    cu = [0]
    for x in segs:
        cu.append(cu[-1] + x)
    k = torch.randn(cu[-1], Hkv, D, generator=case.g).to(torch.bfloat16)
    v = torch.randn(cu[-1], Hkv, D, generator=case.g).to(torch.bfloat16)
    k[0, 0, 0], k[0, 0, 1], k[0, 0, 2] = float("nan"), float("inf"), -3e38
    want = [case.k.clone(), case.v.clone()]
    ww = case.weights.clone()
    for b in range(4):
        for j in range(new[b]):
            pg, off = case.row(b, first[b] + j)
            ww[case.layer, pg, :, off] = 0
            for t, x, i in ((want[0], k, 0), (want[1], v, 1)):
                row = x[cu[b] + j]
                if scales is not None:
                    y = row.float() * (torch.tensor(1.0) / torch.tensor(scales[i]))
                    y = torch.where(torch.isnan(y), y, y.clamp(-448, 448))
                    row = y.to(torch.float8_e4m3fn).view(torch.uint8)
                t[case.layer, pg, :, off] = row
    pk, pv, w, status = case.k.cuda(), case.v.cuda(), case.weights.cuda(), _status()
    ub.paged_pool_write(pk, pv, case.layer, k.cuda(), v.cuda(), _i32(cu), _i32(new), case.table.cuda(), _i32(first),
                        max(new), key_weights=w, dev_status=status, pool_scales=scales)
    _ok(ub, status)
    kind = torch.int16 if scales is None else torch.uint8
    assert torch.equal(pk.cpu().view(kind), want[0].view(kind))
    assert torch.equal(pv.cpu().view(kind), want[1].view(kind))
    assert torch.equal(w.cpu().view(torch.int32), ww.view(torch.int32))


def test_write_rejects_out_of_range_segments(ub):
    case = PagedCase(21, [8, 8, 8], 1, 32, 4)
    k = torch.randn(24, 1, 32, generator=case.g).to(torch.bfloat16)
    cu = [0, 8, 16, 24]
    # too many rows, a negative start, a start past the pages, a page id out of range
    for new, first, page in (([8, 9, 8], [0, 0, 0], None), ([8, 8, 8], [0, -1, 0], None), ([8, 8, 8], [0, 1, 0], None),
                             ([8, 8, 8], [0, 0, 0], 99)):
        table = case.table.clone()
        if page is not None:
            table[1, 1] = page
        pk, pv, status = case.k.cuda(), case.v.cuda(), _status()
        ub.paged_pool_write(pk, pv, case.layer, k.cuda(), k.cuda(), _i32(cu), _i32(new), table.cuda(), _i32(first), 8,
                            dev_status=status)
        torch.cuda.synchronize()
        assert int(status.item()) == -4
        got = pk.cpu()
        for r in range(3):
            for j in range(8):
                pg, off = case.row(r, j)
                moved = r != 1 or (page is not None and j < 4)
                want = k[8 * r + j] if moved else case.k[case.layer, pg, :, off]
                assert torch.equal(got[case.layer, pg, :, off].view(torch.int16), want.view(torch.int16))


# --------------------------------------------------------------------- evict

def _evict_case(ub, case, budget, sinks, recent, max_len=None):
    pk, pv, w, status = case.k.cuda(), case.v.cuda(), case.weights.cuda(), _status()
    kept, new = ub.paged_evict(pk, pv, w, case.layer, case.table.cuda(), _i32(case.lens),
                               max(case.lens) if max_len is None else max_len, budget, n_sinks=sinks, n_recent=recent,
                               dev_status=status)
    _ok(ub, status)
    wk, wv, ww = case.k.clone(), case.v.clone(), case.weights.clone()
    for r, n in enumerate(case.lens):
        assert int(new[r]) == min(n, budget)
        for h in range(case.Hkv):
            vals = [float(case.weights[case.layer, case.row(r, j)[0], h, case.row(r, j)[1]]) for j in range(n)]
            want = evict64(vals, n, budget, sinks, recent)
            assert kept[r, h].tolist() == want + [-1] * (budget - len(want))
            if n <= budget:
                continue
            for i, j in enumerate(want):
                (pi, oi), (pj, oj) = case.row(r, i), case.row(r, j)
                for t, s in ((wk, case.k), (wv, case.v), (ww, case.weights)):
                    t[case.layer, pi, h, oi] = s[case.layer, pj, h, oj]
    kind = torch.int16 if case.scales is None else torch.uint8
    assert torch.equal(pk.cpu().view(kind), wk.view(kind))
    assert torch.equal(pv.cpu().view(kind), wv.view(kind))
    assert torch.equal(w.cpu().view(torch.int32), ww.view(torch.int32))


@pytest.mark.parametrize("D,Hkv,page,scales", [(32, 1, 1, POW2), (64, 2, 7, None), (128, 2, 64, None), (64, 1, 16, ANY)])
@pytest.mark.parametrize("budget,sinks,recent", [(1, 0, 0), (1, 1, 0), (64, 4, 16), (64, 64, 0), (64, 0, 64), (300, 0, 0)])
def test_evict_matches_plain(ub, D, Hkv, page, scales, budget, sinks, recent):
    case = PagedCase(30 + D, [0, 1, 64, 65, 129, 400], Hkv, D, page, scales=scales)
    _evict_case(ub, case, budget, sinks, recent)


@pytest.mark.parametrize("budget,sinks,recent", [(1, 0, 0), (1, 1, 0), (64, 4, 16), (64, 64, 0), (64, 0, 64), (300, 0, 0)])
def test_evict_in_the_larger_block(ub, budget, sinks, recent):
    """The same lengths where max_len asks for the larger selection block, and lengths on both sides of it."""
    case = PagedCase(36, [0, 1, 64, 65, 129, 400, 1024], 2, 32, 48, width=30)
    _evict_case(ub, case, budget, sinks, recent, max_len=1400)
    for n in (512, 513):
        _evict_case(ub, PagedCase(37, [n, 7], 1, 32, 16), budget, sinks, recent)


def test_evict_ties_zeros_and_odd_weights(ub):
    """Equal weights go to the lowest row; -0 is 0, negatives and infinities are ordered, NaN leaves first."""
    case = PagedCase(40, [500, 500, 500, 500], 1, 32, 16)
    for r, n in enumerate(case.lens):
        for j in range(n):
            pg, off = case.row(r, j)
            w = [0.25, float(j % 3), -0.0 if j % 2 else 0.0, [float("nan"), -1.0, float("inf"), -float("inf"), 1e-42][j % 5]][r]
            case.weights[case.layer, pg, 0, off] = w
    for budget, sinks, recent in ((100, 3, 7), (450, 0, 1)):
        _evict_case(ub, case, budget, sinks, recent)


def test_evict_beyond_the_shared_memory_copy(ub):
    """More rows than the selection's shared-memory copy holds (49152): the keys are read again from the pool."""
    n = 50000
    g = torch.Generator().manual_seed(41)
    pk = torch.randn(1, 60, 1, 1000, 32, generator=g).to(torch.bfloat16).cuda()
    pv = torch.randn(1, 60, 1, 1000, 32, generator=g).to(torch.bfloat16).cuda()
    w = (torch.rand(1, 60, 1, 1000, generator=g) * 5000).floor().cuda()      # many ties
    table = torch.randperm(60, generator=g)[:50].to(torch.int32).reshape(1, 50)
    flat = w.cpu()[0, table[0].long(), 0].reshape(-1)
    rows = pk.cpu()[0, table[0].long(), 0].reshape(-1, 32)
    kept, new = ub.paged_evict(pk, pv, w, 0, table.cuda(), _i32([n]), n, 30000, n_sinks=2, n_recent=100)
    want = torch.tensor(evict64(flat.tolist(), n, 30000, 2, 100))
    assert torch.equal(kept[0, 0].cpu().long(), want) and int(new[0]) == 30000
    got = pk.cpu()[0, table[0].long(), 0].reshape(-1, 32)
    assert torch.equal(got[:30000], rows[want]) and torch.equal(got[30000:], rows[30000:])
    assert torch.equal(w.cpu()[0, table[0].long(), 0].reshape(-1)[:30000], flat[want])


def test_evict_rejects_bad_lengths_and_pages(ub):
    case = PagedCase(42, [40, 40, 40], 1, 32, 8)
    for what in ("page", "negative", "long"):
        table, n = case.table.clone(), [40, 40, 40]
        if what == "page":
            table[1, 4] = -1
        else:
            n[1] = -1 if what == "negative" else 41
        pk, pv, w, status = case.k.cuda(), case.v.cuda(), case.weights.cuda(), _status()
        kept, new = ub.paged_evict(pk, pv, w, case.layer, table.cuda(), _i32(n), 40, 10, dev_status=status)
        torch.cuda.synchronize()
        assert int(status.item()) == -4 and new.tolist() == [10, -1, 10]
        assert (kept[1] == -1).all() and (kept[0] >= 0).all()
        for j in range(40):
            pg, off = case.row(1, j)
            assert torch.equal(pk[case.layer, pg, :, off].cpu(), case.k[case.layer, pg, :, off])
            assert torch.equal(w[case.layer, pg, :, off].cpu(), case.weights[case.layer, pg, :, off])

"""Paged pools whose planes pass 2^32 bytes, and captured writes and evictions.

Tolerances as in tests/test_gpu_paged.py."""

import pytest
import torch

pytestmark = pytest.mark.gpu

ROUND, SCORE = 2.0 ** -8, 2.0 ** -12


@pytest.fixture(scope="module")
def ub():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from kv_cache_reuse_falcon_b200 import binding
    return binding


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _rnd(g, *shape):
    return torch.randn(*shape, generator=g).to(torch.bfloat16)


def _plain(q, k, v):
    """q [H, D], k and v [n, Hkv, D], float64: out, sum of weight * |v|, weights [n, Hkv]."""
    G = q.shape[0] // k.shape[1]
    kk, vv = k.double().repeat_interleave(G, 1), v.double().repeat_interleave(G, 1)
    p = torch.softmax(torch.einsum("hd,nhd->hn", q.double(), kk) / q.shape[1] ** 0.5, 1)
    w = p.reshape(k.shape[1], G, -1).sum(1).T
    return torch.einsum("hn,nhd->hd", p, vv), torch.einsum("hn,nhd->hd", p, vv.abs()), w


def test_rows_behind_four_gigabytes(ub):
    """The plane holds 4.7 GB of each of K and V; the requests' pages lie at both ends of it."""
    S, Hkv, ps, D, H = 36000, 2, 256, 128, 8
    free, _ = torch.cuda.mem_get_info()
    if free < 16 << 30:
        pytest.skip("needs 16 GB")
    g = torch.Generator().manual_seed(21)
    pk = torch.empty((1, S, Hkv, ps, D), dtype=torch.bfloat16, device="cuda")
    pv = torch.empty_like(pk)
    w = torch.empty((1, S, Hkv, ps), device="cuda")
    lens = [700, 1]
    table = _i32([[S - 1, 0, S - 2], [S - 3, -1, -1]])
    k, v, q = _rnd(g, 701, Hkv, D), _rnd(g, 701, Hkv, D), _rnd(g, 2, H, D)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    n = _i32(lens)
    ub.paged_pool_write(pk, pv, 0, k.cuda(), v.cuda(), _i32([0, 700, 701]), n, table, _i32([0, 0]), 700, key_weights=w,
                        dev_status=status)
    assert torch.equal(pk[0, S - 2, :, :188].cpu(), k[512:700].transpose(0, 1))
    assert torch.equal(pv[0, S - 1].cpu(), v[:256].transpose(0, 1))
    out = ub.paged_decode_attn(q.cuda(), table, n, pk, pv, 0, 768, key_weights=w, dev_status=status).cpu().double()
    got = torch.cat([w[0, p, :, :m] for p, m in ((S - 1, 256), (0, 256), (S - 2, 188))], 1).T.cpu().double()
    ref, mag, want = _plain(q[0], k[:700], v[:700])
    assert ((out[0] - ref).abs() <= mag * (ROUND + SCORE) + 1e-6).all()
    assert ((got - want).abs() <= want * (SCORE + 2.0 ** -22) + 1e-7).all()
    kept, fewer = ub.paged_evict(pk, pv, w, 0, table, n, 768, 300, 2, 50, dev_status=status)
    assert fewer.tolist() == [300, 1]
    rows = kept[0].cpu().long()
    for h in range(Hkv):
        have = torch.cat([pk[0, S - 1, h], pk[0, 0, h, :44]]).cpu()
        assert torch.equal(have, k[rows[h], h])
        top = got[2:650, h].topk(248).indices.sort().values + 2
        assert rows[h].tolist() == [0, 1] + top.tolist() + list(range(650, 700))
    assert int(status.item()) == 0


def test_captured_write_and_eviction_replay_on_changed_rows(ub):
    """One graph of write, decode and eviction, replayed on other rows and lengths, gives the eager bits."""
    S, Hkv, ps, D, H = 24, 2, 16, 64, 8
    g = torch.Generator().manual_seed(22)
    table = _i32(torch.randperm(S, generator=g)[:20].reshape(2, 10).tolist())
    k, v, q = (torch.empty(160, Hkv, D, dtype=torch.bfloat16, device="cuda"),
               torch.empty(160, Hkv, D, dtype=torch.bfloat16, device="cuda"),
               torch.empty(2, H, D, dtype=torch.bfloat16, device="cuda"))
    cu, new, first = _i32([0, 100, 160]), _i32([100, 60]), _i32([0, 0])

    def state():
        return [torch.zeros((1, S, Hkv, ps, D), dtype=torch.bfloat16, device="cuda"),
                torch.zeros((1, S, Hkv, ps, D), dtype=torch.bfloat16, device="cuda"),
                torch.zeros((1, S, Hkv, ps), device="cuda"), torch.empty((2, H, D), device="cuda"),
                torch.zeros((2, Hkv, 40), dtype=torch.int32, device="cuda"), _i32([0, 0])]

    ws = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")

    def step(s):
        ub.paged_pool_write(s[0], s[1], 0, k, v, cu, new, table, first, 160, key_weights=s[2])
        ub.paged_decode_attn(q, table, new, s[0], s[1], 0, 160, key_weights=s[2], out=s[3], workspace=ws)
        ub.paged_evict(s[0], s[1], s[2], 0, table, new, 160, 40, 4, 8, kept=s[4], new_lens=s[5])

    def fill():
        for x in (k, v, q):
            x.copy_(torch.randn(x.shape, generator=g))

    fill()
    mine, graph = state(), torch.cuda.CUDAGraph()
    step(mine)
    with torch.cuda.graph(graph):
        step(mine)
    eager = state()
    step(eager)
    for lens in ([100, 60], [40, 41], [0, 1], [96, 60]):
        fill()
        new.copy_(_i32(lens))
        step(eager)
        graph.replay()
        for a, b in zip(mine, eager):
            assert torch.equal(a, b)


def test_a_dominant_own_key_does_not_hide_a_nan_value(ub):
    """A weight that underflows to zero times a NaN value is NaN, as in the plain form."""
    q = torch.full((1, 1, 32), 16.0, dtype=torch.bfloat16, device="cuda")
    pk = torch.full((1, 1, 1, 16, 32), -16.0, dtype=torch.bfloat16, device="cuda")
    pv = torch.ones_like(pk)
    own = torch.full((1, 1, 32), 16.0, dtype=torch.bfloat16, device="cuda")
    args = (q, _i32([[0]]), _i32([5]), pk, pv, 0, 16)
    out = ub.paged_decode_attn(*args, k_self=own, v_self=own)
    assert (out == 16).all()
    pv[0, 0, 0, 2, 7] = float("nan")
    out = ub.paged_decode_attn(*args, k_self=own, v_self=own)
    assert torch.isnan(out[0, 0, 7]) and (out[0, 0, :7] == 16).all()


def test_calls_on_an_empty_cache(ub):
    """No page yet (a page table of no columns): the own value, zeros without one, and nothing to evict."""
    g = torch.Generator().manual_seed(23)
    pk = torch.full((1, 4, 2, 16, 64), float("nan"), dtype=torch.bfloat16, device="cuda")
    pv, w = pk.clone(), torch.zeros((1, 4, 2, 16), device="cuda")
    table, lens = torch.empty((3, 0), dtype=torch.int32, device="cuda"), _i32([0, 0, 0])
    q, own = _rnd(g, 3, 4, 64).cuda(), _rnd(g, 3, 2, 64).cuda()
    for weights in (None, w):
        out = ub.paged_decode_attn(q, table, lens, pk, pv, 0, 0, k_self=own, v_self=own, key_weights=weights)
        assert torch.equal(out, own.float().repeat_interleave(2, 1))
        assert (ub.paged_decode_attn(q, table, lens, pk, pv, 0, 0, key_weights=weights) == 0).all()
    kept, fewer = ub.paged_evict(pk, pv, w, 0, table, lens, 0, 5)
    assert (kept == -1).all() and fewer.tolist() == [0, 0, 0] and (w == 0).all()


def test_decode_of_requests_that_share_pages(ub):
    """A common prefix in the same pages: both requests read it, and its weights are the sum of theirs."""
    g = torch.Generator().manual_seed(24)
    Hkv, ps, D, H = 2, 16, 64, 4
    pk, pv = _rnd(g, 1, 8, Hkv, ps, D), _rnd(g, 1, 8, Hkv, ps, D)
    table, lens, q = [[5, 2, 7], [5, 2, 0]], [40, 33], _rnd(g, 2, H, D)
    w = torch.zeros((1, 8, Hkv, ps), device="cuda")
    out = ub.paged_decode_attn(q.cuda(), _i32(table), _i32(lens), pk.cuda(), pv.cuda(), 0, 48, key_weights=w)
    want = torch.zeros((8, Hkv, ps), dtype=torch.float64)
    for r in range(2):
        k = torch.cat([pk[0, p] for p in table[r]], 1)[:, :lens[r]].transpose(0, 1)
        v = torch.cat([pv[0, p] for p in table[r]], 1)[:, :lens[r]].transpose(0, 1)
        ref, mag, wt = _plain(q[r], k, v)
        assert ((out[r].cpu().double() - ref).abs() <= mag * (ROUND + SCORE) + 1e-6).all()
        for j in range(lens[r]):
            want[table[r][j // ps], :, j % ps] += wt[j]
    assert ((w[0].cpu().double() - want).abs() <= want * (SCORE + 2.0 ** -22) + 1e-7).all()

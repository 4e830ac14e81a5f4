"""Refusals of the paged and windowed calls that need no device: argument errors of the C entry points are
found before any CUDA call, and the binding refuses tensors that do not fit before it calls them."""

import ctypes

import pytest
import torch


@pytest.fixture(scope="module")
def ub():
    from kv_cache_reuse_falcon_b200 import build
    build.build()
    from kv_cache_reuse_falcon_b200 import binding
    return binding


INVALID, UNSUPPORTED, MISALIGNED, RANGE = -1, -2, -3, -4
A = 0x10000   # an aligned address that is never read


def _pool(ub, L=2, S=4, H=2, n_cap=16, D=64, dtype=0, ks=1.0, vs=1.0, k=A, v=A):
    return ub.KVPool(k, v, L, S, H, n_cap, D, dtype, ks, vs)


def _write(ub, pool, layer=0, k=A, v=A, cu=A, new=A, table=A, pages=4, first=A, B=2, max_new=8, T=16):
    return ub.LIB.unipin_paged_pool_write(ctypes.byref(pool) if pool else None, layer, k, v, cu, new, table, pages, first,
                                          B, max_new, T, None, None, None)


def _decode(ub, pool, q=A, ks=None, vs=None, out=A, table=A, pages=4, lens=A, R=2, H=4, D=64, max_len=32, window=8,
            sinks=0, scale=0.1, layer=0, weights=None, ws=None, ws_bytes=0):
    return ub.LIB.unipin_paged_decode_attn(q, ks, vs, out, 1, table, pages, lens, R, H, D, max_len, window, sinks, scale,
                                           ctypes.byref(pool) if pool else None, layer, weights, ws, ws_bytes, None, None)


def _evict(ub, pool, layer=0, w=A, table=A, pages=4, lens=A, R=2, max_len=32, budget=8, sinks=0, recent=0, kept=A,
           new=A + 64):
    return ub.LIB.unipin_paged_evict(ctypes.byref(pool) if pool else None, layer, w, table, pages, lens, R, max_len,
                                     budget, sinks, recent, kept, new, None, None)


@pytest.mark.parametrize("pool,want", [
    (dict(D=48), UNSUPPORTED), (dict(layer=2), RANGE), (dict(layer=-1), RANGE), (dict(n_cap=0), INVALID),
    (dict(H=0), INVALID), (dict(k=None), INVALID), (dict(k=A + 8), MISALIGNED), (dict(dtype=2), INVALID),
    (dict(dtype=1, ks=0.0), INVALID), (dict(dtype=1, vs=float("inf")), INVALID), (dict(dtype=1, ks=float("nan")), INVALID),
    (dict(S=1 << 20, H=2, n_cap=1 << 11), UNSUPPORTED),    # 2^32 rows in a layer
])
def test_bad_pools_are_refused_by_every_call(ub, pool, want):
    layer = pool.pop("layer", 0)
    p = _pool(ub, **pool)
    assert _write(ub, p, layer) == want
    assert _evict(ub, p, layer) == want
    assert _decode(ub, p, layer=layer, D=p.D, H=4) == want


def test_write_refusals(ub):
    p = _pool(ub)
    assert _write(ub, None) == INVALID
    for bad in (dict(B=-1), dict(max_new=-1), dict(T=-1), dict(pages=-1), dict(k=None), dict(v=None), dict(cu=None),
                dict(new=None), dict(table=None), dict(first=None), dict(pages=0), dict(B=65536)):
        assert _write(ub, p, **bad) == INVALID, bad
    assert _write(ub, p, max_new=65) == RANGE              # more rows than four pages of 16 hold
    assert _write(ub, p, k=A + 2) == MISALIGNED
    for nothing in (dict(B=0), dict(max_new=0), dict(T=0)):
        assert _write(ub, p, k=None, **nothing) == 0


def test_decode_refusals(ub):
    p = _pool(ub)
    assert _decode(ub, None) == INVALID
    for bad in (dict(R=-1), dict(H=0), dict(H=3), dict(max_len=-1), dict(window=0), dict(sinks=-1), dict(scale=0.0),
                dict(scale=float("nan")), dict(D=32), dict(ks=A), dict(vs=A), dict(q=None), dict(out=None),
                dict(table=None), dict(lens=None), dict(R=65536)):
        assert _decode(ub, p, **bad) == INVALID, bad
    assert _decode(ub, p, D=40) == UNSUPPORTED
    assert _decode(ub, p, max_len=65) == RANGE
    for bad in (dict(q=A + 8), dict(out=A + 4), dict(ks=A + 8, vs=A), dict(ws=A + 8, ws_bytes=1 << 20)):
        assert _decode(ub, p, **bad) == MISALIGNED, bad
    assert _decode(ub, p, R=0, q=None) == 0
    size = ub.LIB.unipin_paged_decode_workspace_size
    assert size(ctypes.byref(p), 2, 4, 32, 8, 0, 0) == 0             # short rows stay in one block
    assert size(ctypes.byref(p), 2, 4, 32, 8, 0, 1) > 0              # collected weights need the scores
    big = _pool(ub, S=1000, n_cap=64)
    assert size(ctypes.byref(big), 2, 4, 60000, 2 ** 31 - 1, 0, 0) > 0
    assert size(ctypes.byref(big), 2, 4, 60000, 100, 4, 0) == 0      # under a window few rows are visible
    assert size(ctypes.byref(p), 2, 3, 32, 8, 0, 0) == 0 and size(None, 2, 4, 32, 8, 0, 0) == 0


def test_evict_refusals(ub):
    p = _pool(ub)
    assert _evict(ub, None) == INVALID
    for bad in (dict(R=-1), dict(max_len=-1), dict(budget=0), dict(sinks=-1), dict(recent=-1), dict(sinks=5, recent=4),
                dict(w=None), dict(table=None), dict(lens=None), dict(kept=None), dict(new=None), dict(new=A, lens=A),
                dict(R=65536)):
        assert _evict(ub, p, **bad) == INVALID, bad
    assert _evict(ub, p, max_len=65) == RANGE
    assert _evict(ub, p, R=0, w=None) == 0


def _prefill(ub, q=A, k=A, v=A, out=A, lse=None, cu=A, past=A, B=2, H=4, Hkv=2, D=64, max_len=16, T=20, window=8, sinks=0,
             scale=0.1):
    return ub.LIB.unipin_windowed_prefill_attn(q, k, v, out, 1, lse, cu, past, B, H, Hkv, D, max_len, T, window, sinks,
                                               scale, None, None)


def _bwd(ub, ptrs=None, ws=A, ws_bytes=1 << 30, B=2, H=4, Hkv=2, D=64, max_len=16, T=20, window=8, sinks=0, scale=0.1, cu=A):
    p = dict(q=A, k=A, v=A, out=A, dout=A, lse=A, dq=A, dk=A, dv=A)
    p.update(ptrs or {})
    return ub.LIB.unipin_windowed_prefill_bwd(p["q"], p["k"], p["v"], p["out"], p["dout"], p["lse"], p["dq"], p["dk"],
                                              p["dv"], 1, cu, A, B, H, Hkv, D, max_len, T, window, sinks, scale, ws,
                                              ws_bytes, None, None)


def test_windowed_refusals(ub):
    for call in (_prefill, _bwd):
        for bad in (dict(B=-1), dict(H=0), dict(Hkv=0), dict(H=3), dict(max_len=-1), dict(T=-1), dict(window=0),
                    dict(sinks=-1), dict(scale=0.0), dict(scale=float("inf")), dict(cu=None)):
            assert call(ub, **bad) == INVALID, (call, bad)
        assert call(ub, D=48) == UNSUPPORTED
        for nothing in (dict(B=0), dict(T=0), dict(max_len=0)):
            assert call(ub, **nothing) == 0
    for bad in (dict(q=None), dict(k=None), dict(v=None), dict(out=None), dict(past=None)):
        assert _prefill(ub, **bad) == INVALID
    for bad in (dict(q=A + 8), dict(out=A + 4), dict(lse=A + 2)):
        assert _prefill(ub, **bad) == MISALIGNED
    for name in ("q", "k", "v", "out", "dout", "lse", "dq", "dk", "dv"):
        assert _bwd(ub, {name: None}) == INVALID
        assert _bwd(ub, {name: A + 2}) == MISALIGNED
    need = ub.windowed_prefill_bwd_workspace_size(2, 4, 2, 64, 16, 20, 8, 0)
    assert need > 0 and _bwd(ub, ws_bytes=need - 1) == INVALID and _bwd(ub, ws=None) == INVALID
    assert _bwd(ub, B=65536, T=0) == 0 and _bwd(ub, B=65536, ws_bytes=1 << 40) == INVALID


def test_binding_refuses_tensors_that_do_not_fit(ub):
    bf = torch.bfloat16
    q, kv = torch.zeros(20, 4, 64, dtype=bf), torch.zeros(20, 2, 64, dtype=bf)
    cu, past = torch.zeros(3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    good = [q, kv, kv, cu, past, 16, 8]
    bad = {0: [q.float(), q[:, :, 0], q.transpose(0, 1)], 1: [kv[:19], kv.half(), kv[:, :, :32]], 2: [kv[:, :1]],
           3: [cu[:2], cu.long(), cu[None]], 4: [past.float(), past[None]], 6: [0, -1]}
    for i, values in bad.items():
        for x in values:
            with pytest.raises(ValueError):
                ub.windowed_prefill_attn(*[x if j == i else y for j, y in enumerate(good)])
    with pytest.raises(ValueError, match="CUDA device"):
        ub.windowed_prefill_attn(*good)                              # tensors on the CPU
    with pytest.raises(ValueError):
        ub.windowed_prefill_attn(*good, n_sinks=-1)
    with pytest.raises(ValueError):
        ub.windowed_prefill_attn(*good, lse=torch.zeros(20, 2))
    with pytest.raises(ValueError):
        ub.windowed_prefill_attn(*good, out=torch.zeros(20, 4, 64, dtype=bf))   # out_fp32 is the default
    with pytest.raises(ValueError):
        ub.windowed_prefill_bwd(q, kv, kv, q, q[:19], torch.zeros(20, 4), cu, past, 16, 8)
    with pytest.raises(ValueError):
        ub.windowed_prefill_bwd(q, kv, kv, q, q, torch.zeros(20, 4), cu, past, 16, 8, dq=torch.zeros(20, 4, 64, dtype=bf))
    pool = torch.zeros(1, 4, 2, 16, 64, dtype=bf)
    with pytest.raises(ValueError):
        ub.paged_pool_write(pool, pool, 0, kv, kv, cu, past, past[:, None], past, 8)   # (a pool on the CPU)
    for f in (ub.paged_decode_attn, ub.paged_evict):
        with pytest.raises(ValueError):
            f(pool, pool, None, 0, past[:, None], past, 16, 8)


def test_sizes_beyond_the_kernels_numbers_are_refused(ub):
    p = _pool(ub, H=16384, S=1, n_cap=1024)
    assert _decode(ub, p, H=16384, R=65535, max_len=100, window=100, pages=1) == INVALID   # units of 31 bits
    one = _pool(ub, H=1, S=64, n_cap=64)
    assert _decode(ub, one, H=8193, weights=A, ws=A, ws_bytes=1 << 40) == UNSUPPORTED   # heads that share weights
    wide = _pool(ub, H=1 << 28, S=1, n_cap=1)
    assert _write(ub, wide, max_new=1, pages=1) == INVALID                           # vectors of a token
    assert _evict(ub, _pool(ub, n_cap=1 << 20, S=8), pages=2000, max_len=(1 << 30) + 1) == INVALID
    assert _decode(ub, _pool(ub, n_cap=1 << 20, S=8), pages=2000, max_len=(1 << 30) + 1) == INVALID

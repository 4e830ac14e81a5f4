"""Timed cases of the paged-cache and sliding-window operators.

Five operators of one serving and training path: histories written into the
pages of a cache pool, one new token per request attending over its pages
(with an optional sliding window, first rows that stay visible, and the
attention weight each cached row collects), eviction of the rows that
collected least, and the sliding-window prefill with its gradients.

``run`` computes an operator in its plain form (elementary torch operations in
float32) or, where ``own`` is true, calls the package's kernels; both take what
``prepare`` made.  ``exact`` is the same from the definition in float64.
"""

import math

import torch

own = False

LAYER, LAYERS = 0, 1


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # -- paged_pool_write: K/V rows of a ragged batch into the requests' pages
        # one new token of each of 32 requests appended after a decode step
        dict(name="write_append_R32", op="write", B=32, n_lo=1, n_hi=1, first_hi=2000, Hkv=8, D=64, page=64,
             e4m3=False, scale_exp=0),
        # the histories of 256 users (ragged, up to 4096 rows) after a prefill, into an E4M3 pool
        dict(name="write_history_e4m3_B256", op="write", B=256, n_lo=32, n_hi=4096, first_hi=0, Hkv=8, D=128,
             page=128, e4m3=True, scale_exp=-6),
        # -- paged_decode_attn: one new token per request over its pages
        # a single request, short history: the latency of a call
        dict(name="decode_R1_n500", op="decode", R=1, n_lo=500, n_hi=500, H=8, Hkv=8, D=64, page=16, e4m3=False,
             scale_exp=0, window=0, sinks=0, self_key=True, weights=False),
        # the retrieval stage's one-token step over 32 requests' histories
        dict(name="decode_R32_n2048", op="decode", R=32, n_lo=1024, n_hi=2048, H=8, Hkv=8, D=64, page=64, e4m3=False,
             scale_exp=0, window=0, sinks=0, self_key=True, weights=False),
        # long histories, grouped heads, collecting each row's attention weight for eviction
        dict(name="decode_weights_R8_n32768", op="decode", R=8, n_lo=777, n_hi=32768, H=8, Hkv=2, D=128, page=64,
             e4m3=False, scale_exp=0, window=0, sinks=0, self_key=False, weights=True),
        # a large batch under a window with first rows kept, E4M3 codes
        dict(name="decode_window_e4m3_R256", op="decode", R=256, n_lo=32, n_hi=4096, H=8, Hkv=8, D=128, page=128,
             e4m3=True, scale_exp=-6, window=1024, sinks=4, self_key=True, weights=False),
        # -- paged_evict: the rows with the least collected weight leave
        # one request down to half its rows
        dict(name="evict_R1_n1000", op="evict", R=1, n_lo=1000, n_hi=1000, Hkv=8, D=64, page=16, e4m3=False,
             budget=500, sinks=4, recent=64),
        # a batch of long histories down to 2048 rows each
        dict(name="evict_R32_n8192", op="evict", R=32, n_lo=1500, n_hi=8192, Hkv=8, D=128, page=64, e4m3=False,
             budget=2048, sinks=4, recent=256),
        # -- windowed_prefill_attn: [past || candidates] under a window with first rows kept
        # a small serving batch
        dict(name="prefill_B2_n300", op="prefill", B=2, n_lo=200, n_hi=300, k_lo=16, k_hi=20, H=8, Hkv=8, D=64,
             window=128, sinks=4),
        # long ragged histories with their candidates
        dict(name="prefill_B16_n2048", op="prefill", B=16, n_lo=500, n_hi=2048, k_lo=50, k_hi=256, H=8, Hkv=8, D=128,
             window=512, sinks=4),
        # -- windowed_prefill_attn with windowed_prefill_bwd: a training step's attention
        dict(name="train_B64_n256", op="train", B=64, n_lo=256, n_hi=256, k_lo=128, k_hi=128, H=8, Hkv=8, D=64,
             window=128, sinks=1),
        dict(name="train_gqa_B8_n1500", op="train", B=8, n_lo=700, n_hi=1500, k_lo=50, k_hi=130, H=8, Hkv=2, D=128,
             window=300, sinks=16),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["write", "decode", "decode", "evict", "prefill", "train"])
    D = rng.choice([32, 64, 128])
    Hkv, G = rng.choice([(8, 1), (2, 4), (1, 8), (3, 2), (4, 3), (8, 2), (1, 16)])
    page = rng.choice([1, 7, 16, 32, 48, 64, 100, 128, 256])
    e4m3 = rng.random() < 0.4
    scale_exp = rng.choice([-7, -6, -5]) if e4m3 else 0
    if op in ("write", "decode", "evict"):
        R = _log_int(rng, 1, 256)
        # the rows of all requests stay within the largest listed case's
        most = min(32768, max(2, 400000 // (R * Hkv)))
        n_hi = _log_int(rng, 2, most)
        n_lo = rng.randint(0 if op == "decode" else 1, n_hi)
    if op == "write":
        return dict(op=op, B=R, n_lo=n_lo, n_hi=n_hi, first_hi=rng.choice([0, 0, 5, 300]), Hkv=Hkv, D=D, page=page,
                    e4m3=e4m3, scale_exp=scale_exp)
    if op == "decode":
        return dict(op=op, R=R, n_lo=n_lo, n_hi=n_hi, H=Hkv * G, Hkv=Hkv, D=D, page=page, e4m3=e4m3,
                    scale_exp=scale_exp, window=rng.choice([0, 0, _log_int(rng, 1, n_hi)]),
                    sinks=rng.choice([0, 0, 1, 4, 70]), self_key=rng.random() < 0.5, weights=rng.random() < 0.4)
    if op == "evict":
        budget = _log_int(rng, 1, n_hi)
        sinks = min(rng.choice([0, 1, 4]), budget)
        return dict(op=op, R=R, n_lo=n_lo, n_hi=n_hi, Hkv=Hkv, D=D, page=page, e4m3=e4m3, budget=budget, sinks=sinks,
                    recent=rng.randint(0, budget - sinks))
    B = _log_int(rng, 1, 16)
    H = Hkv * G
    most = int(min(2048, math.sqrt(3.0e8 / (B * H)))) if op == "prefill" else int(min(1500, math.sqrt(1.0e8 / (B * H))))
    n_hi = _log_int(rng, 8, most)
    k_hi = _log_int(rng, 1, max(2, most // 8))
    return dict(op=op, B=B, n_lo=rng.randint(0, n_hi), n_hi=n_hi, k_lo=rng.randint(0, k_hi), k_hi=k_hi, H=H, Hkv=Hkv,
                D=D, window=_log_int(rng, 1, 2 * n_hi), sinks=rng.choice([0, 1, 4, 16, 100]))


# ------------------------------------------------------------------- geometry

def _spread(lo, hi, count, turn=0.0):
    """`count` lengths between lo and hi, the first of them hi: a fixed low-discrepancy sequence."""
    return [hi if i == 0 else lo + int((hi - lo) * ((i * 0.6180339887 + turn) % 1.0) + 0.5) for i in range(count)]


def _cu(lens):
    at, cu = 0, [0]
    for n in lens:
        at += n
        cu.append(at)
    return cu


def _rows(case):
    """Rows of each request in the cache (write: rows written)."""
    return _spread(case["n_lo"], case["n_hi"], case.get("R") or case["B"])


def _first(case):
    hi = case["first_hi"]
    return [int(hi * ((i * 0.7548776662 + 0.3) % 1.0)) for i in range(case["B"])]


def _segments(case):
    past = _spread(case["n_lo"], case["n_hi"], case["B"])
    cand = _spread(case["k_lo"], case["k_hi"], case["B"], 0.5)
    return past, cand


def _visible(n, window, sinks, own_key):
    """Cached rows that the token after n rows sees (its own key apart)."""
    if window == 0:
        return n
    pos = n if own_key else n - 1
    lo = max(0, pos - window + 1)
    return n - lo + min(sinks, lo)


def _pairs(n, k, window, sinks):
    """Allowed (row, key) pairs of a segment of n past rows and k candidates."""
    total = 0
    edge = min(n, window)
    total += edge * (edge + 1) // 2                     # rows whose window reaches row 0
    rest = n - edge
    total += rest * window
    # sinks below the window of rows i >= window: lo = i - window + 1 = 1 .. rest
    a = min(sinks, rest)
    total += a * (a + 1) // 2 + (rest - a) * a if sinks else 0
    lo = max(0, n - window + 1)
    total += k * (n - lo + min(sinks, lo) + 1)
    return total


def work(case):
    D, Hkv = case["D"], case["Hkv"]
    if case["op"] == "write":
        rows = sum(_rows(case))
        return {"bytes": rows * Hkv * D * 2 * (2 + (1 if case["e4m3"] else 2)), "flops": 0}
    if case["op"] == "decode":
        H, R = case["H"], case["R"]
        vis = sum(_visible(n, case["window"], case["sinks"], case["self_key"]) for n in _rows(case))
        b = vis * Hkv * D * 2 * (1 if case["e4m3"] else 2) + R * H * D * 4
        b += R * Hkv * D * 4 if case["self_key"] else 0
        b += vis * Hkv * 8 if case["weights"] else 0
        return {"bytes": b, "flops": 4 * D * H * (vis + (R if case["self_key"] else 0))}
    if case["op"] == "evict":
        gone = [n for n in _rows(case) if n > case["budget"]]
        elt = 1 if case["e4m3"] else 2
        kept = len(gone) * case["budget"] * Hkv
        return {"bytes": sum(gone) * Hkv * 4 + kept * (2 * 2 * D * elt + 8) + case["R"] * Hkv * case["budget"] * 4,
                "flops": 0}
    past, cand = _segments(case)
    T, H = sum(past) + sum(cand), case["H"]
    pairs = sum(_pairs(n, k, case["window"], case["sinks"]) for n, k in zip(past, cand))
    fwd = T * (2 * H + 2 * Hkv) * D * 2 + T * H * 4
    if case["op"] == "prefill":
        return {"bytes": fwd, "flops": 4 * D * H * pairs}
    # the backward reads q, k, v, out, dout and the row statistic and writes dq, dk, dv
    bwd = T * (4 * H + 4 * Hkv) * D * 2 + T * H * 4
    return {"bytes": fwd + bwd, "flops": 14 * D * H * pairs}


# --------------------------------------------------------------------- inputs

def _pages(case, lens, g):
    """A page table [R, max pages] of distinct pages in random order (-1 where a request has none) and the page count."""
    ps = case["page"]
    need = torch.tensor([(n + ps - 1) // ps for n in lens], device="cuda")
    width = max(1, int(need.max()))
    total = int(need.sum())
    order = torch.randperm(total + 3, generator=g, device="cuda").to(torch.int32)
    at = torch.cumsum(need, 0) - need
    col = torch.arange(width, device="cuda")
    table = torch.where(col[None] < need[:, None], order[(at[:, None] + col[None]).clamp(max=total + 2)],
                        torch.full((), -1, dtype=torch.int32, device="cuda"))
    return table.contiguous(), total + 3


def _pool(case, pages, g, rows):
    """K and V pools: random rows where the cache holds something, zeros where it is only written to."""
    shape = (LAYERS, pages, case["Hkv"], case["page"], case["D"])
    out = []
    for _ in range(2):
        if not rows:
            t = torch.zeros(shape, dtype=torch.bfloat16, device="cuda")
        else:
            t = torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)
        if case["e4m3"]:
            inv = 2.0 ** -case.get("scale_exp", -6)
            # in place in bfloat16: a power of two, so exact before the rounding to codes
            t = t.mul_(inv).clamp_(-448, 448).to(torch.float8_e4m3fn)
        out.append(t)
    return out


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _randn(shape, g):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    D, Hkv = case["D"], case["Hkv"]
    s = {"case": case, "op": case["op"]}
    if case["op"] in ("write", "decode", "evict"):
        scale = 2.0 ** case.get("scale_exp", -6)
        s["scales"] = (scale, scale) if case["e4m3"] else None
    if case["op"] == "write":
        rows, first = _rows(case), _first(case)
        s["table"], pages = _pages(case, [a + n for a, n in zip(first, rows)], g)
        s["pool_k"], s["pool_v"] = _pool(case, pages, g, False)
        s["k"], s["v"] = _randn((sum(rows), Hkv, D), g), _randn((sum(rows), Hkv, D), g)
        s["cu"], s["new"], s["first"] = _i32(_cu(rows)), _i32(rows), _i32(first)
        s["max_new"] = max(rows)
        return s
    if case["op"] in ("decode", "evict"):
        rows = _rows(case)
        s["table"], pages = _pages(case, rows, g)
        s["pool_k"], s["pool_v"] = _pool(case, pages, g, True)
        s["lens"], s["max_len"] = _i32(rows), max(rows)
    if case["op"] == "decode":
        R, H = case["R"], case["H"]
        s["q"] = _randn((R, H, D), g)
        s["k"], s["v"] = (_randn((R, Hkv, D), g), _randn((R, Hkv, D), g)) if case["self_key"] else (None, None)
        s["weights"] = None
        if case["weights"]:   # what earlier steps collected
            s["weights"] = torch.rand((LAYERS, pages, Hkv, case["page"]), generator=g, device="cuda")
        s["out"] = torch.empty((R, H, D), dtype=torch.bfloat16, device="cuda")
        s["ws"] = {}
        return s
    if case["op"] == "evict":
        # heavy-tailed weights, a share of them equal (rows that collected nothing yet)
        shape = (LAYERS, pages, Hkv, case["page"])
        w = torch.randn(shape, generator=g, device="cuda").mul_(2.0).exp_()
        s["weights"] = w.mul_((torch.rand(shape, generator=g, device="cuda") < 0.8).float())
        s["ws"] = {}
        return s
    past, cand = _segments(case)
    lens = [n + k for n, k in zip(past, cand)]
    T, H = sum(lens), case["H"]
    s["q"], s["k"], s["v"] = _randn((T, H, D), g), _randn((T, Hkv, D), g), _randn((T, Hkv, D), g)
    s["cu"], s["past"], s["max_seqlen"] = _i32(_cu(lens)), _i32(past), max(lens)
    s["out"] = torch.empty((T, H, D), dtype=torch.bfloat16, device="cuda")
    s["lse"] = torch.empty((T, H), dtype=torch.float32, device="cuda")
    s["ws"] = {}
    if case["op"] == "train":
        s["dout"] = _randn((T, H, D), g)
    return s


# ---------------------------------------------------------------- plain forms

def _gather(pool, scale, table, cols, page):
    """Rows [R, n, Hkv, D] of a pool layer in float32, row j of request r from its page table."""
    at = table[:, cols // page].clamp(min=0).long()
    off = (cols % page)[None]
    if scale is None:
        return pool[LAYER][at, :, off].float()
    x = pool.view(torch.uint8)[LAYER][at, :, off].view(torch.float8_e4m3fn)
    return (x.float() * scale).to(torch.bfloat16).float()


def _plain_write(s):
    c = s["case"]
    seg = torch.repeat_interleave(torch.arange(c["B"], device="cuda"), s["new"].long())
    row = torch.arange(seg.numel(), device="cuda") - s["cu"].long()[seg] + s["first"].long()[seg]
    page, off = s["table"][seg, row // c["page"]].long(), row % c["page"]
    for pool, x, i in ((s["pool_k"], s["k"], 0), (s["pool_v"], s["v"], 1)):
        if s["scales"] is not None:
            x = (x.float() * (1.0 / s["scales"][i])).clamp(-448, 448).to(torch.float8_e4m3fn)
            pool.view(torch.uint8)[LAYER][page, :, off] = x.view(torch.uint8)
        else:
            pool[LAYER][page, :, off] = x
    return {"pool_k": s["pool_k"], "pool_v": s["pool_v"]}


def _plain_decode(s):
    c = s["case"]
    R, H, Hkv, D, page = c["R"], c["H"], c["Hkv"], c["D"], c["page"]
    G = H // Hkv
    cols = torch.arange(s["max_len"], device="cuda")
    ks, vs = s["scales"] or (None, None)
    n = s["lens"].long()[:, None]
    see = cols[None] < n
    if c["window"]:
        pos = n if c["self_key"] else n - 1
        see = see & ((cols[None] > pos - c["window"]) | (cols[None] < c["sinks"]))
    q = s["q"].float().view(R, Hkv, G, D) / math.sqrt(D)
    K = _gather(s["pool_k"], ks, s["table"], cols, page)
    a = torch.einsum("rhgd,rnhd->rhgn", q, K).masked_fill(~see[:, None, None], -math.inf)
    del K
    if c["self_key"]:
        a = torch.cat([a, (q * s["k"].float()[:, :, None]).sum(-1, keepdim=True)], -1)
    top = a.amax(-1, keepdim=True).clamp(min=-1e30)
    e = torch.exp(a - top)
    e = e / e.sum(-1, keepdim=True).clamp(min=1e-30)
    V = _gather(s["pool_v"], vs, s["table"], cols, page)
    out = torch.einsum("rhgn,rnhd->rhgd", e[..., : s["max_len"]], V)
    if c["self_key"]:
        out = out + e[..., -1:] * s["v"].float()[:, :, None]
    got = {"out": out.reshape(R, H, D).to(torch.bfloat16)}
    if c["weights"]:
        add = e[..., : s["max_len"]].sum(2).permute(0, 2, 1)          # [R, n, Hkv]
        at = s["table"][:, cols // page].clamp(min=0).long()
        heads = torch.arange(Hkv, device="cuda")
        s["weights"][LAYER].index_put_((at[:, :, None], heads, (cols % page)[None, :, None]), add, accumulate=True)
        got["weights"] = s["weights"]
    return got


def _plain_evict(s):
    c = s["case"]
    page, budget, Hkv = c["page"], c["budget"], c["Hkv"]
    cols = torch.arange(s["max_len"], device="cuda")
    n = s["lens"].long()[:, None]
    at = s["table"][:, cols // page].clamp(min=0).long()
    off = (cols % page)[None]
    w = s["weights"][LAYER][at, :, off].permute(0, 2, 1)              # [R, Hkv, n]
    w = torch.where(((cols < c["sinks"]) | (cols >= n - c["recent"]))[:, None], math.inf, w)
    w = torch.where((cols >= n)[:, None], -math.inf, w)
    order = torch.sort(w, dim=-1, descending=True, stable=True).indices[..., :budget]
    rows = torch.arange(order.shape[-1], device="cuda")
    new = n.clamp(max=budget)
    order = torch.where(rows < new[:, None], order, s["max_len"])
    order = torch.sort(order, dim=-1).values                          # [R, Hkv, <= budget]
    live = rows < new[:, None]                                        # [R, 1, rows]
    kept = torch.full((c["R"], Hkv, budget), -1, dtype=torch.int32, device="cuda")
    kept[..., : rows.numel()] = torch.where(live, order, -1).to(torch.int32)
    # move row order[i] to row i where the request shrinks (all others keep their place)
    r, h, i = torch.nonzero((live & (n > budget)[:, None]).expand(-1, Hkv, -1), as_tuple=True)
    j = order[r, h, i]
    src = (s["table"][r, j // page].long(), h, j % page)
    dst = (s["table"][r, i // page].long(), h, i % page)
    for t in (s["pool_k"], s["pool_v"], s["weights"]):
        u = t.view(torch.uint8)[LAYER] if c["e4m3"] and t.dim() == 5 else t[LAYER]
        u[dst] = u[src]
    return {"kept": kept, "new_lens": new[:, 0].to(torch.int32), "pool_k": s["pool_k"], "pool_v": s["pool_v"],
            "weights": s["weights"]}


def _plain_attn(s):
    """Dense padded weights [B, H, S, S] in float32, with what the gradients need."""
    c = s["case"]
    D, G, S = c["D"], c["H"] // c["Hkv"], s["max_seqlen"]
    lens = (s["cu"][1:] - s["cu"][:-1]).long()
    seg = torch.repeat_interleave(torch.arange(c["B"], device="cuda"), lens)
    row = torch.arange(seg.numel(), device="cuda") - s["cu"].long()[seg]

    def pad(x, heads):
        y = torch.zeros((c["B"], S, x.shape[1], D), device="cuda")
        y[seg, row] = x.float()
        y = y.permute(0, 2, 1, 3)
        return y if heads == x.shape[1] else y.repeat_interleave(heads // x.shape[1], 1)

    q, k, v = (pad(s[x], c["H"]) for x in "qkv")
    i, j = torch.arange(S, device="cuda")[:, None], torch.arange(S, device="cuda")[None]
    n = s["past"].long()[:, None, None]
    near = (j > torch.minimum(i, n) - c["window"]) | (j < c["sinks"])
    see = torch.where(i < n, (j <= i) & near, ((j < n) & near) | (j == i)) & (i < lens[:, None, None])
    a = torch.matmul(q, k.transpose(-1, -2)).mul_(1.0 / math.sqrt(D)).masked_fill_(~see[:, None], -math.inf)
    top = a.amax(-1, keepdim=True).clamp_(min=-1e30)
    p = a.sub_(top).exp_()
    total = p.sum(-1, keepdim=True).clamp_(min=1e-30)
    p /= total
    o = torch.matmul(p, v)
    lse = ((top + torch.log(total)) * (1.0 / math.log(2.0)))[..., 0].permute(0, 2, 1)[seg, row]
    return seg, row, pad, q, k, v, p, o, lse, G


def _plain_prefill(s):
    seg, row, _, _, _, _, _, o, lse, _ = _plain_attn(s)
    return {"out": o.permute(0, 2, 1, 3)[seg, row].to(torch.bfloat16), "lse": lse}


def _plain_train(s):
    c = s["case"]
    seg, row, pad, q, k, v, p, o, _, G = _plain_attn(s)
    scale = 1.0 / math.sqrt(c["D"])
    g = pad(s["dout"], c["H"])

    def rows(x):
        return x.permute(0, 2, 1, 3)[seg, row].to(torch.bfloat16)

    def group(x):
        return x.view(c["B"], c["Hkv"], G, x.shape[2], c["D"]).sum(2)

    dv = torch.matmul(p.transpose(-1, -2), g)
    ds = torch.matmul(g, v.transpose(-1, -2)).sub_((g * o).sum(-1, keepdim=True)).mul_(p).mul_(scale)
    return {"out": rows(o), "dq": rows(torch.matmul(ds, k)), "dk": rows(group(torch.matmul(ds.transpose(-1, -2), q))),
            "dv": rows(group(dv))}


# ------------------------------------------------------------- the framework

def _own(s):
    from kv_cache_reuse_falcon_b200 import binding as ub
    c, op = s["case"], s["op"]
    if op == "write":
        ub.paged_pool_write(s["pool_k"], s["pool_v"], LAYER, s["k"], s["v"], s["cu"], s["new"], s["table"], s["first"],
                            s["max_new"], pool_scales=s["scales"])
        return {"pool_k": s["pool_k"], "pool_v": s["pool_v"]}
    if op == "decode":
        if "decode" not in s["ws"]:   # kept by a serving loop from call to call
            s["ws"]["decode"] = torch.empty(max(16, ub.paged_decode_workspace_size(
                s["pool_k"], s["pool_v"], c["R"], c["H"], s["max_len"], weights=c["weights"],
                window=c["window"] or None, n_sinks=c["sinks"], pool_scales=s["scales"])), dtype=torch.uint8,
                device="cuda")
        ub.paged_decode_attn(s["q"], s["table"], s["lens"], s["pool_k"], s["pool_v"], LAYER, s["max_len"],
                             k_self=s["k"], v_self=s["v"], window=c["window"] or None, n_sinks=c["sinks"],
                             key_weights=s["weights"], out=s["out"], out_fp32=False, workspace=s["ws"]["decode"],
                             pool_scales=s["scales"])
        return {"out": s["out"], "weights": s["weights"]} if c["weights"] else {"out": s["out"]}
    if op == "evict":
        kept, new = ub.paged_evict(s["pool_k"], s["pool_v"], s["weights"], LAYER, s["table"], s["lens"], s["max_len"],
                                   c["budget"], n_sinks=c["sinks"], n_recent=c["recent"])
        return {"kept": kept, "new_lens": new, "pool_k": s["pool_k"], "pool_v": s["pool_v"], "weights": s["weights"]}
    ub.windowed_prefill_attn(s["q"], s["k"], s["v"], s["cu"], s["past"], s["max_seqlen"], c["window"], c["sinks"],
                             out=s["out"], out_fp32=False, lse=s["lse"])
    if op == "prefill":
        return {"out": s["out"], "lse": s["lse"]}
    dq, dk, dv = ub.windowed_prefill_bwd(s["q"], s["k"], s["v"], s["out"], s["dout"], s["lse"], s["cu"], s["past"],
                                         s["max_seqlen"], c["window"], c["sinks"], grad_fp32=False)
    return {"out": s["out"], "dq": dq, "dk": dk, "dv": dv}


def run(state):
    if own:
        return _own(state)
    return {"write": _plain_write, "decode": _plain_decode, "evict": _plain_evict, "prefill": _plain_prefill,
            "train": _plain_train}[state["op"]](state)


# ------------------------------------------------- the definition in 64 bits

def _exact_decode(s):
    c = s["case"]
    G, ps, D = c["H"] // c["Hkv"], c["page"], c["D"]
    out = torch.zeros((c["R"], c["H"], D), dtype=torch.float64, device="cuda")
    weights = s["weights"].double() if c["weights"] else None
    for r, n in enumerate(s["lens"].tolist()):
        pages = s["table"][r, : (n + ps - 1) // ps].long()
        window = c["window"] or n + 2
        pos = n if c["self_key"] else n - 1
        idx = torch.tensor([j for j in range(n) if pos - j < window or j < c["sinks"]], dtype=torch.long,
                           device="cuda")
        for h in range(c["Hkv"]):
            K, V = (t[LAYER, pages, h].reshape(-1, D)[idx] if t.dtype == torch.bfloat16 else
                    t.view(torch.uint8)[LAYER, pages, h].reshape(-1, D)[idx].view(torch.float8_e4m3fn)
                    for t in (s["pool_k"], s["pool_v"]))
            K, V = K.double(), V.double()
            if c["e4m3"]:     # powers of two: exact in the type that attention reads
                K, V = K * s["scales"][0], V * s["scales"][1]
            if c["self_key"]:
                K = torch.cat([K, s["k"][r, h].double()[None]])
                V = torch.cat([V, s["v"][r, h].double()[None]])
            if K.shape[0] == 0:
                continue
            p = torch.softmax(s["q"][r, h * G: (h + 1) * G].double() @ K.T / math.sqrt(D), -1)
            out[r, h * G: (h + 1) * G] = p @ V
            if weights is not None:
                weights[LAYER, pages[idx // ps], h, idx % ps] += p[:, : idx.numel()].sum(0)
    return {"out": out, "weights": weights} if weights is not None else {"out": out}


def _exact_attn(s, grads):
    c = s["case"]
    G, D = c["H"] // c["Hkv"], c["D"]
    q, k, v = s["q"].double(), s["k"].double(), s["v"].double()
    out = torch.zeros_like(q)
    lse = torch.zeros(q.shape[:2], dtype=torch.float64, device="cuda")
    dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    cu = s["cu"].tolist()
    for b, n in enumerate(s["past"].tolist()):
        t0, t1 = cu[b], cu[b + 1]
        rows = torch.arange(t1 - t0, device="cuda")
        at = rows.clamp(max=n)          # a candidate stands right after the history
        behind = at[:, None] - at[None]
        ok = (behind >= 0) & ((behind < c["window"]) | (rows[None] < c["sinks"])) & (rows[None] < n)
        ok |= rows[:, None] == rows[None]
        for h in range(c["H"]):
            Q, K, V = q[t0:t1, h], k[t0:t1, h // G], v[t0:t1, h // G]
            a = torch.where(ok, Q @ K.T / math.sqrt(D), -math.inf)
            z = torch.logsumexp(a, -1, keepdim=True)
            p = torch.exp(a - z)
            out[t0:t1, h] = p @ V
            lse[t0:t1, h] = z[:, 0] / math.log(2.0)
            if grads:
                g = s["dout"][t0:t1, h].double()
                dp = g @ V.T
                ds = p * (dp - (p * dp).sum(-1, keepdim=True)) / math.sqrt(D)
                dq[t0:t1, h] = ds @ K
                dk[t0:t1, h // G] += ds.T @ Q
                dv[t0:t1, h // G] += p.T @ g
    return {"out": out, "dq": dq, "dk": dk, "dv": dv} if grads else {"out": out, "lse": lse}


def exact(case, seed):
    if case["op"] in ("write", "evict"):    # values are moved or rounded, none is computed
        return None
    s = prepare(case, seed)
    if case["op"] == "decode":
        return _exact_decode(s)
    return _exact_attn(s, case["op"] == "train")

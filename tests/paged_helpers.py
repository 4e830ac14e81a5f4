"""Paged pools for the tests, and the paged operators' plain forms in float64 on the CPU."""

import math

import torch

E4M3_CODES = torch.arange(256, dtype=torch.int32).to(torch.uint8)


class PagedCase:
    """Requests' rows in a paged pool on the CPU: pages in random order, everything that is not a
    cached row is NaN (0x7F codes in an E4M3 pool)."""

    def __init__(self, seed, lens, Hkv, D, page, L=2, layer=1, scales=None, spare=2, width=None):
        g = torch.Generator().manual_seed(seed)
        self.g, self.lens, self.Hkv, self.D, self.page, self.layer, self.scales = g, lens, Hkv, D, page, layer, scales
        need = [(n + page - 1) // page for n in lens]
        S = sum(need) + spare
        self.width = max([1] + need) if width is None else width
        order = torch.randperm(S, generator=g).tolist()
        self.table = torch.full((len(lens), self.width), -1, dtype=torch.int32)
        at = 0
        for r, n in enumerate(need):
            for i in range(n):
                self.table[r, i] = order[at]
                at += 1
        shape = (L, S, Hkv, page, D)
        if scales is None:
            self.k = torch.full(shape, float("nan"), dtype=torch.bfloat16)
        else:
            self.k = torch.full(shape, 0x7F, dtype=torch.uint8)
        self.v = self.k.clone()
        self.weights = torch.full(shape[:4], float("nan"))
        for r, n in enumerate(lens):
            for j in range(n):
                pg, off = int(self.table[r, j // page]), j % page
                if scales is None:
                    self.k[layer, pg, :, off] = torch.randn(Hkv, D, generator=g).to(torch.bfloat16)
                    self.v[layer, pg, :, off] = torch.randn(Hkv, D, generator=g).to(torch.bfloat16)
                else:
                    for t, s in ((self.k, scales[0]), (self.v, scales[1])):
                        x = (torch.randn(Hkv, D, generator=g) / s).clamp(-448, 448).to(torch.float8_e4m3fn)
                        t[layer, pg, :, off] = x.view(torch.uint8)
                self.weights[layer, pg, :, off] = torch.rand(Hkv, generator=g)

    def row(self, r, j):
        return int(self.table[r, j // self.page]), j % self.page

    def rows64(self, pool, scale, r, idx):
        """Rows idx of request r as attention reads them, float64 [len(idx), Hkv, D]."""
        out = torch.empty((len(idx), self.Hkv, self.D), dtype=torch.float64)
        for i, j in enumerate(idx):
            pg, off = self.row(r, j)
            x = pool[self.layer, pg, :, off]
            if scale is not None:
                x = (x.view(torch.float8_e4m3fn).float() * torch.tensor(scale, dtype=torch.float32)).to(torch.bfloat16)
            out[i] = x.double()
        return out

    def poison_unseen(self, seen):
        """Every row outside seen[r] (a set of rows) becomes NaN: it must not be read into a result."""
        for r, n in enumerate(self.lens):
            for j in range(n):
                if j not in seen[r]:
                    pg, off = self.row(r, j)
                    bad = float("nan") if self.scales is None else 0x7F
                    self.k[self.layer, pg, :, off] = bad
                    self.v[self.layer, pg, :, off] = bad


def visible(n, window, sinks, own):
    pos = n if own else n - 1
    return [j for j in range(n) if window is None or pos - j < window or j < sinks]


def decode64(case, q, k_self, v_self, window, sinks):
    """(out [R, H, D], sum of weight * |v| [R, H, D], {request: (rows, weights [rows, Hkv])}), float64."""
    R, H, D = q.shape
    G = H // case.Hkv
    out = torch.zeros((R, H, D), dtype=torch.float64)
    mag = torch.zeros_like(out)
    weights = {}
    ks, vs = case.scales or (None, None)
    for r in range(R):
        idx = visible(case.lens[r], window, sinks, k_self is not None)
        K, V = case.rows64(case.k, ks, r, idx), case.rows64(case.v, vs, r, idx)
        if k_self is not None:
            K, V = torch.cat([K, k_self[r].double()[None]]), torch.cat([V, v_self[r].double()[None]])
        w = torch.zeros((len(idx), case.Hkv), dtype=torch.float64)
        if K.shape[0]:
            for h in range(H):
                p = torch.softmax((K[:, h // G] @ q[r, h].double()) / math.sqrt(D), 0)
                out[r, h] = p @ V[:, h // G]
                mag[r, h] = p @ V[:, h // G].abs()
                w[:, h // G] += p[: len(idx)]
        weights[r] = (idx, w)
    return out, mag, weights


def evict64(weights, n, budget, sinks, recent):
    """Kept rows of one head: weights a list of n floats."""
    if n <= budget:
        return list(range(n))
    mid = list(range(sinks, n - recent))
    key = [-math.inf if math.isnan(weights[j]) else weights[j] for j in range(n)]
    mid.sort(key=lambda j: (-key[j], 0 if not math.isnan(weights[j]) else 1, j))
    return sorted(list(range(sinks)) + mid[: budget - sinks - recent] + list(range(n - recent, n)))

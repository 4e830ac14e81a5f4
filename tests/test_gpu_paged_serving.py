"""The paged and windowed operators as a serving and a training loop use them: one after another, from CUDA
graphs, on streams of their own.  Tolerances as in test_gpu_paged.py and test_gpu_windowed.py."""

import pytest
import torch

from tests.paged_helpers import PagedCase, decode64, evict64
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


def _rnd(g, *shape):
    return torch.randn(*shape, generator=g).to(torch.bfloat16)


class Serving:
    """Users with histories in a paged pool: device state and a PagedCase that mirrors it on the CPU."""

    def __init__(self, ub, seed, lens, H, Hkv, D, page, spare_rows, window, sinks, scales=None):
        self.ub, self.H, self.window, self.sinks = ub, H, window, sinks
        full = [n + spare_rows for n in lens]
        self.c = PagedCase(seed, full, Hkv, D, page, scales=scales)     # pages for the rows to come, too
        self.c.lens = list(lens)
        c = self.c
        empty = float("nan") if scales is None else 0x7F
        c.k.fill_(empty), c.v.fill_(empty)
        self.k, self.v, self.w = c.k.cuda(), c.v.cuda(), torch.zeros_like(c.weights).cuda()
        self.table, self.status = c.table.cuda(), torch.zeros(1, dtype=torch.int32, device="cuda")

    def ok(self):
        torch.cuda.synchronize()
        assert int(self.status.item()) == 0, self.ub.status_string(int(self.status.item()))

    def mirror(self):
        self.c.k, self.c.v, self.c.weights = self.k.cpu(), self.v.cpu(), self.w.cpu()

    def write(self, k, v, cu, new, first):
        self.ub.paged_pool_write(self.k, self.v, self.c.layer, k.cuda(), v.cuda(), _i32(cu), _i32(new), self.table,
                                 _i32(first), max(new), key_weights=self.w, dev_status=self.status,
                                 pool_scales=self.c.scales)

    def decode(self, q, k_self=None, v_self=None, **kw):
        return self.ub.paged_decode_attn(q.cuda(), self.table, _i32(self.c.lens), self.k, self.v, self.c.layer,
                                         max(self.c.lens) + 8, k_self=None if k_self is None else k_self.cuda(),
                                         v_self=None if v_self is None else v_self.cuda(), window=self.window,
                                         n_sinks=self.sinks, key_weights=self.w, dev_status=self.status,
                                         pool_scales=self.c.scales, **kw)


@pytest.mark.parametrize("scales", [None, (2.0 ** -6, 2.0 ** -6)], ids=["bf16", "e4m3"])
def test_prefill_write_decode_evict_decode(ub, scales):
    """Histories are prefilled under a window, written into pages, decoded token by token with their weights
    collected, evicted, and decoded again; every result against its plain form over the mirrored cache."""
    lens, H, Hkv, D, window, sinks = [70, 5, 133], 4, 2, 64, 50, 3
    g = torch.Generator().manual_seed(3)
    s = Serving(ub, 3, lens, H, Hkv, D, 16, 12, window, sinks, scales)
    past, segs = lens, [n + 1 for n in lens]            # one candidate each
    cu = [0]
    for n in segs:
        cu.append(cu[-1] + n)
    q, k, v = _rnd(g, cu[-1], H, D), _rnd(g, cu[-1], Hkv, D), _rnd(g, cu[-1], Hkv, D)
    out = ub.windowed_prefill_attn(q.cuda(), k.cuda(), v.cuda(), _i32(cu), _i32(past), max(segs), window, sinks,
                                   dev_status=s.status)
    s.write(k, v, cu, past, [0, 0, 0])
    s.ok()
    ref, mag, _ = prefill64(q, k, v, cu, past, window, sinks)
    assert ((out.cpu().double() - ref).abs() <= mag * (ROUND + WEIGHT) + 1e-6).all()
    # the candidate's row again, from the cache: the same pairs (an E4M3 cache holds rounded rows)
    last = [c - 1 for c in cu[1:]]
    s.mirror()
    o = s.decode(q[last], k[last], v[last])
    s.ok()
    ref, mag, weights = decode64(s.c, q[last], k[last], v[last], window, sinks)
    assert ((o.cpu().double() - ref).abs() <= mag * (ROUND + WEIGHT) + 1e-6).all()
    if scales is None:
        assert ((o - out[last]).abs().cpu().double() <= 2 * mag * (ROUND + WEIGHT) + 2e-6).all()
    total = s.c.weights.double()
    for step in range(5):
        for r, (idx, p) in weights.items():             # what the call before added
            for i, j in enumerate(idx):
                pg, off = s.c.row(r, j)
                total[s.c.layer, pg, :, off] += p[i]
        s.mirror()
        near = (s.c.weights.double() - total).abs() <= (step + 1) * 2.0 ** -11
        assert near[s.c.layer].all()
        qn, kn, vn = _rnd(g, 3, H, D), _rnd(g, 3, Hkv, D), _rnd(g, 3, Hkv, D)
        s.write(kn, vn, [0, 1, 2, 3], [1, 1, 1], s.c.lens)      # the token's row first, then its attention
        s.c.lens = [n + 1 for n in s.c.lens]
        s.mirror()
        total = s.c.weights.double()
        o = s.decode(qn)
        s.ok()
        ref, mag, weights = decode64(s.c, qn, None, None, window, sinks)
        assert ((o.cpu().double() - ref).abs() <= mag * (ROUND + WEIGHT) + 1e-6).all()
    s.mirror()
    budget = 40
    kept, new = ub.paged_evict(s.k, s.v, s.w, s.c.layer, s.table, _i32(s.c.lens), max(s.c.lens), budget, n_sinks=sinks,
                               n_recent=8, dev_status=s.status)
    s.ok()
    for r, n in enumerate(s.c.lens):
        for h in range(Hkv):
            w = [float(s.c.weights[s.c.layer, s.c.row(r, j)[0], h, s.c.row(r, j)[1]]) for j in range(n)]
            want = evict64(w, n, budget, sinks, 8)
            assert kept[r, h].tolist() == want + [-1] * (budget - len(want))
    before = s.c
    s.c.lens = new.tolist()
    s.mirror()
    qn, kn, vn = _rnd(g, 3, H, D), _rnd(g, 3, Hkv, D), _rnd(g, 3, Hkv, D)
    o = s.decode(qn, kn, vn, out_fp32=False)
    s.ok()
    ref, mag, _ = decode64(before, qn, kn, vn, window, sinks)
    assert ((o.cpu().double() - ref).abs() <= mag * (ROUND + WEIGHT) + ref.abs() * ROUND + 1e-6).all()


def test_decode_step_from_a_graph_and_a_shared_workspace(ub):
    """A captured step (write, decode) replays on changed inputs and lengths, and two graphs that share a
    workspace, replayed in turn, give the eager results."""
    lens, H, Hkv, D = [1200, 30, 700, 0], 8, 2, 64
    g = torch.Generator().manual_seed(4)
    c = PagedCase(4, lens, Hkv, D, 32, width=45)
    k, v, table = c.k.cuda(), c.v.cuda(), c.table.cuda()
    n = _i32(lens)
    q = [_rnd(g, 4, H, D).cuda() for _ in range(2)]
    ks, vs = _rnd(g, 4, Hkv, D).cuda(), _rnd(g, 4, Hkv, D).cuda()
    ws = torch.empty(ub.paged_decode_workspace_size(k, v, 4, H, 1300), dtype=torch.uint8, device="cuda")
    assert ws.numel() > 0
    outs = [torch.empty(4, H, D, device="cuda") for _ in range(2)]

    def call(i):
        ub.paged_decode_attn(q[i], table, n, k, v, c.layer, 1300, k_self=ks, v_self=vs, out=outs[i], workspace=ws)

    def eager():
        got = []
        for i in range(2):
            call(i)
            got.append(outs[i].clone())
        return got

    want = eager()
    graphs = []
    for i in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call(i)
        graphs.append(graph)
    for change in range(3):
        for i in (0, 1, 0):
            outs[i].fill_(7)
            graphs[i].replay()
            assert torch.equal(outs[i], want[i])
        q[0].copy_(_rnd(g, 4, H, D))
        ks.copy_(_rnd(g, 4, Hkv, D))
        n.copy_(_i32([[600, 30, 1, 0], [1200, 0, 64, 0], [1200, 30, 700, 0]][change]))
        want = eager()


def test_training_step_from_a_graph_beside_an_eager_one(ub):
    """The forward and backward of the same inputs, captured, while an eager step's results are alive."""
    lens, past, window, sinks = [300, 90], [250, 60], 64, 2
    g = torch.Generator().manual_seed(5)
    cu = [0, 300, 390]
    q, k, v, dout = (_rnd(g, 390, h, 64) for h in (4, 2, 2, 4))
    dev = [x.cuda() for x in (q, k, v, dout)]
    out, lse = torch.empty_like(dev[0]), torch.empty(390, 4, device="cuda")
    cu_d, past_d = _i32(cu), _i32(past)
    grads = [torch.empty(x.shape, device="cuda") for x in dev[:3]]
    ws = torch.empty(ub.windowed_prefill_bwd_workspace_size(2, 4, 2, 64, 300, 390, window, sinks), dtype=torch.uint8,
                     device="cuda")

    def step(o, st, gr):
        ub.windowed_prefill_attn(*dev[:3], cu_d, past_d, 300, window, sinks, out=o, out_fp32=False, lse=st)
        ub.windowed_prefill_bwd(*dev[:3], o, dev[3], st, cu_d, past_d, 300, window, sinks, dq=gr[0], dk=gr[1], dv=gr[2],
                                workspace=ws)

    eager = torch.empty_like(out), torch.empty_like(lse), [torch.empty_like(x) for x in grads]
    step(*eager)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(out, lse, grads)
    for _ in range(2):
        graph.replay()
        assert torch.equal(out, eager[0]) and torch.equal(lse, eager[1])
        assert all(torch.equal(a, b) for a, b in zip(grads, eager[2]))
    dev[0].copy_(_rnd(g, 390, 4, 64))
    graph.replay()
    want = grads64(dev[0].cpu(), k, v, dout, cu, past, window, sinks)
    for name, got in zip(("dq", "dk", "dv"), grads):
        assert ((got.cpu().double() - want[name][0]).abs() <= want[name][1] + 1e-6).all()


def test_calls_on_other_streams_at_once(ub):
    """Calls on two streams at a time, workspaces and outputs allocated by the calls, give the results of one
    after the other."""
    lens, H, Hkv, D = [900, 1500, 64], 8, 2, 128
    c = PagedCase(6, lens, Hkv, D, 64)
    k, v, table, n = c.k.cuda(), c.v.cuda(), c.table.cuda(), _i32(lens)
    g = torch.Generator().manual_seed(6)
    q = [_rnd(g, 3, H, D).cuda() for _ in range(6)]
    cu, past = _i32([0, 200, 500]), _i32([150, 300])
    x = [_rnd(g, 500, h, D).cuda() for h in (4, 2, 2)]
    dout, lse = _rnd(g, 500, 4, D).cuda(), torch.empty(500, 4, device="cuda")
    o = ub.windowed_prefill_attn(*x, cu, past, 300, 70, 1, out_fp32=False, lse=lse)
    want = [ub.paged_decode_attn(qq, table, n, k, v, c.layer, 1500) for qq in q]
    want_g = ub.windowed_prefill_bwd(*x, o, dout, lse, cu, past, 300, 70, 1)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got, got_g = [], []
    for i, qq in enumerate(q):
        got.append(ub.paged_decode_attn(qq, table, n, k, v, c.layer, 1500, stream=streams[i % 2]))
        got_g.append(ub.windowed_prefill_bwd(*x, o, dout, lse, cu, past, 300, 70, 1, stream=streams[(i + 1) % 2]))
        torch.empty(1 << 20, device="cuda").fill_(1.0)    # takes what the allocator thinks is free
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    for gr in got_g:
        assert all(torch.equal(a, b) for a, b in zip(gr, want_g))

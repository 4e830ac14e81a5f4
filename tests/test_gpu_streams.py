"""Calls on a stream that is not the current one: what a call allocates belongs to the call's stream, so that
nothing still queued on the current stream can touch it, and outputs are not handed out again while the
current stream uses them.  The allocator's own record says under which stream each allocation was made: no
timing is needed."""

import contextlib

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ub():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from kv_cache_reuse_falcon_b200 import binding
    return binding


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _rnd(*shape):
    return torch.randn(*shape, device="cuda").to(torch.bfloat16)


@contextlib.contextmanager
def allocations(into):
    """The stream of every allocation made inside."""
    torch.cuda.memory._record_memory_history(max_entries=1000, stacks="python")
    try:
        yield
        for e in torch.cuda.memory._snapshot()["device_traces"][torch.cuda.current_device()]:
            if e["action"] == "alloc":
                into.append(e["stream"])
    finally:
        torch.cuda.memory._record_memory_history(enabled=None)


def paged_calls(ub):
    """name -> (call of a stream, allocations of the call)"""
    q, x = _rnd(3, 8, 64), [_rnd(200, h, 64) for h in (4, 2, 2)]
    pk, pv = _rnd(1, 64, 2, 16, 64), _rnd(1, 64, 2, 16, 64)
    w = torch.rand(1, 64, 2, 16, device="cuda")
    table, lens = _i32(torch.arange(60).reshape(3, 20).tolist()), _i32([300, 7, 150])
    cu, past = _i32([0, 120, 200]), _i32([100, 60])
    lse = torch.empty(200, 4, device="cuda")
    o = ub.windowed_prefill_attn(*x, cu, past, 120, 30, 1, out_fp32=False, lse=lse)
    return {
        "decode": (lambda s: [ub.paged_decode_attn(q, table, lens, pk, pv, 0, 300, key_weights=w, stream=s)], 2),
        "evict": (lambda s: ub.paged_evict(pk, pv, w, 0, table, lens, 300, 150, stream=s), 2),
        "prefill": (lambda s: [ub.windowed_prefill_attn(*x, cu, past, 120, 30, 1, stream=s)], 1),
        "prefill_bwd": (lambda s: ub.windowed_prefill_bwd(*x, o, x[0], lse, cu, past, 120, 30, 1, stream=s), 4),
    }


def _check_allocations(call, count):
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    for s, want in ((stream, stream.cuda_stream), (None, torch.cuda.current_stream().cuda_stream),
                    (torch.cuda.current_stream(), torch.cuda.current_stream().cuda_stream)):
        seen = []
        with allocations(seen):
            out = call(s)
        assert seen == [want] * count
        torch.cuda.synchronize()
        del out
    assert torch.cuda.current_stream() == torch.cuda.default_stream()      # as the caller left it


def _check_hand_out(call):
    """An output that the current stream still uses does not go to the call's stream again."""
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    out = list(call(stream))
    torch.cuda.current_stream().wait_stream(stream)
    mine = {(t.untyped_storage().data_ptr(), t.untyped_storage().nbytes()) for t in out}
    torch.cuda._sleep(400_000_000)          # about 0.2 s in which the current stream is not done with it
    used = [t.clone() for t in out]
    shapes = [(t.shape, t.dtype) for t in out]
    del out
    with torch.cuda.stream(stream):
        again = [torch.empty(s, dtype=d, device="cuda") for s, d in shapes]
    assert not mine & {(t.untyped_storage().data_ptr(), t.untyped_storage().nbytes()) for t in again}
    torch.cuda.synchronize()
    del used, again


@pytest.mark.parametrize("name", ["decode", "evict", "prefill", "prefill_bwd"])
def test_paged_and_windowed_calls_allocate_under_their_stream(ub, name):
    call, count = paged_calls(ub)[name]
    _check_allocations(call, count)
    _check_hand_out(call)


def slot_calls(ub):
    x = [_rnd(200, h, 64) for h in (4, 2, 2)]
    cu, past, slots = _i32([0, 120, 200]), _i32([100, 60]), _i32([1, 0])
    pk, pv = _rnd(1, 2, 2, 128, 64), _rnd(1, 2, 2, 128, 64)
    pk8, pv8 = (torch.zeros(1, 2, 2, 128, 64, dtype=torch.uint8, device="cuda") for _ in range(2))
    lse = torch.empty(200, 4, device="cuda")
    o = ub.masked_prefill_attn(*x, cu, past, 120, out_fp32=False, lse=lse)
    cu_c = _i32([0, 120, 200])
    y = torch.rand(1000, device="cuda")
    return {
        "prefill": (lambda s: [ub.masked_prefill_attn(*x, cu, past, 120, stream=s)], 2),
        "prefill_bwd": (lambda s: ub.masked_prefill_bwd(*x, o, x[0], lse, cu, past, 120, stream=s), 4),
        "decode": (lambda s: [ub.rank_decode_attn(*x, cu_c, slots, past, pk, pv, 0, 120, stream=s)], 2),
        "decode_e4m3": (lambda s: [ub.rank_decode_attn(*x, cu_c, slots, past, pk8, pv8, 0, 120, stream=s,
                                                       pool_scales=(0.5, 0.5))], 2),
        "exp2": (lambda s: [ub.selftest_exp2(y, stream=s)], 1),
    }


@pytest.mark.parametrize("name", ["prefill", "prefill_bwd", "decode", "decode_e4m3", "exp2"])
def test_slot_pool_calls_allocate_under_their_stream(ub, name):
    call, count = slot_calls(ub)[name]
    _check_allocations(call, count)
    _check_hand_out(call)


def test_a_foreign_stream_object_is_taken_by_its_handle(ub):
    """Anything with a `cuda_stream`, as the calls' own look-up of the handle allows."""
    class Handle:
        def __init__(self, stream):
            self.cuda_stream = stream.cuda_stream

    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    for calls in (paged_calls(ub), slot_calls(ub)):
        call, count = calls["prefill"]
        torch.cuda.synchronize()
        want, seen = call(None), []
        with allocations(seen):
            got = call(Handle(stream))
        torch.cuda.synchronize()
        assert seen == [stream.cuda_stream] * count and torch.equal(got[0], want[0])


@pytest.mark.parametrize("calls,name", [(paged_calls, "decode"), (paged_calls, "prefill_bwd"), (slot_calls, "prefill"),
                                        (slot_calls, "prefill_bwd")])
def test_calls_on_a_forked_stream_are_captured(ub, calls, name):
    """A stream forked from the capturing one: the call's memory is the graph's, and its replays give the eager bits
    while an eager call's results live."""
    call, _ = calls(ub)[name]
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    first = call(stream)
    torch.cuda.synchronize()
    want = [t.clone() for t in first]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        stream.wait_stream(torch.cuda.current_stream())
        got = call(stream)
        torch.cuda.current_stream().wait_stream(stream)
    for _ in range(2):
        for t in got:
            t.zero_()
        other = call(None)
        graph.replay()
        torch.cuda.synchronize()
        if calls is slot_calls and name == "prefill_bwd":      # float32 sums of a few tiles in any order
            tol = [w.abs().max() * 2.0 ** -18 for w in want]
        else:
            tol = [0.0] * len(want)
        for a, b, c, t in zip(got, want, other, tol):
            assert (a - b).abs().max() <= t and (c - b).abs().max() <= t

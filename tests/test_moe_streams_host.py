"""Which stream the memory of a layer of experts belongs to (no GPU): streams, the
allocator's records and the library's call are stand-ins, the layer is the real one.
Memory that a call makes has to be known to the allocator on every stream whose work
uses it, or it is given away while that work runs."""
import contextlib
import types

import pytest

from shape_driven_tile_amd import binding as sdt
from shape_driven_tile_amd import moe


class Streams:
    """Streams by handle, what each allocation was made on and recorded for, and
    the calls of the library."""

    def __init__(self, monkeypatch):
        import torch
        self.main, self.side = (types.SimpleNamespace(cuda_stream=h) for h in (1, 2))
        self.current = [self.main]
        self.known = {}              # address -> the streams the allocator knows of
        self.calls = []
        self.keep = []               # an address stands for one allocation
        empty = torch.empty

        def make(*args, **kw):
            t = empty(*args, **kw)
            self.keep.append(t)
            self.known[t.data_ptr()] = {self.current[-1].cuda_stream}
            return t

        @contextlib.contextmanager
        def on(stream):
            self.current.append(stream)
            yield
            self.current.pop()

        def call(layer, X, idx, weights, plan, Y, workspace, stream=None):
            self.calls.append(types.SimpleNamespace(
                stream=(stream or self.current[-1]).cuda_stream, plan=plan.counts.data_ptr(),
                out=Y.data_ptr(), workspace=workspace.data_ptr()))

        monkeypatch.setattr(torch, "empty", make)
        monkeypatch.setattr(torch.cuda, "stream", on)
        monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: self.current[-1])
        monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
        monkeypatch.setattr(torch.Tensor, "record_stream",
                            lambda t, s: self.known[t.data_ptr()].add(s.cuda_stream))
        monkeypatch.setattr(sdt, "_stream_handle", lambda s: (s or self.current[-1]).cuda_stream)
        monkeypatch.setattr(sdt, "moe_experts_mx4", call)


@pytest.fixture
def streams(monkeypatch):
    return Streams(monkeypatch)


def layer(E=4, N=64, K=64):
    def matrices(rows, cols):
        return sdt.Mx4.empty(rows, cols, experts=E, device="cpu")
    return moe.Mx4Experts(matrices(N, K), matrices(N, K), matrices(K, N))


def tokens(T, topk=2, K=64):
    import torch
    return (torch.zeros(T, K, dtype=torch.bfloat16), torch.zeros(T, topk, dtype=torch.int32),
            torch.zeros(T, topk))


def check(s):
    """The last call's memory is known on the stream that ran it."""
    c = s.calls[-1]
    for what in ("plan", "out", "workspace"):
        assert c.stream in s.known[getattr(c, what)], what
    return c


def test_memory_of_a_call_on_a_given_stream(streams):
    run = layer()
    y = run(*tokens(5), stream=streams.side)
    c = check(streams)
    assert c.stream == streams.side.cuda_stream
    # the caller, on the current stream, reads y
    assert streams.main.cuda_stream in streams.known[y.data_ptr()]


def test_buffer_used_on_streams_in_turn(streams):
    """The buffer is recorded on each stream that it is used on, so that it outlives
    their work when a larger one replaces it."""
    run = layer()
    run(*tokens(5))
    first = check(streams)
    run(*tokens(5), stream=streams.side)
    assert check(streams).workspace == first.workspace
    run(*tokens(500), stream=streams.side)
    grown = check(streams)
    assert grown.workspace != first.workspace
    run(*tokens(500))
    assert check(streams).workspace == grown.workspace
    run(*tokens(7), stream=streams.side)
    assert check(streams).workspace == grown.workspace


def test_buffer_used_on_another_current_stream(streams):
    import torch
    run = layer()
    run(*tokens(5))
    first = check(streams)
    with torch.cuda.stream(streams.side):
        y = run(*tokens(5))
        assert check(streams).workspace == first.workspace
        run(*tokens(500))
        check(streams)
    assert streams.known[y.data_ptr()] == {streams.side.cuda_stream}


def test_given_memory_stays_the_callers(streams):
    import torch
    run = layer()
    plan = sdt.MoePlan.empty(5, 2, 4, device="cpu")
    out = torch.empty(5, 64, dtype=torch.bfloat16)
    assert run(*tokens(5), plan=plan, out=out, stream=streams.side) is out
    c = streams.calls[-1]
    assert c.stream == streams.side.cuda_stream and c.out == out.data_ptr()
    assert c.plan == plan.counts.data_ptr()


def test_buffer_of_a_captured_call_is_kept(streams, monkeypatch):
    """A graph holds the buffer's address: a larger buffer that replaces it for
    later calls must not free it, and buffers of no graph are not kept."""
    import weakref

    import torch
    capturing = [False]
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: capturing[0])
    run = layer()

    def buffer(T, capture):
        capturing[0] = capture
        run(*tokens(T))
        return weakref.ref(run._workspace)

    refs = [buffer(5, False), buffer(500, False), buffer(500, True), buffer(2000, False),
            buffer(9000, True), buffer(20000, False)]
    streams.keep.clear()
    alive = [r() is not None for r in refs]
    assert alive == [False, True, True, False, True, True]

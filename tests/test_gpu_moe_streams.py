"""The experts' layer on streams of its own: what a call allocates and drops stays
whole until that call's work is done, whatever the current stream allocates then."""
import numpy as np
import pytest

from gpu_helpers import DEV, say
from test_gpu_moe import by_parts, choose, dev, make_layer

pytestmark = pytest.mark.gpu


def inputs(T, topk, E, K, seed):
    import torch
    rng = np.random.default_rng(seed)
    return (torch.from_numpy(rng.standard_normal((T, K))).bfloat16().to(DEV),
            dev(choose(T, topk, E, rng)), dev(rng.random((T, topk)).astype(np.float32)))


def test_dropped_memory_outlives_the_work():
    """Calls on a side stream with plans of their own and a growing buffer; the
    current stream takes and fills memory of the same sizes before anything waits."""
    import torch

    from shape_driven_tile_amd import binding as sdt
    E, topk, N, K = 8, 2, 96, 160
    layer, parts = make_layer(E, N, K, "bf16", 11)
    sizes = (70, 300, 900)
    given = [inputs(T, topk, E, K, T) for T in sizes]
    want = [by_parts(parts, *g, "bf16") for g in given]
    torch.cuda.synchronize()
    say("layer on a side stream, memory dropped")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got, filled = [], []
    for T, g in zip(sizes, given):
        got.append(layer(*g, stream=side))
        for n in (sdt.moe_experts_workspace_size(T, topk, E, N, K), 4 * sdt.MoePlan.empty(
                T, topk, E, device="cpu").rows.numel(), T * K * 2):
            filled.append(torch.full((n,), 0x7f, dtype=torch.uint8, device=DEV))
    torch.cuda.current_stream().wait_stream(side)
    copies = [y.clone() for y in got]            # read on the current stream
    torch.cuda.synchronize()
    for y, w in zip(copies, want):
        assert torch.equal(y, w)
    assert all(bool((f == 0x7f).all()) for f in filled)


def test_streams_in_turn():
    """One buffer on two streams, each call ordered after the last by the caller."""
    import torch
    E, topk, N, K = 4, 2, 64, 96
    layer, parts = make_layer(E, N, K, "bf16", 12)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    say("layer on streams in turn")
    last = torch.cuda.current_stream()
    got, want = [], []
    for i, T in enumerate((40, 40, 500, 500, 20)):
        g = inputs(T, topk, E, K, i)
        want.append(by_parts(parts, *g, "bf16"))
        torch.cuda.synchronize()
        streams[i % 2].wait_stream(last)
        if i < 2:
            got.append(layer(*g, stream=streams[i % 2]))
        else:
            with torch.cuda.stream(streams[i % 2]):
                got.append(layer(*g))
        last = streams[i % 2]
    torch.cuda.synchronize()
    for y, w in zip(got, want):
        assert torch.equal(y, w)


def test_graph_keeps_its_buffer():
    """A graph captured with a small buffer, replayed after larger eager calls have
    replaced it and other tensors have taken and filled memory of its size."""
    import torch

    from shape_driven_tile_amd import binding as sdt
    E, topk, N, K = 8, 2, 96, 160
    layer, parts = make_layer(E, N, K, "bf16", 13)
    small, large = inputs(50, topk, E, K, 1), inputs(700, topk, E, K, 2)
    say("layer in a graph, larger calls between replays")
    layer(*small)
    y = torch.zeros(50, K, dtype=torch.bfloat16, device=DEV)
    plan = sdt.MoePlan.empty(50, topk, E, device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer(*small, plan=plan, out=y)
    need = sdt.moe_experts_workspace_size(50, topk, E, N, K)
    want = by_parts(parts, *small, "bf16")
    want_large = by_parts(parts, *large, "bf16")
    torch.cuda.synchronize()
    for _ in range(3):
        assert torch.equal(layer(*large), want_large)
        filled = [torch.full((need,), 0x7f, dtype=torch.uint8, device=DEV) for _ in range(4)]
        y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want)
        assert all(bool((f == 0x7f).all()) for f in filled)

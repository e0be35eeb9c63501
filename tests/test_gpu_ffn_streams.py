"""The feed-forward operators on the stream that a call is given, from another current one:
behind work that keeps that stream busy, through buffers that the call is given and such as
it makes, and in a graph captured on it."""
import pytest

from gpu_helpers import DEV
from test_gpu_ffn import OUTPUTS, block, block_state, fp8_matrix, normal

pytestmark = pytest.mark.gpu


class On:
    """The binding, each call on one stream by its argument."""

    def __init__(self, stream):
        from shape_driven_tile_amd import binding
        self._sdt, self._stream = binding, stream

    def __getattr__(self, name):
        call = getattr(self._sdt, name)
        return lambda *args, **kw: call(*args, stream=self._stream, **kw)


def split_state(M=100, N=72, K=4000):
    """Products that are split along K, through buffers that the calls make."""
    import torch
    from shape_driven_tile_amd import binding as sdt
    s = {"a": fp8_matrix(M, K, 1, 1)[0], "b": fp8_matrix(N, K, 128, 2)[0],
         "gx": normal((M, K), torch.bfloat16, 3), "gg": normal((N, K), torch.bfloat16, 4, K ** -0.5),
         "gu": normal((N, K), torch.bfloat16, 5, K ** -0.5)}
    assert sdt.gemm_fp8_workspace_size(M, N, K) > 0 and sdt.gated_ff_split_size(M, N, K) > 0
    s["c"], s["gh"] = (torch.empty(M, N, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    s["q"] = torch.empty(M, K, device=DEV)
    return s


def split_block(sdt, s):
    sdt.gemm_fp8_bf16(s["a"], s["b"], s["c"])
    sdt.gated_ff(s["gx"], s["gg"], s["gu"], s["gh"], act="gelu")
    sdt.fp8_dequantize_f32(s["a"], s["q"])


def run(sdt, s):
    block(sdt, s)
    split_block(sdt, s)


def state():
    s = block_state()
    s.update(split_state())
    return s


NAMES = OUTPUTS + ["c", "gh", "q"]


def test_stream_argument():
    """Two states on two streams, every call by the stream argument.  Each stream is first kept
    busy and then clears the outputs: a call that ran elsewhere would run before that."""
    import torch
    from shape_driven_tile_amd import binding
    want = state()
    run(binding, want)
    torch.cuda.synchronize()
    states, streams = [state() for _ in range(2)], [torch.cuda.Stream() for _ in range(2)]
    busy = [torch.empty(1 << 28, device=DEV) for _ in range(2)]            # 1 GiB: 0.2 ms a pass
    torch.cuda.synchronize()
    for turn in range(3):
        for s, stream, b in zip(states, streams, busy):
            with torch.cuda.stream(stream):
                for _ in range(8):
                    b.fill_(turn)
                for name in NAMES:
                    s[name].fill_(float("nan"))
            run(On(stream), s)
        # memory of the current stream's, which the calls' own buffers must not be given meanwhile
        junk = [torch.full((1 << 20,), float("nan"), device=DEV) for _ in range(4)]
        torch.cuda.synchronize()
        for s in states:
            for name in NAMES:
                assert torch.equal(s[name], want[name]), (turn, name)
        del junk


def test_stream_argument_in_a_graph():
    """Captured on the stream that the calls are given; every replay on the inputs it finds."""
    import torch
    from shape_driven_tile_amd import binding
    s, e = state(), state()
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    run(On(stream), s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        run(On(stream), s)
    for turn in range(3):
        for name in ("x", "gx"):
            new = normal(s[name].shape, torch.bfloat16, 70 + turn)
            s[name].copy_(new)
            e[name].copy_(new)
        for name in NAMES:
            s[name].fill_(float("nan"))
        torch.cuda.synchronize()
        graph.replay()
        run(binding, e)
        torch.cuda.synchronize()
        for name in NAMES:
            assert torch.equal(s[name], e[name]), (turn, name)

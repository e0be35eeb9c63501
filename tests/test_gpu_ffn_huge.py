"""Row-wise calls of more rows than a launch has workgroups for, one each: 2^24 and some.
Only rows around the borders hold values; they are compared with the same rows by
themselves, the others with zero."""
import pytest

from gpu_helpers import DEV, say
from test_gpu_ffn import normal

pytestmark = pytest.mark.gpu

ROWS = 2 ** 24 + 13


def places():
    """Some rows at both ends and around 2^24, 2^23 and where 32-bit offsets pass their ends."""
    import torch
    at = [r + d for r in (4, 2 ** 21, 2 ** 22, 2 ** 23, 2 ** 24, ROWS - 5) for d in range(-4, 5)]
    return torch.tensor(sorted(set(at)), device=DEV)


@pytest.fixture(autouse=True)
def room():
    import torch
    torch.cuda.empty_cache()
    yield
    torch.cuda.empty_cache()


def test_quantize():
    import torch
    from shape_driven_tile_amd import binding as sdt
    K = 1032
    say(f"quantise {ROWS}x{K}")
    at = places()
    x = torch.zeros(ROWS, K, dtype=torch.float16, device=DEV)                # 35 GB
    x[at] = normal((len(at), K), torch.float16, 1)
    m = sdt.Fp8.empty(ROWS, K, device=DEV)
    m.s.fill_(-1.0)
    sdt.fp8_quantize_f16(x, m)
    few = x[at].contiguous()
    want = sdt.Fp8.empty(len(at), K, device=DEV)
    sdt.fp8_quantize_f16(few, want)
    assert torch.equal(m.q.view(torch.uint8)[at], want.q.view(torch.uint8))
    assert torch.equal(m.s[:, at], want.s)
    others = torch.ones(ROWS, dtype=torch.bool, device=DEV)
    others[at] = False
    assert bool((m.s[:, others] == 2.0 ** -126).all())
    x.fill_(1.0)
    sdt.fp8_dequantize_f16(m, x)
    back = torch.empty_like(few)
    sdt.fp8_dequantize_f16(want, back)
    assert torch.equal(x[at], back)
    x[at] = 0.0
    assert not bool(x.view(torch.int32).any())


def test_gated_backward():
    import torch
    from shape_driven_tile_amd import binding as sdt
    N, K = 264, 8
    say(f"gated gradients {ROWS}x{N}x{K}")
    at = places()
    t = torch.bfloat16
    w = [normal((N, K), t, i) for i in (1, 2)]
    x = torch.zeros(ROWS, K, dtype=t, device=DEV)
    g = torch.zeros(ROWS, N, device=DEV)                                     # 18 GB each
    u = torch.zeros(ROWS, N, device=DEV)
    dh = torch.zeros(ROWS, N, dtype=t, device=DEV)
    for m, seed in ((x, 3), (g, 4), (u, 5), (dh, 6)):
        m[at] = normal((len(at), m.shape[1]), m.dtype, seed)
    dx = torch.full_like(x, float("nan"))
    ws = torch.empty(sdt.gated_ff_workspace_size(ROWS, N, K), dtype=torch.uint8, device=DEV)
    sdt.gated_ff_backward(x, *w, g, u, dh, dx, None, None, ws)
    few = [m[at].contiguous() for m in (x, g, u, dh)]
    want = torch.empty_like(few[0])
    sdt.gated_ff_backward(few[0], *w, *few[1:], want, None, None,
                          torch.empty(sdt.gated_ff_workspace_size(len(at), N, K), dtype=torch.uint8, device=DEV))
    assert torch.equal(dx[at], want)
    dx[at] = 0.0
    assert not bool(dx.any())

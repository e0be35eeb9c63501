"""Operands of a single row at strides that are no multiple of 16 bytes, NaN right behind
them: products over one k, batches of one row, weights of one row.  Whole numbers (and
halves) whose sums are exact, compared bit for bit."""
import pytest

from gpu_helpers import DEV, say
from test_gpu_ffn import out_like, rows_of, untouched, whole

pytestmark = pytest.mark.gpu

TYPES = ["f16", "bf16"]


def _sdt():
    from shape_driven_tile_amd import binding
    return binding


def _t(name):
    import torch
    return {"f16": torch.float16, "bf16": torch.bfloat16}[name]


def row(width, dtype, seed):
    """One row of whole numbers, its stride its width, NaN from its end on."""
    import torch
    full = torch.full((width + 64,), float("nan"), dtype=dtype, device=DEV)
    full[:width] = whole((width,), dtype, seed)
    return full[:width].view(1, width)


# 64 x 64 tiles, 128 x 128 ones, 256 x 256 ones
@pytest.mark.parametrize("M, N", [(1, 1), (5, 5), (5, 129), (129, 1), (1000, 3), (63, 65), (1501, 1999), (4001, 3999)])
@pytest.mark.parametrize("layout", ["nn", "tn"])
@pytest.mark.parametrize("dtype", TYPES)
def test_one_k(dtype, layout, M, N):
    import torch
    say(f"one k {layout} {dtype} {M}x{N}")
    sdt, t = _sdt(), _t(dtype)
    b = row(N, t, 2)
    a = row(M, t, 1) if layout == "tn" else rows_of(whole((M, 1), t, 1), 0)[0]
    c, full = out_like(M, N, t, pad=8)
    getattr(sdt, f"gemm_{dtype}_{layout}")(a, b, c)
    want = a.float().reshape(M, 1) * b.float()
    assert torch.equal(c, want.to(t))
    assert untouched(full, N)


def gated_parts(M, N, t):
    """dh, g, u whose dg = dh u / 2 (first half of the columns) and du = 40 dh (after it)
    are exact: a(0) = 0, a'(0) = 1 / 2; where u = 0, g = 40 and a(40) = 40 in fp32."""
    import torch
    dh = rows_of(whole((M, N), t, 3), 1, align=1)[0]
    first = torch.arange(N, device=DEV) < (N + 1) // 2
    g = torch.where(first, 0.0, 40.0).expand(M, N)
    u = torch.where(first, whole((M, N), torch.float32, 4), torch.zeros((), device=DEV))
    dg = torch.where(first, dh.double() * u.double() / 2, 0.0)
    du = torch.where(first, 0.0, 40.0 * dh.double())
    return dh, rows_of(g, 0, align=4)[0], rows_of(u, 0, align=4)[0], dg, du


@pytest.mark.parametrize("M, N, K", [(1, 1, 1), (1, 40, 5), (1, 2, 129), (1, 700, 1001), (3, 1, 5), (200, 1, 129),
                                     (1, 1, 333)])
@pytest.mark.parametrize("dtype", TYPES)
def test_gated_backward(dtype, M, N, K):
    """A batch of one row (x), weights of one row (gate and up)."""
    import torch
    say(f"gated backward, single rows {dtype} {M}x{N}x{K}")
    sdt, t = _sdt(), _t(dtype)
    x = row(K, t, 1) if M == 1 else rows_of(whole((M, K), t, 1), 0)[0]
    gate, up = (row(K, t, s) if N == 1 else rows_of(whole((N, K), t, s), 8)[0] for s in (5, 6))
    dh, g, u, dg, du = gated_parts(M, N, t)
    dx, fx = out_like(M, K, t, pad=8)
    dgate, fg = out_like(N, K, t)
    dup, fu = out_like(N, K, t, pad=16)
    ws = torch.full((sdt.gated_ff_workspace_size(M, N, K),), 0xFF, dtype=torch.uint8, device=DEV)
    sdt.gated_ff_backward(x, gate, up, g, u, dh, dx, dgate, dup, ws)
    assert torch.equal(dx, (dg @ gate.double() + du @ up.double()).float().to(t))
    assert torch.equal(dgate, (dg.t() @ x.double()).float().to(t))
    assert torch.equal(dup, (du.t() @ x.double()).float().to(t))
    assert untouched(fx, K) and untouched(fg, K) and untouched(fu, K)


@pytest.mark.parametrize("M, N, K", [(1, 40, 5), (1, 1, 1), (20, 1, 129), (300, 1, 1001), (1, 300, 333)])
@pytest.mark.parametrize("dtype", TYPES)
def test_gated(dtype, M, N, K):
    """Both factors of the gated block."""
    import torch
    say(f"gated, single rows {dtype} {M}x{N}x{K}")
    sdt, t = _sdt(), _t(dtype)
    x = row(K, t, 1) if M == 1 else rows_of(whole((M, K), t, 1), 0)[0]
    gate, up = (row(K, t, s) if N == 1 else rows_of(whole((N, K), t, s), 8)[0] for s in (5, 6))
    h, full = out_like(M, N, t, pad=8)
    g, u = (out_like(M, N, torch.float32)[0] for _ in range(2))
    sdt.gated_ff(x, gate, up, h, g=g, u=u)
    assert torch.equal(g.double(), x.double() @ gate.double().t())
    assert torch.equal(u.double(), x.double() @ up.double().t())
    assert untouched(full, N) and not bool(torch.isnan(h).any())


@pytest.mark.parametrize("M, N, K", [(1, 1, 1), (1, 300, 333), (40, 1, 129), (300, 1, 1001), (1, 40, 5)])
@pytest.mark.parametrize("dtype", TYPES)
def test_fp8(dtype, M, N, K):
    """8-bit operands of one row, NaN codes behind it; scales of one."""
    import torch
    say(f"8 bits, single rows {dtype} {M}x{N}x{K}")
    sdt, t = _sdt(), _t(dtype)

    def codes(rows, seed):
        ld = K if rows == 1 else -(-K // 16) * 16
        full = torch.full((rows * ld + 64,), 0x7F, dtype=torch.uint8, device=DEV)
        q = full[:rows * ld].view(torch.float8_e4m3fn).view(rows, ld)[:, :K]
        q.copy_(whole((rows, K), torch.float32, seed).to(torch.float8_e4m3fn))
        return q
    kb = -(-K // 128)
    a = sdt.Fp8(codes(M, 1), torch.ones(kb, M, device=DEV))
    b = sdt.Fp8(codes(N, 2), torch.ones(-(-N // 128), kb, device=DEV), block=128)
    c, full = out_like(M, N, t, pad=8)
    getattr(sdt, f"gemm_fp8_{dtype}")(a, b, c)
    assert torch.equal(c, (a.q.double() @ b.q.double().t()).float().to(t))
    assert untouched(full, N)

"""The products whose sizes take the 256 x 256 tiles (some 250 of them and more): turned,
8-bit and gated, and the gated block's gradients, on whole numbers small enough for every
sum to be exact in fp32, compared bit for bit, and the 8-bit product on random values
within the bound of the smaller ones.  K from none over one and two k-tiles on."""
import pytest

from gpu_helpers import DEV, say
from test_gpu_ffn import U, check, fp8_matrix, mfma_bound, out_like, rows_of, untouched, whole

pytestmark = pytest.mark.gpu

# tiles of 256: 16 x 16 with ragged ends, 15 x 17, 16 x 16 full
SIZES = [(4000, 3999, 1001), (3800, 4300, 330), (4096, 4096, 320), (4000, 3999, 128), (4096, 4096, 40),
         (3800, 4300, 0)]


def _sdt():
    from shape_driven_tile_amd import binding
    return binding


def operand(rows, K, dtype, seed, pad=8):
    return rows_of(whole((rows, K), dtype, seed), pad)[0]


@pytest.mark.parametrize("layout", ["nn", "tn"])
@pytest.mark.parametrize("M, N, K", SIZES)
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_turned(dtype, M, N, K, layout):
    import torch
    say(f"large {layout} {dtype} {M}x{N}x{K}")
    sdt, t = _sdt(), torch.float16 if dtype == "f16" else torch.bfloat16
    a = operand(M, K, t, 1) if layout == "nn" else operand(K, M, t, 1)
    b = operand(K, N, t, 2, pad=16)
    c, full = out_like(M, N, t, pad=8)
    getattr(sdt, f"gemm_{dtype}_{layout}")(a, b, c)
    want = (a if layout == "nn" else a.t()).double() @ b.double()     # at most 9 K < 2^24
    assert torch.equal(c, want.float().to(t))
    assert untouched(full, N)


@pytest.mark.parametrize("M, N, K", [(4000, 3999, 1001), (3800, 4300, 400), (4096, 4096, 512), (4000, 3999, 200),
                                     (4096, 4096, 100), (3800, 4300, 0)])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_fp8(dtype, M, N, K):
    import torch
    say(f"large 8-bit {dtype} {M}x{N}x{K}")
    sdt, t = _sdt(), torch.float16 if dtype == "f16" else torch.bfloat16
    for plain in (True, False):
        a, av = fp8_matrix(M, K, 1, 1, plain)
        b, bv = fp8_matrix(N, K, 128, 2, plain)
        c, full = out_like(M, N, t, pad=8)
        getattr(sdt, f"gemm_fp8_{dtype}")(a, b, c)
        want = av @ bv.t()
        if plain:
            assert torch.equal(c, want.float().to(t))
        else:
            check(c, want, (K + 4) * U * (av.abs() @ bv.abs().t()) + mfma_bound(av, bv), "gemm_fp8")
        assert untouched(full, N)


@pytest.mark.parametrize("M, N, K", [(4000, 1999, 1001), (3800, 2150, 330), (4096, 2048, 320), (4000, 1999, 100),
                                     (3800, 2150, 0)])
@pytest.mark.parametrize("wide", [True, False])
def test_gated(M, N, K, wide):
    """The factors bit for bit; h within the activation's steps of its exact value."""
    import torch
    say(f"large gated {M}x{N}x{K} wide {wide}")
    sdt, t = _sdt(), torch.bfloat16
    x, gate, up = operand(M, K, t, 1), operand(N, K, t, 2), operand(N, K, t, 3, pad=16)
    kept = torch.float32 if wide else t
    h, full = out_like(M, N, t, pad=8)
    g, gf = out_like(M, N, kept, pad=8)
    u, uf = out_like(M, N, kept, pad=8)
    sdt.gated_ff(x, gate, up, h, g=g, u=u)
    wg, wu = x.double() @ gate.double().t(), x.double() @ up.double().t()
    assert torch.equal(g, wg.to(kept)) and torch.equal(u, wu.to(kept))
    want = wg * torch.sigmoid(wg) * wu
    # 16 steps of the activation, one of the product with u; past g = -88 the exponential
    # stays where it is there: off by less than e^-88 |g u| < 2^-126 |g u|
    check(h, want, 17 * U * want.abs() + 2.0 ** -126 * (wg * wu).abs(), "h")
    assert untouched(full, N) and untouched(gf, N) and untouched(uf, N)


@pytest.mark.parametrize("N", [1999, 100, 40])
@pytest.mark.parametrize("pads", [(8, 8), (8, 16)])
def test_gated_gradients(pads, N):
    """Both weights' strides alike and not (only alike take the large tiles for dx)."""
    import torch
    sdt, t = _sdt(), torch.bfloat16
    M, K = 4000, 3900
    say(f"large gradients {M}x{N}x{K} {pads}")
    x, dh = operand(M, K, t, 1), operand(M, N, t, 2)
    gate, up = operand(N, K, t, 3, pads[0]), operand(N, K, t, 4, pads[1])
    # a'(0) = 1/2 and a(0) = 0 in the rows' first half: dg = dh u / 2, du = 0; u = 0
    # after it: dg = 0.  There g = 40, where a(g) = 40 in fp32: du = 40 dh, whole and
    # below 128.
    g = torch.zeros(M, N, device=DEV)
    g[:, N // 2:] = 40.0
    u = whole((M, N), torch.float32, 5)
    u[:, N // 2:] = 0.0
    g, u = rows_of(g, 1, align=4)[0], rows_of(u, 1, align=4)[0]
    dx, fx = out_like(M, K, t, pad=8)
    dgate, fg = out_like(N, K, t, pad=8)
    dup, fu = out_like(N, K, t, pad=16)
    ws = torch.empty(sdt.gated_ff_workspace_size(M, N, K), dtype=torch.uint8, device=DEV)
    sdt.gated_ff_backward(x, gate, up, g, u, dh, dx, dgate, dup, ws)
    dg = torch.where(g == 0, dh.double() * u.double() / 2, 0.0)
    du = torch.where(g == 0, 0.0, 40.0 * dh.double())
    # sums of halves up to 13.5 N and of whole numbers up to 360 N: below 2^24 halves
    assert torch.equal(dx, (dg @ gate.double() + du @ up.double()).float().to(t))
    assert torch.equal(dgate, (dg.t() @ x.double()).float().to(t))
    assert torch.equal(dup, (du.t() @ x.double()).float().to(t))
    assert untouched(fx, K) and untouched(fg, K) and untouched(fu, K)

"""MX4 products of large grids (128 x 128 and 256 x 256 tiles) and quantisation past
the caches, against the 64-bit definitions of mx4_reference: whole numbers bit for
bit, others within the bound of their roundings (test_gpu_mx4)."""
import numpy as np
import pytest

import mx4_reference as ref
from gpu_helpers import DEV, say
from test_gpu_mx4 import _sdt, _t, device_matrix, product_bound, random_matrix, run_gemm

pytestmark = pytest.mark.gpu

TYPES = ["f16", "bf16"]


# k-tiles of 256: one (whole and partial), two, three, four and seven; grids that
# are not and that are made of 16 x 16 blocks
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,N,K", [(2900, 3100, 32), (2817, 2818, 256), (2900, 3100, 257),
                                   (3300, 2570, 700), (4096, 3841, 1000), (4090, 4096, 1700)])
def test_gemm_whole_numbers(dtype, M, N, K):
    import torch
    rng = np.random.default_rng(M * 7 + N * 3 + K)
    ca, sa = random_matrix(M, K, rng, whole=True)
    cb, sb = random_matrix(N, K, rng, whole=True)
    say(f"large gemm whole {dtype} {M}x{N}x{K}")
    got = run_gemm(dtype, device_matrix(ca, sa, M, K, 16), device_matrix(cb, sb, N, K, 48), M, N)
    # sums of products of at most 36 over K <= 2^15: whole numbers below 2^24
    want = torch.from_numpy(ref.values(ca, sa, K).astype(np.float32)
                            @ ref.values(cb, sb, K).astype(np.float32).T)
    assert torch.equal(got, want.to(_t(dtype)))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,N,K", [(2900, 3100, 530), (3000, 2900, 1311)])
def test_gemm_random(dtype, M, N, K):
    rng = np.random.default_rng(M + N * 5 + K * 11)
    ca, sa = random_matrix(M, K, rng)
    cb, sb = random_matrix(N, K, rng)
    sa = np.maximum(sa, 12) - 10                     # fp16's range
    say(f"large gemm random {dtype} {M}x{N}x{K}")
    got = run_gemm(dtype, device_matrix(ca, sa, M, K), device_matrix(cb, sb, N, K), M, N)
    a, b = ref.values(ca, sa, K), ref.values(cb, sb, K)
    want = a @ b.T
    err = np.abs(got.double().numpy() - want)
    assert (err <= product_bound(a, b, want, dtype)).all()


def test_gemm_far_scales_and_nan():
    """Scales at both ends of their range, and NaN blocks: exactly their rows."""
    import torch
    rng = np.random.default_rng(3)
    M, N, K = 2900, 3100, 600
    ca, sa = random_matrix(M, K, rng, whole=True)
    cb, sb = random_matrix(N, K, rng, whole=True)
    sa[:] = 0                                        # 2^-127
    sb[:] = 254                                      # 2^127
    sa[M - 1, 18] = 255
    sa[130, 2] = 255
    sb[0, 9] = 255
    want = torch.from_numpy(ref.values(ca, sa, K) @ ref.values(cb, sb, K).T).float().bfloat16()
    nan = np.zeros((M, N), dtype=bool)
    nan[[130, M - 1]] = True
    nan[:, 0] = True
    say("large gemm far and nan scales")
    got = run_gemm("bf16", device_matrix(ca, sa, M, K), device_matrix(cb, sb, N, K), M, N)
    assert np.array_equal(torch.isnan(got).numpy(), nan)
    ok = ~torch.from_numpy(nan)
    assert torch.equal(got[ok], want[ok])


def test_gemm_empty_k():
    import torch
    sdt = _sdt()
    M, N = 2900, 3104
    c = torch.full((M, N), float("nan"), dtype=torch.float16, device=DEV)
    say("large gemm empty k")
    sdt.gemm_mx4_f16(sdt.Mx4.empty(M, 0, device=DEV), sdt.Mx4.empty(N, 0, device=DEV), c)
    torch.cuda.synchronize()
    assert bool((c == 0).all())


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,K,ld", [(4100, 8190, 8193), (33, 1048577, 1048584), (131100, 257, 257)])
def test_quantize_past_the_caches(dtype, rows, K, ld):
    """Matrices of 2^25 elements and more against 256 rows at a time (whose values
    test_gpu_mx4 compares with the definition), and some rows against it here."""
    import torch
    sdt = _sdt()
    g = torch.Generator(device=DEV).manual_seed(rows)
    x = torch.randn(rows, ld, device=DEV, generator=g).to(_t(dtype))[:, :K]
    x[rows - 1, K - 1] = float("nan")
    m = sdt.Mx4.empty(rows, K, device=DEV)
    m.q.fill_(0xee)
    m.s.fill_(0xee)
    y = torch.full((rows, ld), 7.0, dtype=_t(dtype), device=DEV)
    say(f"quantize past the caches {dtype} {rows}x{K}")
    getattr(sdt, f"mx4_quantize_{dtype}")(x, m)
    getattr(sdt, f"mx4_dequantize_{dtype}")(m, y[:, :K])
    torch.cuda.synchronize()
    assert bool((y[:, K:] == 7.0).all())
    tile_rows = -(-K // 256) * 512                   # scale bytes of 64 rows
    for r in range(0, rows, 256):
        n = min(256, rows - r)
        p = sdt.Mx4.empty(n, K, device=DEV)
        v = torch.empty(n, K, dtype=_t(dtype), device=DEV)
        getattr(sdt, f"mx4_quantize_{dtype}")(x[r:r + n], p)
        getattr(sdt, f"mx4_dequantize_{dtype}")(p, v)
        assert torch.equal(p.q, m.q[r:r + n])
        assert torch.equal(p.s, m.s[r // 64 * tile_rows:][:p.s.numel()])
        got = y[r:r + n, :K]
        assert torch.equal(torch.isnan(got), torch.isnan(v))
        assert torch.equal(torch.nan_to_num(got), torch.nan_to_num(v))
    for r in (0, rows // 2, rows - 1):
        codes, scales = ref.quantize(x[r:r + 1].double().cpu().numpy())
        assert np.array_equal(m.q[r].cpu().numpy(), ref.pack(codes)[0])
        want = torch.from_numpy(ref.values(codes, scales, K)).to(_t(dtype))[0]
        got = y[r, :K].cpu()
        assert torch.equal(torch.isnan(got), torch.isnan(want))
        assert torch.equal(torch.nan_to_num(got), torch.nan_to_num(want))


# grids of one full round of 256 x 256 tiles (the larger tiles' rule takes them at
# every K), ragged, and of two rounds
@pytest.mark.parametrize("M,N,K", [(4000, 4090, 32), (3850, 4096, 256), (4096, 4001, 300),
                                   (4090, 3849, 700), (4096, 4096, 1025), (8000, 4090, 512)])
def test_gemm_full_rounds(M, N, K):
    import torch
    rng = np.random.default_rng(M + N + K)
    ca, sa = random_matrix(M, K, rng, whole=True)
    cb, sb = random_matrix(N, K, rng, whole=True)
    say(f"full rounds {M}x{N}x{K}")
    got = run_gemm("f16", device_matrix(ca, sa, M, K, 16), device_matrix(cb, sb, N, K, 48), M, N)
    want = torch.from_numpy(ref.values(ca, sa, K).astype(np.float32)
                            @ ref.values(cb, sb, K).astype(np.float32).T)
    assert torch.equal(got, want.half())


def test_gemm_full_round_random_far_and_nan():
    import torch
    rng = np.random.default_rng(77)
    M, N, K = 4000, 4090, 1311
    ca, sa = random_matrix(M, K, rng)
    cb, sb = random_matrix(N, K, rng)
    say("full round random")
    got = run_gemm("bf16", device_matrix(ca, sa, M, K), device_matrix(cb, sb, N, K), M, N)
    a, b = ref.values(ca, sa, K), ref.values(cb, sb, K)
    want = a @ b.T
    err = np.abs(got.double().numpy() - want)
    assert (err <= product_bound(a, b, want, "bf16")).all()
    ca, sa = random_matrix(M, K, rng, whole=True)
    cb, sb = random_matrix(N, K, rng, whole=True)
    sa[:] = 0                                        # 2^-127
    sb[:] = 254                                      # 2^127
    sa[M - 1, 40] = 255
    sa[130, 2] = 255
    sb[0, 9] = 255
    want = torch.from_numpy(ref.values(ca, sa, K) @ ref.values(cb, sb, K).T).float().bfloat16()
    nan = np.zeros((M, N), dtype=bool)
    nan[[130, M - 1]] = True
    nan[:, 0] = True
    say("full round far and nan scales")
    got = run_gemm("bf16", device_matrix(ca, sa, M, K), device_matrix(cb, sb, N, K), M, N)
    assert np.array_equal(torch.isnan(got).numpy(), nan)
    ok = ~torch.from_numpy(nan)
    assert torch.equal(got[ok], want[ok])


def test_gemm_full_round_empty_k():
    import torch
    sdt = _sdt()
    M, N = 4000, 4096
    c = torch.full((M, N), float("nan"), dtype=torch.float16, device=DEV)
    say("full round empty k")
    sdt.gemm_mx4_f16(sdt.Mx4.empty(M, 0, device=DEV), sdt.Mx4.empty(N, 0, device=DEV), c)
    torch.cuda.synchronize()
    assert bool((c == 0).all())


# between one 64 x 64 and one 64 x 128 tile a CU; few rows in two groups
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,N,K", [(500, 4000, 33), (500, 4000, 300), (449, 3970, 700),
                                   (512, 4096, 1100), (500, 4000, 2100), (65, 1000, 600),
                                   (100, 4001, 1300), (128, 8000, 257)])
def test_gemm_middle_sizes(dtype, M, N, K):
    import torch
    rng = np.random.default_rng(M + N + 2 * K)
    ca, sa = random_matrix(M, K, rng, whole=True)
    cb, sb = random_matrix(N, K, rng, whole=True)
    say(f"middle sizes {dtype} {M}x{N}x{K}")
    got = run_gemm(dtype, device_matrix(ca, sa, M, K, 16), device_matrix(cb, sb, N, K, 48), M, N)
    want = torch.from_numpy(ref.values(ca, sa, K).astype(np.float32)
                            @ ref.values(cb, sb, K).astype(np.float32).T)
    assert torch.equal(got, want.to(_t(dtype)))

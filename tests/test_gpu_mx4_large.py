"""MX4 products whose grids run the 256 x 256 tiles, against the 64-bit
definitions of mx4_reference: whole numbers bit for bit, others within the bound
of their roundings (test_gpu_mx4)."""
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

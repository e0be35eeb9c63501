"""Products between one and two rounds of 128 x 128 tiles, where either tile size may be
taken: whole numbers bit for bit, whichever runs."""
import pytest

import test_gpu_ffn_large as large

pytestmark = pytest.mark.gpu

# 520 to 740 tiles of 128 x 128, 130 to 192 of 256 x 256; a k-tile and less, several, many
SIZES = [(3000, 2999, 1001), (2560, 4090, 130), (2300, 4090, 50), (1720, 6353, 520), (2560, 3328, 2050), (2900, 4096, 0)]


@pytest.mark.parametrize("layout", ["nn", "tn"])
@pytest.mark.parametrize("M, N, K", SIZES)
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_turned(dtype, M, N, K, layout):
    large.test_turned(dtype, M, N, K, layout)


@pytest.mark.parametrize("M, N, K", SIZES)
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_fp8(dtype, M, N, K):
    large.test_fp8(dtype, M, N, K)


@pytest.mark.parametrize("M, N, K", [(3000, 1499, 1001), (2560, 2045, 130), (1720, 3177, 520), (2900, 2048, 0)])
@pytest.mark.parametrize("wide", [True, False])
def test_gated(M, N, K, wide):
    large.test_gated(M, N, K, wide)

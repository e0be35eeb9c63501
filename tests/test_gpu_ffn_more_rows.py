"""The row-wise kernels at the sizes where a workgroup takes several rows at a time (short
rows from 32768 on, values back from 8192 row tiles on) and around, where a workgroup of the norm's gradient takes rows in turn, and the signs of
zeros among the codes."""
import numpy as np
import pytest

import ffn_reference as ref
import test_gpu_ffn as base
from gpu_helpers import DEV, say
from test_gpu_ffn import normal, out_like, rows_of, untouched

pytestmark = pytest.mark.gpu

TYPES = ["f16", "bf16"]


def _sdt():
    from shape_driven_tile_amd import binding
    return binding


def _t(name):
    import torch
    return {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}[name]


def quantized(x, block):
    """Code values (fp32) and scales of x, by the definition: ref.quantize for whole matrices."""
    rows, K = x.shape
    kb, height = -(-K // 128), 1 if block == 1 else 128
    nb = -(-rows // height)
    v = np.zeros((nb * height, kb * 128))
    v[:rows, :K] = x
    t = v.reshape(nb, height, kb, 128)
    top = np.abs(t).max(axis=(1, 3)).astype(np.float32)
    scales = np.maximum(top / np.float32(448.0), ref.SMALLEST_SCALE)
    codes = ref.e4m3(t.astype(np.float32) / scales[:, None, :, None])
    codes = codes.reshape(nb * height, kb * 128)[:rows, :K]
    return codes.astype(np.float32), np.ascontiguousarray(scales.T) if block == 1 else scales


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("block", [1, 128])
@pytest.mark.parametrize("rows, K, pad", [(4096, 8, 0), (5003, 9, 0), (4099, 130, 1), (4101, 7, 0), (2051, 2100, 4),
                                          (1371, 4097, 0), (8200, 300, 0), (4100, 2050, 1), (32768, 8, 0),
                                          (33001, 9, 2), (32771, 130, 0), (40003, 33, 0), (32769, 7, 0)])
def test_quantize_many_rows(dtype, block, rows, K, pad):
    import torch
    say(f"quantize many rows {dtype} block {block} {rows}x{K}+{pad}")
    sdt, t = _sdt(), _t(dtype)
    v = normal((rows, K), t, 1)
    v[:, ::7] *= 12
    v.view(-1)[::97] = 0
    x, _ = rows_of(v, pad, align=1)
    m = sdt.Fp8.empty(rows, K, block=block, device=DEV)
    full = m.q if m.q.shape[1] == m.q.stride(0) else m.q.as_strided((rows, m.q.stride(0)), m.q.stride())
    full.view(torch.uint8).fill_(0x55)
    getattr(sdt, f"fp8_quantize_{dtype}")(x, m)
    codes, scales = quantized(x.double().cpu().numpy(), block)
    assert np.array_equal(m.s.cpu().numpy(), scales)
    assert np.array_equal(m.q.float().cpu().numpy(), codes)
    if full.shape[1] > K:
        assert bool((full.view(torch.uint8)[:, K:] == 0x55).all())
    want = codes * ref.scale_map(scales, block, rows, K)
    for out in ("f32", "f16", "bf16"):
        y, rest = out_like(rows, K, _t(out), pad, align=1)
        getattr(sdt, f"fp8_dequantize_{out}")(m, y)
        assert torch.equal(y, torch.from_numpy(want).to(DEV).to(_t(out))), out
        assert untouched(rest, K)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("block", [1, 128])
@pytest.mark.parametrize("rows", [3, 5000, 33000])
def test_signs_of_zeros(dtype, block, rows):
    """The quotient's sign is the code's, of zeros and of quotients that round to zero."""
    import torch
    sdt, t = _sdt(), _t(dtype)
    say(f"signs of zeros {dtype} block {block} {rows}")
    x = normal((rows, 200), t, 2)
    x[:, 1::5] = 0.0
    x[:, 2::5] = -0.0
    x[:, 3::5] *= 2.0 ** -13
    x[rows // 2, :128] = -0.0                                # a row's block of nothing else
    m = sdt.Fp8.empty(rows, 200, block=block, device=DEV)
    getattr(sdt, f"fp8_quantize_{dtype}")(x, m)
    negative = (m.q.view(torch.uint8) & 0x80) != 0
    assert torch.equal(negative, torch.signbit(x))
    y = torch.empty_like(x)
    getattr(sdt, f"fp8_dequantize_{dtype}")(m, y)
    assert torch.equal(torch.signbit(y), torch.signbit(x))
    # the norm's rows in 8 bits
    q = sdt.Fp8.empty(rows, 200, device=DEV)
    sdt.rms_norm(x, None, q=q)
    assert torch.equal((q.q.view(torch.uint8) & 0x80) != 0, torch.signbit(x))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M, N, K", [(4099, 70, 40), (2050, 2060, 72), (5000, 1, 8), (32771, 70, 40),
                                     (33000, 3, 8)])
@pytest.mark.parametrize("act, kept", [("silu", "wide"), ("gelu", "type")])
def test_gated_backward_many_rows(dtype, M, N, K, act, kept):
    base.test_gated_backward(dtype, M, N, K, act, kept)


# one wave a row, four rows a workgroup; then one to four chunks a lane, 128 to 1024 lanes
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows, K", [(4100, 300), (1100, 1000), (1030, 4097), (700, 8170), (530, 16390)])
@pytest.mark.parametrize("weight, extra, pad", [(True, True, 0), (False, False, 3)])
def test_norm_backward_rows_in_turn(dtype, rows, K, weight, extra, pad):
    base.test_norm_backward(dtype, rows, K, weight, extra, pad)

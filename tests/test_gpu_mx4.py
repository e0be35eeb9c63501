"""MX4 quantisation, the values back and the products on the GPU, against the
64-bit definitions of mx4_reference.  Codes, scales and values are compared bit
for bit.  A product's bound counts its roundings: K additions in fp32, each off
by at most half a step (2^-24) of a running sum no larger than sum |a b|, and
half a step of the output type; on operands whose products and sums are whole
numbers below 2^24 it is exact before that last rounding."""
import numpy as np
import pytest

import mx4_reference as ref
from gpu_helpers import DEV, say

pytestmark = pytest.mark.gpu

TYPES = ["f16", "bf16"]


def _t(name):
    import torch
    return {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}[name]


def _sdt():
    from shape_driven_tile_amd import binding
    return binding


def device_matrix(codes, scales, rows, K, pad=0):
    """An Mx4 on the device from codes and row-major scales; `pad` extra bytes
    (16 at a time) between rows, filled with junk."""
    import torch
    sdt = _sdt()
    nb16 = ref.row_bytes(K)
    q = np.random.default_rng(5).integers(0, 256, (rows, nb16 + pad), dtype=np.uint8)
    q[:, :nb16] = ref.pack(codes)
    return sdt.Mx4(torch.from_numpy(q).to(DEV),
                   torch.from_numpy(ref.tile_scales(scales, rows, K)).to(DEV), rows, K)


def random_matrix(rows, K, rng, whole=False):
    """Random codes and scales (whole: the scales make every value a whole number
    of magnitude at most 6, so sums of up to 4e5 products stay below 2^24)."""
    nb = -(-K // 32)
    codes = rng.integers(0, 16, (rows, nb * 32), dtype=np.uint8)
    codes[:, K:] = 0
    if whole:
        codes = np.where(np.isin(codes & 7, [1, 3]), codes & 8, codes)   # no halves
        scales = np.full((rows, nb), 127, dtype=np.uint8)
    else:
        scales = rng.integers(120, 134, (rows, nb), dtype=np.uint8)
    return codes.astype(np.uint8), scales


def product_bound(a, b, out, dtype):
    """|error| of a product: see the module's docstring."""
    import torch
    step = torch.finfo(_t(dtype)).eps / 2
    tiny = 2.0 ** -24 if dtype == "f16" else 2.0 ** -133
    K = a.shape[1]
    acc = (K + 1) * 2.0 ** -24 * (np.abs(a) @ np.abs(b).T)
    return acc * (1 + step) + step * np.abs(out) + tiny / 2


# ---- quantisation -----------------------------------------------------------------


@pytest.mark.parametrize("dtype", TYPES)
def test_quantize_every_pattern(dtype):
    """Every 16-bit pattern, in blocks of random company (infinities and NaN among
    it), in blocks of finite values, and in blocks of like magnitude, where ties
    and every code occur."""
    import torch
    sdt = _sdt()
    rng = np.random.default_rng(1)
    every = rng.permutation(65536).astype(np.uint16)
    mag = 0x7BFF if dtype == "f16" else 0x7F7F
    finite = every[(every & 0x7FFF) <= mag][:63488 // 256 * 256]
    ordered = np.arange(65536, dtype=np.uint16)
    ordered = ordered[(ordered & 0x7FFF) <= mag]
    ordered = ordered[:len(ordered) // 256 * 256]
    # like magnitudes: 32 patterns with one exponent or its two neighbours below
    frac = 10 if dtype == "f16" else 7
    near = []
    for e in range(0, 31 if dtype == "f16" else 255):
        ex = np.maximum(e - rng.integers(0, 4, 256), 0)
        near.append((ex << frac) | rng.integers(0, 8, 256) << (frac - 3) | (rng.integers(0, 2, 256) << 15))
    near = np.concatenate(near).astype(np.uint16)
    for name, bits in (("every", every), ("finite", finite), ("ordered", ordered), ("near", near)):
        say(f"quantize patterns {dtype} {name}")
        x = torch.from_numpy(bits.reshape(-1, 256).view(np.int16).copy()).view(_t(dtype))
        want_c, want_s = ref.quantize(x.double().numpy())
        m = sdt.Mx4.empty(x.shape[0], 256, device=DEV)
        getattr(sdt, f"mx4_quantize_{dtype}")(x.to(DEV), m)
        torch.cuda.synchronize()
        got_s = m.s.cpu().numpy()
        assert np.array_equal(got_s, ref.tile_scales(want_s, x.shape[0], 256)), name
        got = ref.unpack(m.q.cpu().numpy())
        bad = np.argwhere(got != want_c)
        assert bad.size == 0, (name, len(bad), bad[0], x[tuple(bad[0])].item(),
                               got[tuple(bad[0])], want_c[tuple(bad[0])],
                               want_s[bad[0][0], bad[0][1] // 32])


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,K,extra,shift", [
    (1, 1, 0, 0), (1, 31, 0, 0), (1, 4096, 0, 0), (2, 32, 0, 1), (63, 33, 3, 0), (64, 256, 0, 0),
    (65, 255, 1, 3), (130, 257, 7, 0), (7, 1000, 0, 0), (200, 520, 8, 0)])
def test_quantize_shapes(dtype, rows, K, extra, shift):
    """Odd sizes, strides and alignments; padding of the codes' rows untouched."""
    import torch
    sdt = _sdt()
    g = torch.Generator().manual_seed(rows * 1000 + K)
    flat = (torch.randn(rows * (K + extra) + shift, generator=g) * 3).to(_t(dtype))
    x = flat[shift:].view(rows, K + extra)[:, :K]
    want_c, want_s = ref.quantize(x.double().numpy())
    rb = ref.row_bytes(K)
    q = torch.full((rows, rb + 32), 0xA5, dtype=torch.uint8, device=DEV)
    s = torch.full((ref.scale_bytes(rows, K),), 0xA5, dtype=torch.uint8, device=DEV)
    m = sdt.Mx4(q[:, :rb] if rows > 1 else q[:, :rb], s, rows, K)
    dx = flat.to(DEV)[shift:].view(rows, K + extra)[:, :K]
    say(f"quantize {dtype} {rows}x{K}+{extra} shift {shift}")
    getattr(sdt, f"mx4_quantize_{dtype}")(dx, m)
    torch.cuda.synchronize()
    assert np.array_equal(ref.unpack(q[:, :rb].cpu().numpy()), want_c)
    assert np.array_equal(s.cpu().numpy(), ref.tile_scales(want_s, rows, K))
    assert bool((q[:, rb:] == 0xA5).all())


@pytest.mark.parametrize("dtype", TYPES)
def test_quantize_rows_by_list(dtype):
    """Rows named by a list: divided, negative and outside entries, rows in place."""
    import torch
    sdt = _sdt()
    rng = np.random.default_rng(3)
    K, T = 300, 9
    x = torch.from_numpy(rng.standard_normal((T, K))).to(_t(dtype))
    codes, scales = ref.quantize(x.double().numpy())
    index = rng.integers(-2, T * 3, 130).astype(np.int32)
    index[64:128] = -1
    index[5], index[6] = T * 3, T * 3 + 500        # outside X
    for divisor in (3, 0):
        src = index // 3 if divisor else np.arange(130)
        ok = (index >= 0) & (src < T)
        src = np.where(ok, src, 0)
        rb = ref.row_bytes(K)
        q = torch.full((130, rb), 0xA5, dtype=torch.uint8, device=DEV)
        m = sdt.Mx4(q, torch.full((ref.scale_bytes(130, K),), 0xA5, dtype=torch.uint8, device=DEV),
                    130, K)
        say(f"quantize rows {dtype} divisor {divisor}")
        getattr(sdt, f"mx4_quantize_rows_{dtype}")(x.to(DEV), torch.from_numpy(index).to(DEV),
                                                   divisor, m)
        torch.cuda.synchronize()
        want_q = np.where(ok[:, None], ref.pack(codes)[src], 0xA5)
        want_s = np.where(ok[:, None], scales[src], 0)
        assert np.array_equal(q.cpu().numpy(), want_q)
        assert np.array_equal(m.s.cpu().numpy(), ref.tile_scales(want_s, 130, K))


@pytest.mark.parametrize("dtype", TYPES + ["f32"])
def test_dequantize_every_code_and_scale(dtype):
    import torch
    sdt = _sdt()
    rows, K = 256, 52                     # row r: scale byte r; a partial second block
    codes = np.tile(np.arange(64, dtype=np.uint8) % 16, (rows, 1))
    codes[:, K:] = 0
    scales = np.tile(np.arange(256, dtype=np.uint8)[:, None], (1, 2))
    m = device_matrix(codes, scales, rows, K, pad=16)
    for ld in (52, 53, 56):
        y = torch.full((rows, ld), -7.0, dtype=_t(dtype), device=DEV)
        say(f"dequantize {dtype} ld {ld}")
        getattr(sdt, f"mx4_dequantize_{dtype}")(m, y[:, :K])
        torch.cuda.synchronize()
        want = torch.from_numpy(ref.values(codes, scales, K)).float().to(_t(dtype))
        got = y[:, :K].cpu()
        assert torch.equal(torch.isnan(got), torch.isnan(want))
        assert torch.equal(got.nan_to_num(0.5, 1e30, -1e30).float(),
                           want.nan_to_num(0.5, 1e30, -1e30).float())
        assert bool((y[:, K:] == -7.0).all())


def test_pack_scales():
    import torch
    sdt = _sdt()
    rng = np.random.default_rng(9)
    for rows, K in ((1, 1), (64, 256), (65, 257), (200, 1000)):
        sc = rng.integers(0, 256, (rows, -(-K // 32)), dtype=np.uint8)
        m = sdt.Mx4.empty(rows, K, device=DEV)
        m.s.fill_(0xA5)
        say(f"pack scales {rows}x{K}")
        sdt.mx4_pack_scales(torch.from_numpy(sc).to(DEV), m)
        torch.cuda.synchronize()
        assert np.array_equal(m.s.cpu().numpy(), ref.tile_scales(sc, rows, K))


# ---- products -----------------------------------------------------------------------

SHAPES = [(1, 1, 1), (1, 64, 32), (2, 17, 33), (15, 33, 256), (16, 100, 257), (17, 129, 1000),
          (33, 64, 2048), (64, 300, 700), (65, 40, 100), (100, 200, 300), (128, 128, 512),
          (129, 257, 1111), (300, 515, 2300), (1500, 1100, 640)]


def run_gemm(dtype, a, b, M, N):
    import torch
    sdt = _sdt()
    ld = -(-N // 8) * 8 + 8
    full = torch.full((M, ld), float("nan"), dtype=_t(dtype), device=DEV)
    getattr(sdt, f"gemm_mx4_{dtype}")(a, b, full[:, :N])
    torch.cuda.synchronize()
    assert bool(torch.isnan(full[:, N:]).all()), "padding of C was written"
    return full[:, :N].cpu()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_gemm_whole_numbers(dtype, M, N, K):
    import torch
    rng = np.random.default_rng(M * 7 + N * 3 + K)
    ca, sa = random_matrix(M, K, rng, whole=True)
    cb, sb = random_matrix(N, K, rng, whole=True)
    say(f"gemm whole {dtype} {M}x{N}x{K}")
    got = run_gemm(dtype, device_matrix(ca, sa, M, K, 16), device_matrix(cb, sb, N, K, 48), M, N)
    want = torch.from_numpy(ref.values(ca, sa, K) @ ref.values(cb, sb, K).T).float().to(_t(dtype))
    assert torch.equal(got, want)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_gemm_random(dtype, M, N, K):
    rng = np.random.default_rng(M + N * 5 + K * 11)
    ca, sa = random_matrix(M, K, rng)
    cb, sb = random_matrix(N, K, rng)
    sa = np.maximum(sa, 12) - 10                     # fp16's range
    say(f"gemm random {dtype} {M}x{N}x{K}")
    got = run_gemm(dtype, device_matrix(ca, sa, M, K), device_matrix(cb, sb, N, K), M, N)
    a, b = ref.values(ca, sa, K), ref.values(cb, sb, K)
    want = a @ b.T
    err = np.abs(got.double().numpy() - want)
    assert (err <= product_bound(a, b, want, dtype)).all()


@pytest.mark.parametrize("M", [1, 16, 80, 200])
def test_gemm_far_scales_and_nan(M):
    """Scales at both ends of their range, and NaN blocks: exactly their rows."""
    import torch
    rng = np.random.default_rng(M)
    N, K = 70, 300
    ca, sa = random_matrix(M, K, rng, whole=True)
    cb, sb = random_matrix(N, K, rng, whole=True)
    sa[:] = 0                                        # 2^-127
    sb[:] = 254                                      # 2^127
    a1 = device_matrix(ca, sa, M, K)
    want = torch.from_numpy(ref.values(ca, sa, K) @ ref.values(cb, sb, K).T).float().bfloat16()
    say(f"gemm far scales M {M}")
    assert torch.equal(run_gemm("bf16", a1, device_matrix(cb, sb, N, K), M, N), want)
    sa[M // 2, 3] = 255
    sb[11, 0] = 255
    nan = np.zeros((M, N), dtype=bool)
    nan[M // 2] = True
    nan[:, 11] = True
    say(f"gemm nan scales M {M}")
    got = run_gemm("bf16", device_matrix(ca, sa, M, K), device_matrix(cb, sb, N, K), M, N)
    assert np.array_equal(torch.isnan(got).numpy(), nan)
    assert torch.equal(got[~torch.from_numpy(nan)], want[~torch.from_numpy(nan)])


@pytest.mark.parametrize("dtype", TYPES)
def test_gemm_empty(dtype):
    import torch
    sdt = _sdt()
    for M, N in ((3, 5), (100, 130)):
        c = torch.full((M, -(-N // 8) * 8), float("nan"), dtype=_t(dtype), device=DEV)
        a, b = sdt.Mx4.empty(M, 0, device=DEV), sdt.Mx4.empty(N, 0, device=DEV)
        say(f"gemm empty k {dtype} {M}x{N}")
        getattr(sdt, f"gemm_mx4_{dtype}")(a, b, c[:, :N])
        torch.cuda.synchronize()
        assert bool((c[:, :N] == 0).all()) and bool(torch.isnan(c[:, N:]).all())
    y = torch.full((7,), float("nan"), dtype=_t(dtype), device=DEV)
    x = torch.empty(0, dtype=_t(dtype), device=DEV)
    getattr(sdt, f"gemv_mx4_m1_{dtype}")(x, sdt.Mx4.empty(7, 0, device=DEV), y)
    torch.cuda.synchronize()
    assert bool((y == 0).all())


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("N,K,shift", [(1, 1, 0), (5, 31, 0), (16, 32, 1), (17, 33, 0), (64, 256, 0),
                                       (100, 257, 3), (1000, 1000, 0), (515, 4100, 0),
                                       (4099, 1000, 0), (300, 12300, 8)])
def test_gemv(dtype, N, K, shift):
    """x holds an infinity and a NaN past its K values: neither may be read."""
    import torch
    sdt = _sdt()
    rng = np.random.default_rng(N + K)
    cb, sb = random_matrix(N, K, rng)
    sb = sb - 7
    flat = torch.from_numpy(rng.standard_normal(shift + K + 40)).to(_t(dtype))
    flat[shift + K:shift + K + 20] = float("inf")
    flat[shift + K + 20:] = float("nan")
    x = flat.to(DEV)[shift:shift + K]
    y = torch.full((N + 8,), -7.0, dtype=_t(dtype), device=DEV)
    say(f"gemv {dtype} {N}x{K} shift {shift}")
    getattr(sdt, f"gemv_mx4_m1_{dtype}")(x, device_matrix(cb, sb, N, K, 16), y[:N])
    torch.cuda.synchronize()
    a, b = flat[shift:shift + K].double().numpy()[None], ref.values(cb, sb, K)
    want = (a @ b.T)
    # the block sums are multiplied by their scale in fp32: exact (a power of two)
    err = np.abs(y[:N].double().cpu().numpy() - want[0])
    assert (err <= product_bound(a, b, want, dtype)[0]).all()
    assert bool((y[N:] == -7.0).all())


def test_side_stream_and_graph():
    """The products on a stream of their own, and captured into a graph that is
    replayed between eager calls: the same bits every time."""
    import torch
    sdt = _sdt()
    rng = np.random.default_rng(77)
    a = device_matrix(*random_matrix(200, 512, rng, whole=True), 200, 512)
    b = device_matrix(*random_matrix(136, 512, rng, whole=True), 136, 512)
    x = torch.from_numpy(rng.standard_normal((200, 512))).to(torch.bfloat16).to(DEV)
    want = torch.empty(200, 136, dtype=torch.bfloat16, device=DEV)
    say("mx4 side stream")
    m = sdt.Mx4.empty(200, 512, device=DEV)
    sdt.mx4_quantize_bf16(x, m)
    sdt.gemm_mx4_bf16(m, b, want)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    c = torch.zeros_like(want)
    m2 = sdt.Mx4.empty(200, 512, device=DEV)
    side.wait_stream(torch.cuda.current_stream())
    sdt.mx4_quantize_bf16(x, m2, stream=side)
    sdt.gemm_mx4_bf16(m2, b, c, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(c, want)
    say("mx4 graph")
    c.zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sdt.mx4_quantize_bf16(x, m2)
        sdt.gemm_mx4_bf16(m2, b, c)
    for _ in range(3):
        c.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(c, want)
        sdt.gemm_mx4_bf16(a, b, c)
        torch.cuda.synchronize()

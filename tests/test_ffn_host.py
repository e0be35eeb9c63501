"""Refusals and sizes of the 8-bit, norm, gated feed-forward and turned-product entry
points, on the host: every call here is refused (or has nothing to do) before
anything is enqueued."""
import ctypes

import pytest

from shape_driven_tile_amd import binding as sdt

OK, INVALID, UNSUPPORTED = sdt.SDT_OK, sdt.SDT_ERR_INVALID_ARG, sdt.SDT_ERR_UNSUPPORTED
P = 0x10000          # an address that is never read


def fp8(a, names):
    """An sdt_fp8 of some of a's values, which leave it."""
    return ctypes.byref(sdt.SdtFp8(*[a.pop(n) for n in names]))


def call(name, *args):
    return int(getattr(sdt.lib(), name)(*args))


@pytest.mark.parametrize("t", ["f16", "bf16"])
@pytest.mark.parametrize("change, want", [
    ({}, None), ({"rows": -1}, INVALID), ({"K": -1}, INVALID), ({"ldx": 199}, INVALID),
    ({"X": None}, INVALID), ({"Q": None}, INVALID), ({"S": None}, INVALID), ({"block": 64}, INVALID),
    ({"ldq": 192}, INVALID), ({"ldq": 200}, UNSUPPORTED), ({"lds": 9}, INVALID),
    ({"block": 128, "lds": 1}, INVALID), ({"X": P + 1}, UNSUPPORTED), ({"Q": P + 8}, UNSUPPORTED),
    ({"S": P + 2}, UNSUPPORTED), ({"ldq": 1 << 23}, UNSUPPORTED),
    ({"K": 1 << 24, "ldx": 1 << 24, "ldq": 1 << 24}, UNSUPPORTED), ({"lds": 1 << 31}, UNSUPPORTED),
    ({"rows": 0}, OK), ({"K": 0}, OK), ({"rows": 0, "block": 3}, INVALID),
])
def test_quantize_refusals(t, change, want):
    a = dict(rows=10, K=200, X=P, ldx=200, Q=P, ldq=208, S=P, lds=10, block=1)
    a.update(change)
    if want is None:
        return            # the base case would launch: the GPU tests run it
    out = fp8(a, ("Q", "ldq", "S", "lds", "block"))
    assert call(f"fp8_quantize_{t}", *a.values(), out, None) == want


@pytest.mark.parametrize("t", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("change, want", [
    ({"rows": -1}, INVALID), ({"ldy": 199}, INVALID), ({"Y": None}, INVALID), ({"S": None}, INVALID),
    ({"Y": P + 1}, UNSUPPORTED), ({"ldq": 207}, UNSUPPORTED), ({"rows": 0}, OK), ({"K": 0}, OK),
])
def test_dequantize_refusals(t, change, want):
    a = dict(rows=10, K=200, Q=P, ldq=208, S=P, lds=10, block=1, Y=P, ldy=200)
    a.update(change)
    m = fp8(a, ("Q", "ldq", "S", "lds", "block"))
    assert call(f"fp8_dequantize_{t}", a["rows"], a["K"], m, a["Y"], a["ldy"], None) == want


@pytest.mark.parametrize("t", ["f16", "bf16"])
@pytest.mark.parametrize("change, want", [
    ({"M": -1}, INVALID), ({"K": -1}, INVALID), ({"C": None}, INVALID), ({"ldc": 299}, INVALID),
    ({"ldc": 300}, UNSUPPORTED), ({"C": P + 8}, UNSUPPORTED), ({"A": None}, INVALID),
    ({"lda": 192}, INVALID), ({"lda": 200}, UNSUPPORTED), ({"ldsa": 9}, INVALID), ({"ldsb": 1}, INVALID),
    ({"B": P + 4}, UNSUPPORTED), ({"SB": P + 1}, UNSUPPORTED), ({"M": 0}, OK), ({"N": 0}, OK),
    ({"M": 2 ** 31 - 200, "ldsa": 2 ** 31 - 1}, UNSUPPORTED), ({"ws": None, "bytes": 4}, INVALID),
    ({"bytes": -1}, INVALID), ({"ws": P + 8}, UNSUPPORTED), ({"block_a": 128}, INVALID),
    ({"block_b": 1}, INVALID), ({"block_b": 0}, INVALID),
])
def test_gemm_refusals(t, change, want):
    a = dict(M=10, N=300, K=200, A=P, lda=208, SA=P, ldsa=10, B=P, ldb=208, SB=P, ldsb=2, C=P, ldc=304,
             ws=P, bytes=1 << 20, block_a=1, block_b=128)
    a.update(change)
    m = fp8(a, ("A", "lda", "SA", "ldsa", "block_a")), fp8(a, ("B", "ldb", "SB", "ldsb", "block_b"))
    assert call(f"gemm_fp8_{t}", a["M"], a["N"], a["K"], *m, a["C"], a["ldc"], a["ws"], a["bytes"],
                None) == want


def _struct(kind, base, change):
    a = dict(base)
    a.update(change)
    return ctypes.byref(kind(**a))


NORM = dict(rows=4, K=100, x=P, ldx=100, residual=P, ldr=100, weight=P, eps=1e-6, total=P, ldt=100, y=P,
            ldy=100, q=P, ldq=112, s=P, lds=4, rstd=P)


@pytest.mark.parametrize("t", ["f16", "bf16"])
@pytest.mark.parametrize("change, want", [
    ({"rows": -1}, INVALID), ({"K": -1}, INVALID), ({"x": None}, INVALID), ({"ldx": 99}, INVALID),
    ({"ldr": 99}, INVALID), ({"ldt": 99}, INVALID), ({"ldy": 99}, INVALID), ({"ldq": 96}, INVALID),
    ({"s": None}, INVALID), ({"lds": 3}, INVALID), ({"eps": float("nan")}, INVALID),
    ({"eps": -1.0}, INVALID), ({"total": None, "y": None, "q": None, "rstd": None}, INVALID),
    ({"x": P + 1}, UNSUPPORTED), ({"weight": P + 1}, UNSUPPORTED), ({"rstd": P + 2}, UNSUPPORTED),
    ({"q": P + 8}, UNSUPPORTED), ({"ldq": 104}, UNSUPPORTED), ({"rows": 0}, OK), ({"K": 0}, OK),
    ({"K": 32769, **{k: 1 << 20 for k in ("ldx", "ldr", "ldt", "ldy", "ldq")}}, UNSUPPORTED),
    # 2^22 rows of 1024 threads: one more than a launch has
    ({"K": 16384, "rows": 1 << 22, "lds": 1 << 22,
      **{k: 16384 for k in ("ldx", "ldr", "ldt", "ldy", "ldq")}}, UNSUPPORTED),
])
def test_norm_refusals(t, change, want):
    assert call(f"rms_norm_{t}", _struct(sdt.SdtNorm, NORM, change), None) == want


def test_null_structs():
    assert call("fp8_quantize_f16", 1, 1, P, 1, None, None) == INVALID
    assert call("fp8_dequantize_f32", 1, 1, None, P, 1, None) == INVALID
    assert call("gemm_fp8_bf16", 1, 1, 1, None, None, P, 8, None, 0, None) == INVALID
    for name in ("rms_norm_f16", "rms_norm_backward_bf16", "gated_ff_f16", "gated_ff_backward_bf16"):
        assert call(name, None, None) == INVALID


NORM_GRAD = dict(rows=4, K=100, total=P, ldt=100, weight=P, rstd=P, dy=P, lddy=100, dtotal=P, lddt=100,
                 dx=P, lddx=100, dweight=P, workspace=P, workspace_bytes=1600)


@pytest.mark.parametrize("t", ["f16", "bf16"])
@pytest.mark.parametrize("change, want", [
    ({"rows": -1}, INVALID), ({"total": None}, INVALID), ({"rstd": None}, INVALID), ({"dy": None}, INVALID),
    ({"dx": None}, INVALID), ({"lddx": 99}, INVALID), ({"lddt": 99}, INVALID),
    ({"workspace": None}, INVALID), ({"workspace_bytes": 399}, INVALID), ({"workspace": P + 8}, UNSUPPORTED),
    ({"dweight": P + 2}, UNSUPPORTED), ({"dy": P + 1}, UNSUPPORTED), ({"K": 0}, OK),
    ({"rows": 0, "dweight": None}, OK),
])
def test_norm_backward_refusals(t, change, want):
    assert call(f"rms_norm_backward_{t}", _struct(sdt.SdtNormGrad, NORM_GRAD, change), None) == want


GATED = dict(M=10, N=300, K=200, x=P, ldx=200, gate=P, ldgate=200, up=P, ldup=208, act=0, h=P, ldh=304,
             g=P, ldg=300, u=P, ldu=300, wide=1, workspace=P, workspace_bytes=1 << 20)


@pytest.mark.parametrize("t", ["f16", "bf16"])
@pytest.mark.parametrize("change, want", [
    ({"M": -1}, INVALID), ({"act": 2}, INVALID), ({"act": -1}, INVALID), ({"x": None}, INVALID),
    ({"up": None}, INVALID), ({"h": None}, INVALID), ({"ldx": 199}, INVALID), ({"ldup": 204}, UNSUPPORTED),
    ({"ldh": 300}, UNSUPPORTED), ({"h": P + 2}, UNSUPPORTED), ({"gate": P + 8}, UNSUPPORTED),
    ({"g": None}, INVALID), ({"ldu": 299}, INVALID), ({"wide": 2}, INVALID), ({"ldg": 301}, UNSUPPORTED),
    ({"wide": 0}, UNSUPPORTED), ({"ldgate": 1 << 22}, UNSUPPORTED), ({"M": 0}, OK), ({"N": 0}, OK),
    ({"workspace": None}, INVALID), ({"workspace_bytes": -1}, INVALID), ({"workspace": P + 8}, UNSUPPORTED),
])
def test_gated_refusals(t, change, want):
    assert call(f"gated_ff_{t}", _struct(sdt.SdtGatedFf, GATED, change), None) == want


GATED_GRAD = dict(M=10, N=300, K=200, x=P, ldx=200, gate=P, ldgate=200, up=P, ldup=208, act=0, g=P, ldg=300,
                  u=P, ldu=300, wide=1, dh=P, lddh=300, dx=P, lddx=200, dgate=P, lddgate=200, dup=P,
                  lddup=200, workspace=P, workspace_bytes=1 << 30)


@pytest.mark.parametrize("t", ["f16", "bf16"])
@pytest.mark.parametrize("change, want", [
    ({"N": -1}, INVALID), ({"act": 2}, INVALID), ({"dgate": None}, INVALID),
    ({"dx": None, "dgate": None, "dup": None}, INVALID), ({"g": None}, INVALID), ({"dh": None}, INVALID),
    ({"lddh": 299}, INVALID), ({"lddx": 196}, INVALID), ({"lddup": 204}, UNSUPPORTED),
    ({"workspace": None}, INVALID), ({"workspace_bytes": 100}, INVALID), ({"workspace": P + 4}, UNSUPPORTED),
    ({"gate": P + 8}, UNSUPPORTED), ({"dh": P + 1}, UNSUPPORTED), ({"K": 0}, OK), ({"M": 0, "N": 0}, OK),
])
def test_gated_backward_refusals(t, change, want):
    assert call(f"gated_ff_backward_{t}", _struct(sdt.SdtGatedFfGrad, GATED_GRAD, change), None) == want


@pytest.mark.parametrize("t", ["f16", "bf16"])
@pytest.mark.parametrize("layout, change, want", [
    ("nn", {"M": -1}, INVALID), ("tn", {"K": -1}, INVALID), ("nn", {"lda": 40}, INVALID),
    ("tn", {"lda": 32}, INVALID), ("nn", {"ldb": 56}, INVALID), ("nn", {"lda": 52}, UNSUPPORTED),
    ("tn", {"ldb": 1 << 22}, UNSUPPORTED), ("nn", {"A": P + 8}, UNSUPPORTED), ("tn", {"C": None}, INVALID),
    ("tn", {"B": None}, INVALID), ("nn", {"ws": None, "bytes": 4}, INVALID), ("nn", {"bytes": -1}, INVALID),
    ("nn", {"ws": P + 4}, UNSUPPORTED), ("nn", {"M": 0}, OK), ("tn", {"N": 0}, OK),
])
def test_turned_refusals(t, layout, change, want):
    a = dict(M=40, N=60, K=50, A=P, lda=56, B=P, ldb=64, C=P, ldc=64, ws=P, bytes=1 << 20)
    a.update(change)
    assert call(f"gemm_{t}_{layout}", *a.values(), None) == want


def test_workspace_sizes():
    assert sdt.rms_norm_workspace_size(0, 4096) == 0
    assert sdt.rms_norm_workspace_size(1, 4096) == 4096 * 4
    assert sdt.rms_norm_workspace_size(10 ** 6, 4096) == sdt.rms_norm_workspace_size(10 ** 5, 4096)
    for bad in ((-1, 8), (8, -1), (8, 32769)):
        with pytest.raises(sdt.SdtError):
            sdt.rms_norm_workspace_size(*bad)
    # both factors' gradients, in 16 bits, are held at least
    assert sdt.gated_ff_workspace_size(100, 300, 200) >= 100 * 2 * 304 * 2
    assert sdt.gated_ff_workspace_size(0, 300, 200) >= 0
    with pytest.raises(sdt.SdtError):
        sdt.gated_ff_workspace_size(1, -1, 1)
    for size in (sdt.gemm_fp8_workspace_size, sdt.gated_ff_split_size):
        assert size(16, 64, 8192) == 0                                  # streamed
        assert size(100, 64, 8192) > 0
        assert size(100, 64, 256) == 0
        assert size(4096, 4096, 4096) == 0
        with pytest.raises(sdt.SdtError):
            size(-1, 1, 1)
    assert sdt.gemm_turned_workspace_size(8192, 8192, 8192) == 0        # tiles enough
    assert sdt.gemm_turned_workspace_size(64, 64, 8192) > 0             # one tile, long
    assert sdt.gemm_turned_workspace_size(64, 64, 100) == 0             # and short
    with pytest.raises(sdt.SdtError):
        sdt.gemm_turned_workspace_size(1, 1, -1)


def test_host_tensors_are_refused():
    """No address of the host's goes to the device."""
    import torch
    x, v = torch.zeros(4, 128, dtype=torch.float16), torch.zeros(128, dtype=torch.float16)
    with pytest.raises(TypeError):
        sdt.rms_norm(x, v, y=x)
    with pytest.raises(TypeError):
        sdt.gated_ff(x, x, x, torch.zeros(4, 4, dtype=torch.float16))
    with pytest.raises(TypeError):
        sdt.gemm_f16_nn(x, torch.zeros(128, 4, dtype=torch.float16), torch.zeros(4, 4, dtype=torch.float16))
    with pytest.raises(TypeError):
        sdt.Fp8(torch.zeros(4, 128, dtype=torch.float8_e4m3fn), torch.ones(1, 4))
    with pytest.raises(TypeError):
        sdt.Fp8(torch.zeros(4, 128), torch.ones(1, 4))
    with pytest.raises(ValueError):
        sdt.Fp8.empty(4, 128, block=64, device="cpu")
    with pytest.raises(TypeError):
        sdt.fp8_quantize_f16(x, sdt.Fp8.empty(4, 128, device="cpu"))
    with pytest.raises(TypeError):
        sdt.rms_norm(x.float(), v, y=x)
    with pytest.raises(TypeError):
        sdt.rms_norm_backward(x, v, torch.zeros(4), x, x)


def test_fp8_follows_its_tensors():
    """The tensors cannot be exchanged, and memory that they are given later is found."""
    import torch
    m = sdt.Fp8.empty(4, 128, device="cpu")
    for name in ("q", "s"):
        with pytest.raises(AttributeError):
            setattr(m, name, getattr(m, name).clone())
        first = m._packed()
        assert m._packed() == first
        kept = getattr(m, name).data                     # not freed: the next one lies elsewhere
        getattr(m, name).data = torch.empty_like(kept)
        assert m._packed() != first
        assert m._packed() == sdt._pack_fp8(*m._args(), 1)


@pytest.mark.parametrize("rows, K, block, stride", [(64, 512, 1, 0), (64, 512, 1, 1), (64, 512, 1, 63), (300, 512, 128, 0),
                                                    (300, 512, 128, 3), (300, 100, 128, 0)])
def test_fp8_scales_that_overlap(rows, K, block, stride):
    """Scales expanded over the blocks, or rows of them that overlap: their stride is passed
    on as it is and refused, not read as if every row had memory of its own."""
    import torch
    m = sdt.Fp8.empty(rows, K, block=block, device="cpu")
    shape = tuple(m.s.shape)
    assert shape[0] > 1
    few = torch.ones(shape[0] * shape[1])
    m.s.set_(few.as_strided(shape, (stride, 1)))
    assert m._args()[3] == stride
    X = torch.zeros(1, dtype=torch.float16)                 # never read
    assert call("fp8_quantize_f16", rows, K, X.data_ptr(), K, m._packed(), None) == INVALID
    assert call("fp8_dequantize_f16", rows, K, m._packed(), X.data_ptr(), K, None) == INVALID


def test_fp8_one_row_of_scales():
    """Its stride is of no matter."""
    import torch
    for rows, K, block in ((64, 100, 1), (100, 512, 128), (1, 1, 1)):
        m = sdt.Fp8.empty(rows, K, block=block, device="cpu")
        wide = tuple(m.s.shape)[1]
        m.s.set_(torch.ones(wide).as_strided((1, wide), (0, 1)))
        assert m._args()[3] == wide


def test_fp8_follows_its_tensors_strides():
    """Other strides at the same address are found; another shape is refused."""
    import torch
    m = sdt.Fp8.empty(64, 512, device="cpu")
    scales, codes = torch.ones(4 * 80), torch.zeros(64 * 640, dtype=torch.uint8).view(torch.float8_e4m3fn)
    m.s.set_(scales.as_strided((4, 64), (64, 1)))
    m.q.set_(codes.as_strided((64, 512), (512, 1)))
    assert m._packed() == sdt._pack_fp8(codes.data_ptr(), 512, scales.data_ptr(), 64, 1)
    m.s.set_(scales.as_strided((4, 64), (80, 1)))
    assert m._packed() == sdt._pack_fp8(codes.data_ptr(), 512, scales.data_ptr(), 80, 1)
    m.q.set_(codes.as_strided((64, 512), (640, 1)))
    assert m._packed() == sdt._pack_fp8(codes.data_ptr(), 640, scales.data_ptr(), 80, 1)
    assert m._args() == (codes.data_ptr(), 640, scales.data_ptr(), 80)
    for name, other in (("s", torch.ones(2, 64)), ("s", torch.ones(4, 128)[:, ::2]),
                        ("q", codes[:64 * 256].view(64, 256)), ("q", codes[:64 * 512].view(512, 64).t())):
        t = getattr(m, name)
        kept = t.data
        t.set_(other)
        with pytest.raises(ValueError):
            m._packed()
        with pytest.raises(ValueError):
            m._args()
        t.set_(kept)
        assert m._args() == (codes.data_ptr(), 640, scales.data_ptr(), 80)


def test_workspace_sizes_outside_the_limits():
    """No size for what the calls refuse: -1 from the library, an error from the binding."""
    top = 2 ** 31 - 256
    for size, refused in [
            # rows of dg and du past gemm operands' strides (2 N' < 2^22)
            (sdt.gated_ff_workspace_size, [(4, 1 << 22, 64), (4, 1 << 21, 64), (top, top, 8), (top, 1 << 21, 8)]),
            # rows of x past them; of both operands of one layout and of the other
            (sdt.gated_ff_split_size, [(20, 64, 1 << 22)]),
            (sdt.gemm_turned_workspace_size, [(4, 1 << 22, 64), (1 << 22, 64, 1 << 22)]),
            (sdt.gemm_fp8_workspace_size, [(100, 64, 1 << 23)])]:
        entry = getattr(sdt.lib(), "sdt_" + size.__name__)
        for sizes in refused:
            assert entry(*sizes) == -1, (size.__name__, sizes)
            with pytest.raises(sdt.SdtError):
                size(*sizes)
    with pytest.raises(sdt.SdtError):
        sdt.rms_norm_workspace_size(1 << 31, 64)
    # the largest that are taken
    assert sdt.gated_ff_workspace_size(4, (1 << 21) - 8, 64) >= 4 * 2 * ((1 << 21) - 8) * 2
    assert sdt.gemm_turned_workspace_size(1 << 22, 64, 64) == 0 and sdt.gemm_turned_workspace_size(64, 64, 1 << 22) > 0
    assert sdt.gated_ff_split_size(20, 64, (1 << 22) - 8) > 0
    assert sdt.gemm_fp8_workspace_size(100, 64, (1 << 23) - 16) > 0
    # nothing to compute, nothing refused
    assert sdt.gated_ff_workspace_size(0, 1 << 22, 64) >= 0 and sdt.gated_ff_workspace_size(4, 1 << 22, 0) >= 0


@pytest.mark.parametrize("t", ["f16", "bf16"])
def test_sizes_that_are_refused(t):
    """The calls themselves, at those sizes and strides that would hold them."""
    n = 1 << 21
    a = dict(GATED_GRAD, N=n, **{k: n for k in ("ldg", "ldu", "lddh")}, workspace_bytes=1 << 40)
    assert call(f"gated_ff_backward_{t}", _struct(sdt.SdtGatedFfGrad, a, {}), None) == UNSUPPORTED
    a = dict(GATED, K=1 << 22, **{k: 1 << 22 for k in ("ldx", "ldgate", "ldup")})
    assert call(f"gated_ff_{t}", _struct(sdt.SdtGatedFf, a, {}), None) == UNSUPPORTED
    for layout, (M, N, K) in (("nn", (4, 1 << 22, 64)), ("tn", (4, 1 << 22, 64)), ("nn", (1 << 22, 64, 1 << 22)),
                              ("tn", (1 << 22, 64, 1 << 22))):
        lda = K if layout == "nn" else M
        assert call(f"gemm_{t}_{layout}", M, N, K, P, lda, P, N, P, N, None, 0, None) == UNSUPPORTED
    K = 1 << 23
    A, B = (ctypes.byref(sdt.SdtFp8(P, K, P, 1 << 16, block)) for block in (1, 128))
    assert call(f"gemm_fp8_{t}", 100, 64, K, A, B, P, 64, None, 0, None) == UNSUPPORTED


def test_fp8_packed_by_two_threads():
    """What a matrix keeps of its memory is there before it counts as kept: another thread that
    finds the same memory in between would use the rest."""
    import torch

    class Watched(sdt.Fp8):
        __slots__ = ("order",)

        def __setattr__(self, name, value):
            object.__setattr__(self, name, value)
            if hasattr(self, "order") and name != "order":
                self.order.append(name)
    m = Watched.empty(4, 128, device="cpu")
    m.order = []
    m._packed()
    m.s.set_(torch.ones(1, 4))
    m._packed()
    m._args()
    assert len(m.order) == 6 and m.order[2] == m.order[5] == "_at"

"""Thin ctypes binding over ``libsdt.so`` (C ABI in ``include/sdt.h``).

Argument marshalling only: every step of the computation runs in the HIP
kernels of the library.  Tensors are torch tensors on a ROCm device, used for
device memory and streams; the library is handed raw pointers, strides in
elements, and the current stream.  A missing library raises immediately: there
is no fallback path.
"""
from __future__ import annotations

import ctypes
import os
import struct

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libsdt.so")

SDT_OK = 0
SDT_ERR_INVALID_ARG = 1
SDT_ERR_UNSUPPORTED = 2
SDT_ERR_HIP = 3

# Every function include/sdt.h declares.
EXPORTS = (
    "gemm_f16", "gemv_f16_m1", "gemm_f16_ex", "gemv_f16_m1_ex", "sdt_gemv_num_variants",
    "gemv_f16_m1_kn", "gemv_f16_m1_kn_ex", "sdt_gemv_kn_num_variants", "sdt_check_gemv_kn_args",
    "gemm_bf16", "gemm_bf16_ex", "gemv_bf16_m1", "gemv_bf16_m1_kn",
    "sdt_pick_tile", "sdt_pick_rung", "sdt_num_tiles", "sdt_tile_info",
    "sdt_stagger_eligible", "sdt_stagger_ktile", "sdt_check_gemm_args",
    "sdt_status_string", "sdt_last_hip_error", "sdt_empty_kernel", "sdt_stream_read",
    "sdt_plan_tile",
    "gemm_f16_cfg", "gemm_bf16_cfg",
    "gemm_f16_ws", "gemm_bf16_ws", "sdt_gemm_workspace_size", "sdt_launch_workspace_size",
    "sdt_workspace_init", "sdt_pick_tile_ws", "sdt_abi_version", "sdt_stream_read_grid",
    "gemm_f16_noalloc", "gemv_f16_m1_kn_ws", "gemv_bf16_m1_kn_ws", "sdt_gemv_kn_workspace_size",
    "sdt_stream_read_runs", "sdt_mfma_ceiling",
    "sdt_mx4_row_bytes", "sdt_mx4_scale_bytes", "mx4_pack_scales",
    "mx4_quantize_f16", "mx4_quantize_bf16", "mx4_quantize_rows_f16", "mx4_quantize_rows_bf16",
    "mx4_dequantize_f16", "mx4_dequantize_bf16", "mx4_dequantize_f32",
    "gemm_mx4_f16", "gemm_mx4_bf16", "gemv_mx4_m1_f16", "gemv_mx4_m1_bf16",
    "moe_route_f32", "moe_route_f16", "moe_route_bf16",
    "moe_route_backward_f32", "moe_route_backward_f16", "moe_route_backward_bf16",
    "sdt_moe_plan_rows", "moe_plan", "moe_gemm_mx4_f16", "moe_gemm_mx4_bf16",
    "moe_combine_f16", "moe_combine_bf16",
    "sdt_moe_experts_workspace_size", "moe_experts_mx4_f16", "moe_experts_mx4_bf16",
    "fp8_quantize_f16", "fp8_quantize_bf16",
    "fp8_dequantize_f16", "fp8_dequantize_bf16", "fp8_dequantize_f32",
    "gemm_fp8_f16", "gemm_fp8_bf16", "sdt_gemm_fp8_workspace_size",
    "rms_norm_f16", "rms_norm_bf16", "rms_norm_backward_f16", "rms_norm_backward_bf16",
    "sdt_rms_norm_workspace_size",
    "gated_ff_f16", "gated_ff_bf16", "sdt_gated_ff_split_size",
    "gated_ff_backward_f16", "gated_ff_backward_bf16",
    "sdt_gated_ff_workspace_size",
    "gemm_f16_nn", "gemm_bf16_nn", "gemm_f16_tn", "gemm_bf16_tn",
    "sdt_gemm_turned_workspace_size",
)

# The include/sdt.h version these structures and signatures follow.
ABI_VERSION = 7


class SdtTile(ctypes.Structure):
    _fields_ = [("id", ctypes.c_int), ("bm", ctypes.c_int), ("bn", ctypes.c_int),
                ("bk", ctypes.c_int), ("waves_m", ctypes.c_int), ("waves_n", ctypes.c_int),
                ("threads", ctypes.c_int), ("stages", ctypes.c_int),
                ("lds_bytes", ctypes.c_int), ("kgroups", ctypes.c_int),
                ("stagger", ctypes.c_int), ("long_stages", ctypes.c_int),
                ("splits", ctypes.c_int), ("split_algo", ctypes.c_int),
                ("persistent", ctypes.c_int), ("ksplit", ctypes.c_int),
                ("loaders", ctypes.c_int)]

    def as_dict(self) -> dict:
        return {name: getattr(self, name) for name, _ in self._fields_}


class SdtLaunch(ctypes.Structure):
    """sdt_launch: -1 in a field = the automatic choice."""
    _fields_ = [("tile_id", ctypes.c_int), ("stages", ctypes.c_int),
                ("kgroups", ctypes.c_int), ("stagger", ctypes.c_int),
                ("splits", ctypes.c_int), ("split_algo", ctypes.c_int),
                ("persistent", ctypes.c_int), ("loaders", ctypes.c_int)]


class SdtRoute(ctypes.Structure):
    """sdt_route: how tokens choose experts (route_cfg makes one)."""
    _fields_ = [("topk", ctypes.c_int), ("score", ctypes.c_int), ("groups", ctypes.c_int),
                ("groups_kept", ctypes.c_int), ("group_top", ctypes.c_int),
                ("renormalize", ctypes.c_int), ("scale", ctypes.c_float)]


class SdtMoePlan(ctypes.Structure):
    _fields_ = [("tokens", ctypes.c_int64), ("topk", ctypes.c_int), ("experts", ctypes.c_int),
                ("counts", ctypes.c_void_p), ("offsets", ctypes.c_void_p),
                ("rows", ctypes.c_void_p), ("pos", ctypes.c_void_p), ("tiles", ctypes.c_void_p)]


class SdtMx4Experts(ctypes.Structure):
    """sdt_mx4_experts.  Made from an Mx4 it knows how many matrices its addresses
    hold and where they lie; a struct of plain addresses does not."""
    experts = device = None
    _fields_ = [("q", ctypes.c_void_p), ("ldq", ctypes.c_int64), ("q_expert", ctypes.c_int64),
                ("s", ctypes.c_void_p), ("s_expert", ctypes.c_int64)]


class SdtMoeLayer(ctypes.Structure):
    """sdt_moe_layer, with what its matrices know of themselves: moe_experts_mx4
    refuses a plan of other experts, and operands of another device."""
    experts = device = None
    _fields_ = [("N", ctypes.c_int64), ("K", ctypes.c_int64), ("gate", SdtMx4Experts),
                ("up", SdtMx4Experts), ("down", SdtMx4Experts)]

    def __init__(self, *args, **kw):
        super().__init__(*args, **kw)
        matrices = [m for m in (*args[2:], *kw.values()) if isinstance(m, SdtMx4Experts)]
        for what in ("experts", "device"):
            known = {getattr(m, what) for m in matrices} - {None}
            if len(known) > 1:
                raise TypeError(f"the layer's matrices do not agree: {what} {sorted(known)}")
            if known:
                setattr(self, what, known.pop())


def _fields(text):
    """ctypes fields from "name type" words: p a pointer, i an int64, n an int, f a float."""
    kinds = {"p": ctypes.c_void_p, "i": ctypes.c_int64, "n": ctypes.c_int, "f": ctypes.c_float}
    words = text.split()
    return [(name, kinds[kind]) for name, kind in zip(words[::2], words[1::2])]


def _packer(cls):
    """A function that packs values into the bytes of such a struct: a sixth of the time of making the
    struct, and a call takes the bytes as its address."""
    letters = {ctypes.c_void_p: "P", ctypes.c_int64: "q", ctypes.c_int: "i", ctypes.c_float: "f"}
    form = "@" + "".join(letters[kind] for _, kind in cls._fields_) + "0q"
    packer = struct.Struct(form)
    if packer.size != ctypes.sizeof(cls):
        raise RuntimeError(f"{cls.__name__}: {packer.size} bytes, not {ctypes.sizeof(cls)}")
    return packer.pack


class SdtFp8(ctypes.Structure):
    _fields_ = _fields("q p ldq i s p lds i block n")


class SdtNorm(ctypes.Structure):
    _fields_ = _fields("rows i K i x p ldx i residual p ldr i weight p eps f total p ldt i y p ldy i "
                       "q p ldq i s p lds i rstd p")


class SdtNormGrad(ctypes.Structure):
    _fields_ = _fields("rows i K i total p ldt i weight p rstd p dy p lddy i dtotal p lddt i "
                       "dx p lddx i dweight p workspace p workspace_bytes i")


class SdtGatedFf(ctypes.Structure):
    _fields_ = _fields("M i N i K i x p ldx i gate p ldgate i up p ldup i act n h p ldh i "
                       "g p ldg i u p ldu i wide n workspace p workspace_bytes i")


class SdtGatedFfGrad(ctypes.Structure):
    _fields_ = _fields("M i N i K i x p ldx i gate p ldgate i up p ldup i act n g p ldg i u p ldu i "
                       "wide n dh p lddh i dx p lddx i dgate p lddgate i dup p lddup i "
                       "workspace p workspace_bytes i")


_pack_fp8, _pack_norm, _pack_norm_grad, _pack_gated, _pack_gated_grad = (
    _packer(cls) for cls in (SdtFp8, SdtNorm, SdtNormGrad, SdtGatedFf, SdtGatedFfGrad))


class SdtError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        msg = status_string(status)
        if status == SDT_ERR_HIP:
            msg += f" (hipError {last_hip_error()})"
        super().__init__(f"{where}: {msg}")


_lib = None
_i64 = ctypes.c_int64
_vp = ctypes.c_void_p
_int = ctypes.c_int


def lib():
    """Load libsdt.so once; raise if it is not built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is not built: run `python -m shape_driven_tile_amd.build`")
    # torch first: it loads its own HIP and HSA runtimes, whose sonames then
    # satisfy libsdt.so's dependencies, so the process holds one runtime.
    # Loaded the other way round, libsdt.so pulls in the system runtime and
    # torch adds its copy; the second to touch the GPU finds no device.
    import torch  # noqa: F401
    L = ctypes.CDLL(LIB_PATH)
    L.gemm_f16.argtypes = [_i64, _i64, _i64, _vp, _i64, _vp, _i64, _vp, _i64, _vp]
    L.gemm_f16_ex.argtypes = L.gemm_f16.argtypes + [_int, _int]
    L.gemv_f16_m1.argtypes = [_i64, _i64, _vp, _vp, _i64, _vp, _vp]
    L.gemv_f16_m1_ex.argtypes = L.gemv_f16_m1.argtypes + [_int]
    L.sdt_gemv_num_variants.argtypes = []
    L.gemv_f16_m1_kn.argtypes = [_i64, _i64, _vp, _vp, _i64, _vp, _vp]
    L.gemm_bf16.argtypes = L.gemm_f16.argtypes
    L.gemm_bf16_ex.argtypes = L.gemm_f16_ex.argtypes
    L.gemv_bf16_m1.argtypes = L.gemv_f16_m1.argtypes
    L.gemv_bf16_m1_kn.argtypes = L.gemv_f16_m1_kn.argtypes
    L.gemv_f16_m1_kn_ex.argtypes = L.gemv_f16_m1_kn.argtypes + [_int]
    L.sdt_gemv_kn_num_variants.argtypes = []
    L.sdt_check_gemv_kn_args.argtypes = [_i64, _i64, _vp, _vp, _i64, _vp]
    L.sdt_pick_tile.argtypes = [_i64, _i64, _i64, _int, ctypes.POINTER(SdtTile)]
    L.sdt_pick_rung.argtypes = [_i64, _i64, _int, _int, _int, ctypes.POINTER(_i64)]
    L.sdt_num_tiles.argtypes = []
    L.sdt_tile_info.argtypes = [_int, ctypes.POINTER(SdtTile)]
    L.sdt_plan_tile.argtypes = [_int, _i64, _i64, _i64, _int, ctypes.POINTER(SdtTile)]
    L.gemm_f16_ws.argtypes = [_i64, _i64, _i64, _vp, _i64, _vp, _i64, _vp, _i64, _vp, _i64, _vp]
    L.gemm_bf16_ws.argtypes = L.gemm_f16_ws.argtypes
    L.gemm_f16_cfg.argtypes = L.gemm_f16_ws.argtypes + [ctypes.POINTER(SdtLaunch)]
    L.gemm_bf16_cfg.argtypes = L.gemm_f16_cfg.argtypes
    L.sdt_gemm_workspace_size.argtypes = [_i64, _i64, _i64, _int]
    L.sdt_gemm_workspace_size.restype = _i64
    L.sdt_launch_workspace_size.argtypes = [_i64, _i64, _i64, ctypes.POINTER(SdtLaunch)]
    L.sdt_launch_workspace_size.restype = _i64
    L.sdt_workspace_init.argtypes = [_vp, _i64, _vp]
    L.sdt_pick_tile_ws.argtypes = [_i64, _i64, _i64, _int, _i64, ctypes.POINTER(SdtTile)]
    L.sdt_abi_version.argtypes = []
    L.gemm_f16_noalloc.argtypes = L.gemm_f16.argtypes
    L.sdt_stream_read_grid.argtypes = [_vp, _i64, _vp, _int, _vp]
    L.gemv_f16_m1_kn_ws.argtypes = [_i64, _i64, _vp, _vp, _i64, _vp, _vp, _i64, _vp]
    L.gemv_bf16_m1_kn_ws.argtypes = L.gemv_f16_m1_kn_ws.argtypes
    L.sdt_gemv_kn_workspace_size.argtypes = [_i64, _i64]
    L.sdt_gemv_kn_workspace_size.restype = _i64
    L.sdt_stream_read_runs.argtypes = [_vp, _i64, _i64, _int, _int, _vp, _vp]
    L.sdt_mfma_ceiling.argtypes = [_vp, _int, _vp, _int, _int, _vp]
    L.sdt_stagger_eligible.argtypes = [_i64]
    L.sdt_stagger_ktile.argtypes = [_i64, _i64, _i64]
    L.sdt_stagger_ktile.restype = _i64
    L.sdt_check_gemm_args.argtypes = [_i64, _i64, _i64, _vp, _i64, _vp, _i64, _vp, _i64]
    L.sdt_status_string.argtypes = [_int]
    L.sdt_status_string.restype = ctypes.c_char_p
    L.sdt_last_hip_error.argtypes = []
    L.sdt_empty_kernel.argtypes = [_vp]
    L.sdt_stream_read.argtypes = [_vp, _i64, _vp, _vp]
    for name in ("gemm_f16", "gemm_f16_ex", "gemv_f16_m1", "gemv_f16_m1_ex",
                 "gemv_f16_m1_kn", "gemv_f16_m1_kn_ex", "sdt_gemv_kn_num_variants",
                 "gemm_bf16", "gemm_bf16_ex", "gemv_bf16_m1", "gemv_bf16_m1_kn",
                 "sdt_check_gemv_kn_args",
                 "sdt_gemv_num_variants", "sdt_pick_tile", "sdt_pick_rung", "sdt_num_tiles",
                 "sdt_tile_info", "sdt_stagger_eligible", "sdt_plan_tile", "sdt_check_gemm_args",
                 "gemm_f16_cfg", "gemm_bf16_cfg", "gemm_f16_ws", "gemm_bf16_ws",
                 "sdt_workspace_init", "sdt_pick_tile_ws", "sdt_abi_version",
                 "sdt_stream_read_grid", "gemm_f16_noalloc", "sdt_last_hip_error", "sdt_empty_kernel", "sdt_stream_read",
                 "gemv_f16_m1_kn_ws", "gemv_bf16_m1_kn_ws", "sdt_stream_read_runs",
                 "sdt_mfma_ceiling"):
        getattr(L, name).restype = _int
    _declare_mx4(L)
    _declare_ffn(L)
    if L.sdt_abi_version() != ABI_VERSION:
        raise RuntimeError(f"{LIB_PATH} has ABI version {L.sdt_abi_version()}, this binding "
                           f"expects {ABI_VERSION}: rebuild the library")
    _lib = L
    return L


def _declare_mx4(L):
    plan, experts = ctypes.POINTER(SdtMoePlan), ctypes.POINTER(SdtMx4Experts)
    route, layer = ctypes.POINTER(SdtRoute), ctypes.POINTER(SdtMoeLayer)
    L.sdt_mx4_row_bytes.argtypes = [_i64]
    L.sdt_mx4_scale_bytes.argtypes = [_i64, _i64]
    L.mx4_pack_scales.argtypes = [_i64, _i64, _vp, _i64, _vp, _vp]
    L.sdt_moe_plan_rows.argtypes = [_i64, _int, _int]
    L.moe_plan.argtypes = [_vp, plan, _vp]
    L.sdt_moe_experts_workspace_size.argtypes = [_i64, _int, _int, _i64, _i64]
    for t in ("f16", "bf16"):
        getattr(L, f"mx4_quantize_{t}").argtypes = [_i64, _i64, _vp, _i64, _vp, _i64, _vp, _vp]
        getattr(L, f"mx4_quantize_rows_{t}").argtypes = [_i64, _i64, _vp, _i64, _i64, _vp, _int,
                                                         _vp, _i64, _vp, _vp]
        getattr(L, f"gemm_mx4_{t}").argtypes = [_i64, _i64, _i64, _vp, _i64, _vp, _vp, _i64, _vp,
                                                _vp, _i64, _vp]
        getattr(L, f"gemv_mx4_m1_{t}").argtypes = [_i64, _i64, _vp, _vp, _i64, _vp, _vp, _vp]
        getattr(L, f"moe_gemm_mx4_{t}").argtypes = [plan, _i64, _i64, _vp, _i64, _vp, experts,
                                                    experts, _vp, _i64, _vp]
        getattr(L, f"moe_combine_{t}").argtypes = [plan, _i64, _vp, _i64, _vp, _vp, _i64, _vp]
        getattr(L, f"moe_experts_mx4_{t}").argtypes = [layer, _vp, _vp, plan, _vp, _i64, _vp, _i64,
                                                       _vp, _i64, _vp]
    for t in ("f32", "f16", "bf16"):
        getattr(L, f"mx4_dequantize_{t}").argtypes = [_i64, _i64, _vp, _i64, _vp, _vp, _i64, _vp]
        getattr(L, f"moe_route_{t}").argtypes = [_i64, _i64, _vp, _i64, _vp, route, _vp, _vp, _vp]
        getattr(L, f"moe_route_backward_{t}").argtypes = [_i64, _i64, _vp, _i64, route, _vp, _vp,
                                                          _vp, _i64, _vp]
    for name in EXPORTS[EXPORTS.index("sdt_mx4_row_bytes"):EXPORTS.index("fp8_quantize_f16")]:
        getattr(L, name).restype = _int
    for name in ("sdt_mx4_row_bytes", "sdt_mx4_scale_bytes", "sdt_moe_plan_rows",
                 "sdt_moe_experts_workspace_size"):
        getattr(L, name).restype = _i64


def _declare_ffn(L):
    # structs as plain addresses: they are given as packed bytes
    for t in ("f16", "bf16"):
        getattr(L, f"fp8_quantize_{t}").argtypes = [_i64, _i64, _vp, _i64, _vp, _vp]
        getattr(L, f"gemm_fp8_{t}").argtypes = [_i64, _i64, _i64, _vp, _vp, _vp, _i64, _vp, _i64, _vp]
        for layout in ("nn", "tn"):
            getattr(L, f"gemm_{t}_{layout}").argtypes = [_i64, _i64, _i64, _vp, _i64, _vp, _i64, _vp,
                                                         _i64, _vp, _i64, _vp]
        for entry in ("rms_norm", "rms_norm_backward", "gated_ff", "gated_ff_backward"):
            getattr(L, f"{entry}_{t}").argtypes = [_vp, _vp]
    for t in ("f32", "f16", "bf16"):
        getattr(L, f"fp8_dequantize_{t}").argtypes = [_i64, _i64, _vp, _vp, _i64, _vp]
    L.sdt_rms_norm_workspace_size.argtypes = [_i64, _i64]
    for name in ("sdt_gated_ff_workspace_size", "sdt_gated_ff_split_size",
                 "sdt_gemm_fp8_workspace_size"):
        getattr(L, name).argtypes = [_i64, _i64, _i64]
    L.sdt_gemm_turned_workspace_size.argtypes = [_i64, _i64, _i64]
    for name in EXPORTS[EXPORTS.index("fp8_quantize_f16"):]:
        getattr(L, name).restype = _i64 if name.startswith("sdt_") else _int


# ---- host-only helpers ------------------------------------------------------

def status_string(status: int) -> str:
    return lib().sdt_status_string(int(status)).decode()


def last_hip_error() -> int:
    return int(lib().sdt_last_hip_error())


def num_tiles() -> int:
    return int(lib().sdt_num_tiles())


def tile_info(tile_id: int) -> dict:
    t = SdtTile()
    rc = lib().sdt_tile_info(int(tile_id), ctypes.byref(t))
    if rc != SDT_OK:
        raise SdtError(rc, "sdt_tile_info")
    return t.as_dict()


def plan_tile(tile_id: int, M: int, N: int, K: int, num_cu: int = 256) -> dict:
    """How a launch of rung tile_id on M x N x K is configured (stages, kgroups)."""
    t = SdtTile()
    rc = lib().sdt_plan_tile(int(tile_id), int(M), int(N), int(K), int(num_cu), ctypes.byref(t))
    if rc != SDT_OK:
        raise SdtError(rc, "sdt_plan_tile")
    return t.as_dict()


def launch_cfg(tile_id=-1, stages=-1, kgroups=-1, stagger=-1, splits=-1, split_algo=-1,
               persistent=-1, loaders=-1) -> SdtLaunch:
    return SdtLaunch(int(tile_id), int(stages), int(kgroups), int(stagger), int(splits),
                     int(split_algo), int(persistent), int(loaders))


def pick_tile_ws(M: int, N: int, K: int, num_cu: int, workspace_bytes: int) -> dict:
    """The plan gemm_f16_ws makes with a workspace of that many bytes."""
    t = SdtTile()
    rc = lib().sdt_pick_tile_ws(int(M), int(N), int(K), int(num_cu), int(workspace_bytes),
                                ctypes.byref(t))
    if rc != SDT_OK:
        raise SdtError(rc, "sdt_pick_tile_ws")
    return t.as_dict()


def gemm_workspace_size(M: int, N: int, K: int, num_cu: int = 0) -> int:
    """Workspace bytes gemm_f16_ws's automatic plan uses (0: no split)."""
    v = int(lib().sdt_gemm_workspace_size(int(M), int(N), int(K), int(num_cu)))
    if v < 0:
        raise SdtError(SDT_ERR_INVALID_ARG, "sdt_gemm_workspace_size")
    return v


def launch_workspace_size(M: int, N: int, K: int, **cfg) -> int:
    """Workspace bytes a forced launch configuration needs (0: no split)."""
    c = launch_cfg(**cfg)
    v = int(lib().sdt_launch_workspace_size(int(M), int(N), int(K), ctypes.byref(c)))
    if v < 0:
        raise SdtError(SDT_ERR_INVALID_ARG, "sdt_launch_workspace_size")
    return v


class Workspace:
    """A device workspace for the k-split entry points: `nbytes` bytes of a
    torch uint8 tensor (16-byte aligned by torch's allocator), its counters
    zeroed once by sdt_workspace_init on the current stream."""

    def __init__(self, nbytes: int, device="cuda", stream=None):
        import torch
        self.nbytes = (int(nbytes) + 15) // 16 * 16
        self.tensor = torch.empty(max(self.nbytes, 16), dtype=torch.uint8, device=device)
        if self.nbytes:
            rc = lib().sdt_workspace_init(self.tensor.data_ptr(), self.nbytes,
                                          _stream_handle(stream))
            if rc != SDT_OK:
                raise SdtError(rc, "sdt_workspace_init")

    def ptr(self):
        return self.tensor.data_ptr() if self.nbytes else None


def _ws_args(workspace):
    if workspace is None:
        return None, 0
    return workspace.ptr(), workspace.nbytes


def pick_tile(M: int, N: int, K: int, num_cu: int) -> dict:
    t = SdtTile()
    rc = lib().sdt_pick_tile(int(M), int(N), int(K), int(num_cu), ctypes.byref(t))
    if rc != SDT_OK:
        raise SdtError(rc, "sdt_pick_tile")
    return t.as_dict()


def pick_rung(M: int, N: int, ref_bm: int, ref_bn: int, min_blocks) -> int:
    arr = (_i64 * len(min_blocks))(*[int(v) for v in min_blocks])
    return int(lib().sdt_pick_rung(int(M), int(N), int(ref_bm), int(ref_bn), len(min_blocks), arr))


def stagger_eligible(K: int) -> bool:
    return bool(lib().sdt_stagger_eligible(int(K)))


def stagger_ktile(wg: int, i: int, nkt: int) -> int:
    return int(lib().sdt_stagger_ktile(int(wg), int(i), int(nkt)))


def check_gemm_args(M, N, K, A_ptr, lda, B_ptr, ldb, C_ptr, ldc) -> int:
    return int(lib().sdt_check_gemm_args(int(M), int(N), int(K), A_ptr, int(lda), B_ptr,
                                         int(ldb), C_ptr, int(ldc)))


def gemv_num_variants() -> int:
    return int(lib().sdt_gemv_num_variants())


def gemv_kn_num_variants() -> int:
    return int(lib().sdt_gemv_kn_num_variants())


def check_gemv_kn_args(N, K, x_ptr, B_ptr, ldb, y_ptr) -> int:
    return int(lib().sdt_check_gemv_kn_args(int(N), int(K), x_ptr, B_ptr, int(ldb), y_ptr))


# ---- compute entry points (torch tensors on a ROCm device) -------------------

def _stream_handle(stream):
    """The HIP stream of `stream`, or the current one of the current device (asked
    for its handle where torch has the calls: a torch.cuda.Stream object would cost
    2.8 us a call)."""
    if stream is not None:
        return stream.cuda_stream
    import torch
    try:
        return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
    except AttributeError:
        return torch.cuda.current_stream().cuda_stream


def _rows(t, name, dtype=None):
    if dtype is None:
        import torch
        dtype = torch.float16
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise TypeError(f"{name} must be a device tensor")
    shape, stride = t.shape, t.stride()
    if len(shape) != 2 or (shape[1] > 1 and stride[1] != 1):
        raise ValueError(f"{name} must be 2-D with unit stride along its rows")
    return t.data_ptr(), (stride[0] if shape[0] > 1 else max(stride[0], shape[1]))


def gemm_f16(A, B, C, stream=None) -> None:
    """C[M, N] = A[M, K] . B[N, K]^T (B stored K-major), fp32 accumulate, fp16 out."""
    M, K = A.shape
    N = B.shape[0]
    if B.shape[1] != K or tuple(C.shape) != (M, N):
        raise ValueError(f"shape mismatch A{tuple(A.shape)} B{tuple(B.shape)} C{tuple(C.shape)}")
    pa, lda = _rows(A, "A")
    pb, ldb = _rows(B, "B")
    pc, ldc = _rows(C, "C")
    rc = lib().gemm_f16(M, N, K, pa, lda, pb, ldb, pc, ldc, _stream_handle(stream))
    if rc != SDT_OK:
        raise SdtError(rc, "gemm_f16")


def gemm_f16_ex(A, B, C, tile_id: int = -1, stagger: int = -1, stream=None) -> None:
    M, K = A.shape
    N = B.shape[0]
    if B.shape[1] != K or tuple(C.shape) != (M, N):
        raise ValueError(f"shape mismatch A{tuple(A.shape)} B{tuple(B.shape)} C{tuple(C.shape)}")
    pa, lda = _rows(A, "A")
    pb, ldb = _rows(B, "B")
    pc, ldc = _rows(C, "C")
    rc = lib().gemm_f16_ex(M, N, K, pa, lda, pb, ldb, pc, ldc, _stream_handle(stream),
                           int(tile_id), int(stagger))
    if rc != SDT_OK:
        raise SdtError(rc, "gemm_f16_ex")


def gemv_f16_m1(x, B, y, stream=None, variant: int | None = None) -> None:
    """y[N] = x[K] . B[N, K]^T for the M=1 decode shape (B stored K-major)."""
    import torch
    if x.dtype != torch.float16 or y.dtype != torch.float16:
        raise TypeError("x and y must be float16")
    if x.dim() != 1 or y.dim() != 1 or x.stride(0) != 1 or y.stride(0) != 1:
        raise ValueError("x and y must be contiguous vectors")
    N, K = B.shape
    if x.shape[0] != K or y.shape[0] != N:
        raise ValueError(f"shape mismatch x{tuple(x.shape)} B{tuple(B.shape)} y{tuple(y.shape)}")
    pb, ldb = _rows(B, "B")
    h = _stream_handle(stream)
    if variant is None:
        rc = lib().gemv_f16_m1(N, K, x.data_ptr(), pb, ldb, y.data_ptr(), h)
    else:
        rc = lib().gemv_f16_m1_ex(N, K, x.data_ptr(), pb, ldb, y.data_ptr(), h, int(variant))
    if rc != SDT_OK:
        raise SdtError(rc, "gemv_f16_m1")


def stream_read(buf, out, stream=None) -> None:
    """Enqueue the library's read-only streaming kernel over the bytes of the
    contiguous device tensor `buf` (a multiple of 8192 bytes); `out` is a
    contiguous device tensor of at least numel(buf) * itemsize / 8192 int32
    words."""
    nbytes = buf.numel() * buf.element_size()
    if not buf.is_contiguous() or not out.is_contiguous() or \
            out.numel() * out.element_size() < (nbytes // 8192) * 4:
        raise ValueError("stream_read: contiguous buf, and out of one int32 word per 8 KB")
    rc = lib().sdt_stream_read(buf.data_ptr(), nbytes, out.data_ptr(), _stream_handle(stream))
    if rc != SDT_OK:
        raise SdtError(rc, "sdt_stream_read")


def stream_read_grid(buf, out, workgroups: int, stream=None) -> None:
    """Enqueue the library's grid-stride read-only kernel over the bytes of the
    contiguous device tensor `buf`; `out` holds at least `workgroups` int32
    words."""
    nbytes = buf.numel() * buf.element_size()
    if not buf.is_contiguous() or not out.is_contiguous() or \
            out.numel() * out.element_size() < 4 * int(workgroups):
        raise ValueError("stream_read_grid: contiguous buf, and out of one int32 word per workgroup")
    rc = lib().sdt_stream_read_grid(buf.data_ptr(), nbytes, out.data_ptr(), int(workgroups),
                                    _stream_handle(stream))
    if rc != SDT_OK:
        raise SdtError(rc, "sdt_stream_read_grid")


MFMA_CEILING_FRAGS = 24          # operand fragments per lane (one k-tile of a 128 x 64 wave tile)
MFMA_CEILING_FLOP_PER_ITER = 8 * 64 * 2 * 16 * 16 * 32   # per workgroup: 8 waves x 64 MFMAs


def mfma_ceiling(frags, iters: int, out, workgroups: int, bf16: bool = False,
                 mfma32: bool = False, stream=None) -> None:
    """Enqueue the library's register-only MFMA loop (16x16x32 MFMAs, or
    32x32x16 with mfma32): `frags` is a contiguous 16-bit device tensor of
    24 x 64 x 8 values (fragment f of lane l at [(f * 64 + l) * 8, +8)),
    `out` a float32 tensor of at least workgroups x 512 values."""
    if frags.element_size() != 2 or frags.numel() < MFMA_CEILING_FRAGS * 64 * 8 or \
            not frags.is_contiguous() or out.element_size() != 4 or \
            out.numel() < 512 * int(workgroups) or not out.is_contiguous():
        raise ValueError("mfma_ceiling: 24 x 64 x 8 16-bit fragments, workgroups x 512 floats out")
    flags = (1 if bf16 else 0) | (2 if mfma32 else 0)
    rc = lib().sdt_mfma_ceiling(frags.data_ptr(), int(iters), out.data_ptr(), int(workgroups),
                                flags, _stream_handle(stream))
    if rc != SDT_OK:
        raise SdtError(rc, "sdt_mfma_ceiling")


def empty_kernel(stream=None) -> None:
    """Enqueue the library's empty kernel (launch-floor measurement)."""
    rc = lib().sdt_empty_kernel(_stream_handle(stream))
    if rc != SDT_OK:
        raise SdtError(rc, "sdt_empty_kernel")


def gemv_f16_m1_kn(x, B, y, stream=None, variant: int | None = None) -> None:
    """y[N] = x[K] . B[K, N] for the M=1 decode shape with the weights stored
    as K rows of N (the N of a row contiguous)."""
    import torch
    if x.dtype != torch.float16 or y.dtype != torch.float16:
        raise TypeError("x and y must be float16")
    if x.dim() != 1 or y.dim() != 1 or x.stride(0) != 1 or y.stride(0) != 1:
        raise ValueError("x and y must be contiguous vectors")
    K, N = B.shape
    if x.shape[0] != K or y.shape[0] != N:
        raise ValueError(f"shape mismatch x{tuple(x.shape)} B{tuple(B.shape)} y{tuple(y.shape)}")
    pb, ldb = _rows(B, "B")
    h = _stream_handle(stream)
    if variant is None:
        rc = lib().gemv_f16_m1_kn(N, K, x.data_ptr(), pb, ldb, y.data_ptr(), h)
    else:
        rc = lib().gemv_f16_m1_kn_ex(N, K, x.data_ptr(), pb, ldb, y.data_ptr(), h, int(variant))
    if rc != SDT_OK:
        raise SdtError(rc, "gemv_f16_m1_kn")


def _gemm_16(entry, A, B, C, stream, dtype, extra=()):
    M, K = A.shape
    N = B.shape[0]
    if B.shape[1] != K or tuple(C.shape) != (M, N):
        raise ValueError(f"shape mismatch A{tuple(A.shape)} B{tuple(B.shape)} C{tuple(C.shape)}")
    pa, lda = _rows(A, "A", dtype)
    pb, ldb = _rows(B, "B", dtype)
    pc, ldc = _rows(C, "C", dtype)
    rc = getattr(lib(), entry)(M, N, K, pa, lda, pb, ldb, pc, ldc, _stream_handle(stream),
                               *extra)
    if rc != SDT_OK:
        raise SdtError(rc, entry)


def _gemm_16_ws(entry, A, B, C, workspace, stream, dtype, extra=()):
    M, K = A.shape
    N = B.shape[0]
    if B.shape[1] != K or tuple(C.shape) != (M, N):
        raise ValueError(f"shape mismatch A{tuple(A.shape)} B{tuple(B.shape)} C{tuple(C.shape)}")
    pa, lda = _rows(A, "A", dtype)
    pb, ldb = _rows(B, "B", dtype)
    pc, ldc = _rows(C, "C", dtype)
    wp, wn = _ws_args(workspace)
    rc = getattr(lib(), entry)(M, N, K, pa, lda, pb, ldb, pc, ldc, wp, wn,
                               _stream_handle(stream), *extra)
    if rc != SDT_OK:
        raise SdtError(rc, entry)


def gemm_f16_noalloc(A, B, C, stream=None) -> None:
    """gemm_f16_ws with the library's own per-device scratch as the workspace
    (no allocation; calls overlapping on one GPU race)."""
    import torch
    _gemm_16("gemm_f16_noalloc", A, B, C, stream, torch.float16)


def gemm_f16_ws(A, B, C, workspace=None, stream=None) -> None:
    """gemm_f16 with a Workspace: the plan may split K across workgroups."""
    import torch
    _gemm_16_ws("gemm_f16_ws", A, B, C, workspace, stream, torch.float16)


def gemm_bf16_ws(A, B, C, workspace=None, stream=None) -> None:
    import torch
    _gemm_16_ws("gemm_bf16_ws", A, B, C, workspace, stream, torch.bfloat16)


def gemm_f16_cfg(A, B, C, tile_id=-1, stages=-1, kgroups=-1, stagger=-1, splits=-1,
                 split_algo=-1, persistent=-1, workspace=None, stream=None, loaders=-1) -> None:
    """gemm_f16_ws with any part of the launch configuration forced (-1 = automatic)."""
    import torch
    cfg = launch_cfg(tile_id, stages, kgroups, stagger, splits, split_algo, persistent, loaders)
    _gemm_16_ws("gemm_f16_cfg", A, B, C, workspace, stream, torch.float16, (ctypes.byref(cfg),))


def gemm_bf16_cfg(A, B, C, tile_id=-1, stages=-1, kgroups=-1, stagger=-1, splits=-1,
                  split_algo=-1, persistent=-1, workspace=None, stream=None, loaders=-1) -> None:
    import torch
    cfg = launch_cfg(tile_id, stages, kgroups, stagger, splits, split_algo, persistent, loaders)
    _gemm_16_ws("gemm_bf16_cfg", A, B, C, workspace, stream, torch.bfloat16, (ctypes.byref(cfg),))


def gemm_bf16(A, B, C, stream=None) -> None:
    """C[M, N] = A[M, K] . B[N, K]^T with torch.bfloat16 tensors, fp32
    accumulate, bf16 out (round to nearest even)."""
    import torch
    _gemm_16("gemm_bf16", A, B, C, stream, torch.bfloat16)


def gemm_bf16_ex(A, B, C, tile_id: int = -1, stagger: int = -1, stream=None) -> None:
    import torch
    _gemm_16("gemm_bf16_ex", A, B, C, stream, torch.bfloat16, (int(tile_id), int(stagger)))


def _gemv_16(entry, x, B, y, stream, dtype, kn):
    if x.dtype != dtype or y.dtype != dtype:
        raise TypeError(f"x and y must be {dtype}")
    if x.dim() != 1 or y.dim() != 1 or x.stride(0) != 1 or y.stride(0) != 1:
        raise ValueError("x and y must be contiguous vectors")
    if kn:
        K, N = B.shape
    else:
        N, K = B.shape
    if x.shape[0] != K or y.shape[0] != N:
        raise ValueError(f"shape mismatch x{tuple(x.shape)} B{tuple(B.shape)} y{tuple(y.shape)}")
    pb, ldb = _rows(B, "B", dtype)
    rc = getattr(lib(), entry)(N, K, x.data_ptr(), pb, ldb, y.data_ptr(), _stream_handle(stream))
    if rc != SDT_OK:
        raise SdtError(rc, entry)


def stream_read_runs(buf, rows: int, row_bytes: int, run_bytes: int, rows_per_wg: int, out,
                     stream=None) -> None:
    """Enqueue the run-length read measurement kernel over a device buffer
    (rows x row_bytes bytes); out: an int32 device tensor of at least
    (row_bytes // run_bytes) * (rows // rows_per_wg) elements."""
    rc = lib().sdt_stream_read_runs(buf.data_ptr(), int(rows), int(row_bytes), int(run_bytes),
                                    int(rows_per_wg), out.data_ptr(), _stream_handle(stream))
    if rc != SDT_OK:
        raise SdtError(rc, "sdt_stream_read_runs")


def gemv_kn_workspace_size(N: int, K: int) -> int:
    """Bytes of workspace gemv_f16_m1_kn_ws splits with (0: no split)."""
    return int(lib().sdt_gemv_kn_workspace_size(int(N), int(K)))


def _gemv_kn_ws(entry, x, B, y, workspace, stream, dtype):
    if x.dtype != dtype or y.dtype != dtype:
        raise TypeError(f"x and y must be {dtype}")
    if x.dim() != 1 or y.dim() != 1 or x.stride(0) != 1 or y.stride(0) != 1:
        raise ValueError("x and y must be contiguous vectors")
    K, N = B.shape
    if x.shape[0] != K or y.shape[0] != N:
        raise ValueError(f"shape mismatch x{tuple(x.shape)} B{tuple(B.shape)} y{tuple(y.shape)}")
    pb, ldb = _rows(B, "B", dtype)
    wp, wb = _ws_args(workspace)
    rc = getattr(lib(), entry)(N, K, x.data_ptr(), pb, ldb, y.data_ptr(), wp, wb,
                               _stream_handle(stream))
    if rc != SDT_OK:
        raise SdtError(rc, entry)


def gemv_f16_m1_kn_ws(x, B, y, workspace=None, stream=None) -> None:
    """gemv_f16_m1_kn split over K through `workspace` (a Workspace of at least
    gemv_kn_workspace_size(N, K) bytes; smaller or None: the one-launch kernel)."""
    import torch
    _gemv_kn_ws("gemv_f16_m1_kn_ws", x, B, y, workspace, stream, torch.float16)


def gemv_bf16_m1_kn_ws(x, B, y, workspace=None, stream=None) -> None:
    import torch
    _gemv_kn_ws("gemv_bf16_m1_kn_ws", x, B, y, workspace, stream, torch.bfloat16)


def gemv_bf16_m1(x, B, y, stream=None) -> None:
    """y[N] = x[K] . B[N, K]^T with torch.bfloat16 tensors (B stored K-major)."""
    import torch
    _gemv_16("gemv_bf16_m1", x, B, y, stream, torch.bfloat16, kn=False)


def gemv_bf16_m1_kn(x, B, y, stream=None) -> None:
    """y[N] = x[K] . B[K, N] with torch.bfloat16 tensors (B as K rows of N)."""
    import torch
    _gemv_16("gemv_bf16_m1_kn", x, B, y, stream, torch.bfloat16, kn=True)


def gemm_f16_raw(M, N, K, A_ptr, lda, B_ptr, ldb, C_ptr, ldc, stream_ptr=None) -> int:
    """The C call with raw integers/pointers; returns the status."""
    return int(lib().gemm_f16(int(M), int(N), int(K), A_ptr, int(lda), B_ptr, int(ldb),
                              C_ptr, int(ldc), stream_ptr))


def gemv_f16_m1_raw(N, K, x_ptr, B_ptr, ldb, y_ptr, stream_ptr=None) -> int:
    return int(lib().gemv_f16_m1(int(N), int(K), x_ptr, B_ptr, int(ldb), y_ptr, stream_ptr))


# ---- MX4 matrices ---------------------------------------------------------------

def mx4_row_bytes(K: int) -> int:
    return -(-int(K) // 32) * 16


def mx4_scale_bytes(rows: int, K: int) -> int:
    return -(-int(rows) // 64) * -(-int(K) // 256) * 512


class Mx4:
    """An MX4 matrix on the device (the format: include/sdt.h): uint8 codes `q`
    [rows, >= mx4_row_bytes(K)] with unit stride along a row, and the tiled scale
    bytes `s` [mx4_scale_bytes(rows, K)].  With a leading dimension on both, one
    matrix per expert."""

    __slots__ = ("q", "s", "rows", "K", "device")      # device: its index, -1 the host

    def __init__(self, q, s, rows: int, K: int):
        import torch
        rows, K = int(rows), int(K)
        u8 = torch.uint8
        if q.dtype is not u8 or s.dtype is not u8:
            raise TypeError("Mx4: codes and scales must be uint8")
        where = q.get_device() if q.is_cuda else -1
        if where < 0 or not s.is_cuda or s.get_device() != where:
            raise TypeError("Mx4: codes and scales must be on one device")
        qs, ss = q.shape, s.shape
        if len(qs) not in (2, 3) or len(ss) != len(qs) - 1 or (len(qs) == 3 and qs[0] != ss[0]):
            raise ValueError(f"Mx4: codes {tuple(qs)} and scales {tuple(ss)} do not match")
        if qs[-2] != rows or qs[-1] < -(-K // 32) * 16 or \
                ss[-1] < -(-rows // 64) * -(-K // 256) * 512:
            raise ValueError(f"Mx4: codes {tuple(qs)} and scales {tuple(ss)} cannot hold "
                             f"{rows} x {K}")
        if q.stride()[-1] != 1 or s.stride()[-1] != 1:
            raise ValueError("Mx4: unit stride along rows of codes and along the scales")
        self.q, self.s, self.rows, self.K, self.device = q, s, rows, K, where

    @classmethod
    def empty(cls, rows: int, K: int, experts: int | None = None, device="cuda") -> "Mx4":
        import torch
        rows, K = int(rows), int(K)
        lead = () if experts is None else (int(experts),)
        m = cls.__new__(cls)                 # tensors that fit by construction: no checks
        m.q = torch.empty(lead + (rows, -(-K // 32) * 16), dtype=torch.uint8, device=device)
        m.s = torch.empty(lead + (-(-rows // 64) * -(-K // 256) * 512,), dtype=torch.uint8,
                          device=device)
        m.rows, m.K, m.device = rows, K, m.q.get_device()
        return m

    def ldq(self) -> int:
        """Bytes from row to row (a single row's are its own bytes)."""
        return self.q.stride(-2) if self.rows > 1 else max(self.q.stride(-2), mx4_row_bytes(self.K))

    def _one(self, name):
        q = self.q
        stride = q.stride()
        if len(stride) != 2:
            raise ValueError(f"{name} must be one matrix, not one per expert")
        ld = stride[0]
        if self.rows <= 1:
            ld = max(ld, -(-self.K // 32) * 16)
        return q.data_ptr(), ld, self.s.data_ptr()

    def _experts(self, experts, name) -> SdtMx4Experts:
        if self.q.dim() != 3 or self.q.shape[0] != experts:
            raise ValueError(f"{name} must hold one matrix for each of {experts} experts")
        given = SdtMx4Experts(self.q.data_ptr(), self.ldq(), self.q.stride(0), self.s.data_ptr(),
                              self.s.stride(0))
        given.experts, given.device = experts, self.device
        return given


def _check(rc: int, where: str) -> None:
    if rc != SDT_OK:
        raise SdtError(rc, where)


def _apart(where: str, *devices):
    """Operands of different devices (-1: the host): the C ABI takes addresses, which
    do not tell, so no call is made with them."""
    return TypeError(f"{where}: operands must be on one device, not on {devices} (-1: the host)")


def _quantize(entry, X, out, dtype, stream):
    px, ldx = _rows(X, "X", dtype)
    if X.shape != (out.rows, out.K):
        raise ValueError(f"shape mismatch X{tuple(X.shape)} out ({out.rows}, {out.K})")
    if out.device != X.get_device():
        raise _apart(entry, X.get_device(), out.device)
    q, ldq, s = out._one("out")
    _check(getattr(lib(), entry)(out.rows, out.K, px, ldx, q, ldq, s, _stream_handle(stream)), entry)


def mx4_quantize_f16(X, out: Mx4, stream=None) -> None:
    """out = X [rows, K] quantised to MX4."""
    import torch
    _quantize("mx4_quantize_f16", X, out, torch.float16, stream)


def mx4_quantize_bf16(X, out: Mx4, stream=None) -> None:
    import torch
    _quantize("mx4_quantize_bf16", X, out, torch.bfloat16, stream)


def _quantize_rows(entry, X, index, divisor, out, dtype, stream):
    import torch
    px, ldx = _rows(X, "X", dtype)
    if X.shape[1] != out.K or tuple(index.shape) != (out.rows,):
        raise ValueError(f"shape mismatch X{tuple(X.shape)} index{tuple(index.shape)} out "
                         f"({out.rows}, {out.K})")
    _ints(index, "index")
    if not (out.device == X.get_device() == index.get_device()):
        raise _apart(entry, X.get_device(), index.get_device(), out.device)
    q, ldq, s = out._one("out")
    _check(getattr(lib(), entry)(out.rows, out.K, px, X.shape[0], ldx, index.data_ptr(),
                                 int(divisor), q, ldq, s, _stream_handle(stream)), entry)


def mx4_quantize_rows_f16(X, index, divisor: int, out: Mx4, stream=None) -> None:
    """Row p of out = row index[p] // divisor of X (divisor 0: row p), quantised;
    rows with index[p] < 0 keep their codes and get zero scales."""
    import torch
    _quantize_rows("mx4_quantize_rows_f16", X, index, divisor, out, torch.float16, stream)


def mx4_quantize_rows_bf16(X, index, divisor: int, out: Mx4, stream=None) -> None:
    import torch
    _quantize_rows("mx4_quantize_rows_bf16", X, index, divisor, out, torch.bfloat16, stream)


def _dequantize(entry, m, Y, dtype, stream):
    py, ldy = _rows(Y, "Y", dtype)
    if Y.shape != (m.rows, m.K):
        raise ValueError(f"shape mismatch matrix ({m.rows}, {m.K}) Y{tuple(Y.shape)}")
    if m.device != Y.get_device():
        raise _apart(entry, m.device, Y.get_device())
    q, ldq, s = m._one("matrix")
    _check(getattr(lib(), entry)(m.rows, m.K, q, ldq, s, py, ldy, _stream_handle(stream)), entry)


def mx4_dequantize_f16(m: Mx4, Y, stream=None) -> None:
    """Y [rows, K] = the values of an MX4 matrix."""
    import torch
    _dequantize("mx4_dequantize_f16", m, Y, torch.float16, stream)


def mx4_dequantize_bf16(m: Mx4, Y, stream=None) -> None:
    import torch
    _dequantize("mx4_dequantize_bf16", m, Y, torch.bfloat16, stream)


def mx4_dequantize_f32(m: Mx4, Y, stream=None) -> None:
    import torch
    _dequantize("mx4_dequantize_f32", m, Y, torch.float32, stream)


def mx4_pack_scales(scales, out: Mx4, stream=None) -> None:
    """out.s = row-major scale bytes [rows, ceil(K / 32)], tiled."""
    import torch
    p, ld = _rows(scales, "scales", torch.uint8)
    if tuple(scales.shape) != (out.rows, -(-out.K // 32)):
        raise ValueError(f"shape mismatch scales{tuple(scales.shape)} out ({out.rows}, {out.K})")
    if out.device != scales.get_device():
        raise _apart("mx4_pack_scales", scales.get_device(), out.device)
    _, _, s = out._one("out")
    _check(lib().mx4_pack_scales(out.rows, out.K, p, ld, s, _stream_handle(stream)),
           "mx4_pack_scales")


def _gemm_mx4(entry, A, B, C, dtype, stream):
    if A.K != B.K or C.shape != (A.rows, B.rows):
        raise ValueError(f"shape mismatch A({A.rows}, {A.K}) B({B.rows}, {B.K}) C{tuple(C.shape)}")
    pa, lda, sa = A._one("A")
    pb, ldb, sb = B._one("B")
    pc, ldc = _rows(C, "C", dtype)
    if not (A.device == B.device == C.get_device()):
        raise _apart(entry, A.device, B.device, C.get_device())
    _check(getattr(lib(), entry)(A.rows, B.rows, A.K, pa, lda, sa, pb, ldb, sb, pc, ldc,
                                 _stream_handle(stream)), entry)


def gemm_mx4_f16(A: Mx4, B: Mx4, C, stream=None) -> None:
    """C[M, N] = A[M, K] . B[N, K]^T for MX4 matrices, fp32 accumulate, fp16 out."""
    import torch
    _gemm_mx4("gemm_mx4_f16", A, B, C, torch.float16, stream)


def gemm_mx4_bf16(A: Mx4, B: Mx4, C, stream=None) -> None:
    import torch
    _gemm_mx4("gemm_mx4_bf16", A, B, C, torch.bfloat16, stream)


def _gemv_mx4(entry, x, B, y, dtype, stream):
    if x.dtype != dtype or y.dtype != dtype:
        raise TypeError(f"x and y must be {dtype}")
    if not x.is_cuda or not y.is_cuda:
        raise TypeError("x and y must be device tensors")
    if x.stride() != (1,) or y.stride() != (1,):
        raise ValueError("x and y must be contiguous vectors")
    if x.shape[0] != B.K or y.shape[0] != B.rows:
        raise ValueError(f"shape mismatch x{tuple(x.shape)} B({B.rows}, {B.K}) y{tuple(y.shape)}")
    if not (B.device == x.get_device() == y.get_device()):
        raise _apart(entry, x.get_device(), B.device, y.get_device())
    pb, ldb, sb = B._one("B")
    _check(getattr(lib(), entry)(B.rows, B.K, x.data_ptr(), pb, ldb, sb, y.data_ptr(),
                                 _stream_handle(stream)), entry)


def gemv_mx4_m1_f16(x, B: Mx4, y, stream=None) -> None:
    """y[N] = x[K] . B[N, K]^T with 16-bit activations and MX4 weights."""
    import torch
    _gemv_mx4("gemv_mx4_m1_f16", x, B, y, torch.float16, stream)


def gemv_mx4_m1_bf16(x, B: Mx4, y, stream=None) -> None:
    import torch
    _gemv_mx4("gemv_mx4_m1_bf16", x, B, y, torch.bfloat16, stream)


# ---- experts -----------------------------------------------------------------------

_SCORES = {"softmax": 0, "sigmoid": 1}


def route_cfg(topk: int, score: str = "softmax", groups: int = 1, groups_kept: int = 1,
              group_top: int = 1, renormalize: bool = True, scale: float = 1.0) -> SdtRoute:
    """How tokens choose experts (sdt_route)."""
    if score not in _SCORES:
        raise ValueError(f"score must be one of {sorted(_SCORES)}, got {score!r}")
    return SdtRoute(int(topk), _SCORES[score], int(groups), int(groups_kept), int(group_top),
                    1 if renormalize else 0, float(scale))


def _ints(t, name):
    import torch
    if t.dtype is not torch.int32:
        raise TypeError(f"{name} must be int32, got {t.dtype}")
    if not t.is_cuda:
        raise TypeError(f"{name} must be a device tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _floats(t, name):
    import torch
    if t.dtype is not torch.float32:
        raise TypeError(f"{name} must be float32, got {t.dtype}")
    if not t.is_cuda:
        raise TypeError(f"{name} must be a device tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _logit_type(t, name):
    import torch
    dtype = t.dtype
    if dtype is torch.float32:
        return "f32"
    if dtype is torch.float16:
        return "f16"
    if dtype is torch.bfloat16:
        return "bf16"
    raise TypeError(f"{name} must be float32, float16 or bfloat16, got {dtype}")


def moe_route(logits, idx, weights, cfg: SdtRoute, bias=None, stream=None) -> None:
    """idx [T, topk] int32, weights [T, topk] float32 = the experts of T tokens
    from their logits [T, E]."""
    kind = _logit_type(logits, "logits")
    p, ld = _rows(logits, "logits", logits.dtype)
    T, E = logits.shape
    chosen = (T, cfg.topk)
    if idx.shape != chosen or weights.shape != chosen:
        raise ValueError(f"shape mismatch logits{tuple(logits.shape)} topk {cfg.topk} "
                         f"idx{tuple(idx.shape)} weights{tuple(weights.shape)}")
    if bias is not None and tuple(bias.shape) != (E,):
        raise ValueError(f"bias must hold {E} values")
    b = None if bias is None else _floats(bias, "bias")
    entry = "moe_route_" + kind
    where = logits.get_device()
    if not (idx.get_device() == weights.get_device() == where) or \
            (bias is not None and bias.get_device() != where):
        raise _apart(entry, where, idx.get_device(), weights.get_device(),
                     where if bias is None else bias.get_device())
    _check(getattr(lib(), entry)(T, E, p, ld, b, ctypes.byref(cfg), _ints(idx, "idx"),
                                 _floats(weights, "weights"), _stream_handle(stream)), entry)


def moe_route_backward(logits, idx, dweights, dlogits, cfg: SdtRoute, stream=None) -> None:
    """dlogits [T, E] (the logits' type) from dweights [T, topk] float32."""
    kind = _logit_type(logits, "logits")
    p, ld = _rows(logits, "logits", logits.dtype)
    d, ldd = _rows(dlogits, "dlogits", logits.dtype)
    T, E = logits.shape
    if tuple(idx.shape) != (T, cfg.topk) or tuple(dweights.shape) != (T, cfg.topk) or \
            tuple(dlogits.shape) != (T, E):
        raise ValueError(f"shape mismatch logits{tuple(logits.shape)} topk {cfg.topk} "
                         f"idx{tuple(idx.shape)} dweights{tuple(dweights.shape)} "
                         f"dlogits{tuple(dlogits.shape)}")
    entry = "moe_route_backward_" + kind
    where = logits.get_device()
    if not (idx.get_device() == dweights.get_device() == dlogits.get_device() == where):
        raise _apart(entry, where, idx.get_device(), dweights.get_device(), dlogits.get_device())
    _check(getattr(lib(), entry)(T, E, p, ld, ctypes.byref(cfg), _ints(idx, "idx"),
                                 _floats(dweights, "dweights"), d, ldd, _stream_handle(stream)),
           entry)


def moe_plan_rows(tokens: int, topk: int, experts: int) -> int:
    """Rows of a plan's segments, enough for any choice of experts."""
    v = int(lib().sdt_moe_plan_rows(int(tokens), int(topk), int(experts)))
    if v < 0:
        raise SdtError(SDT_ERR_INVALID_ARG, "sdt_moe_plan_rows")
    return v


class MoePlan:
    """The arrays of a plan (sdt_moe_plan) for `tokens` tokens of `topk` experts
    each out of `experts`: int32 device tensors counts, offsets, rows, pos, tiles."""

    __slots__ = ("tokens", "topk", "experts", "size", "counts", "offsets", "rows", "pos", "tiles",
                 "device", "_struct")

    @classmethod
    def empty(cls, tokens: int, topk: int, experts: int, device="cuda") -> "MoePlan":
        import torch
        p = cls()
        p.tokens, p.topk, p.experts = tokens, topk, experts = int(tokens), int(topk), int(experts)
        p.size = size = moe_plan_rows(tokens, topk, experts)
        sizes = (experts, experts + 1, size, tokens * topk, size // 64)
        flat = torch.empty(sum(sizes), dtype=torch.int32, device=device)
        p.counts, p.offsets, p.rows, p.pos, p.tiles = flat.split(sizes)
        p.device = flat.get_device()         # its index, -1 the host
        at = flat.data_ptr()
        offsets = at + 4 * experts
        rows = offsets + 4 * experts + 4
        pos = rows + 4 * size
        p._struct = SdtMoePlan(tokens, topk, experts, at, offsets, rows, pos,
                               pos + 4 * tokens * topk)
        return p


def moe_plan(idx, plan: MoePlan, stream=None) -> None:
    """Fills plan from idx [tokens, topk]: the slots sorted by expert."""
    if tuple(idx.shape) != (plan.tokens, plan.topk):
        raise ValueError(f"idx must be ({plan.tokens}, {plan.topk}), got {tuple(idx.shape)}")
    if plan.device != idx.get_device():
        raise _apart("moe_plan", idx.get_device(), plan.device)
    _check(lib().moe_plan(_ints(idx, "idx"), ctypes.byref(plan._struct), _stream_handle(stream)),
           "moe_plan")


def _moe_gemm_mx4(entry, plan, A, B, C, up, dtype, stream):
    if A.K != B.K or A.rows != plan.size or tuple(C.shape) != (plan.size, B.rows) or \
            (up is not None and (up.K, up.rows) != (B.K, B.rows)):
        raise ValueError(f"shape mismatch plan {plan.size} rows A({A.rows}, {A.K}) "
                         f"B({B.rows}, {B.K}) C{tuple(C.shape)}")
    pa, lda, sa = A._one("A")
    pc, ldc = _rows(C, "C", dtype)
    b = B._experts(plan.experts, "B")
    u = None if up is None else ctypes.byref(up._experts(plan.experts, "up"))
    if not (plan.device == A.device == B.device == C.get_device()) or \
            (up is not None and up.device != plan.device):
        raise _apart(entry, plan.device, A.device, B.device, C.get_device(),
                     B.device if up is None else up.device)
    _check(getattr(lib(), entry)(ctypes.byref(plan._struct), B.rows, B.K, pa, lda, sa,
                                 ctypes.byref(b), u, pc, ldc, _stream_handle(stream)), entry)


def moe_gemm_mx4_f16(plan: MoePlan, A: Mx4, B: Mx4, C, up: Mx4 | None = None, stream=None) -> None:
    """C[p] = A[p] . B_e^T for the plan's rows, e a row's expert; with `up`,
    silu(A . B_e^T) * (A . up_e^T)."""
    import torch
    _moe_gemm_mx4("moe_gemm_mx4_f16", plan, A, B, C, up, torch.float16, stream)


def moe_gemm_mx4_bf16(plan: MoePlan, A: Mx4, B: Mx4, C, up: Mx4 | None = None,
                      stream=None) -> None:
    import torch
    _moe_gemm_mx4("moe_gemm_mx4_bf16", plan, A, B, C, up, torch.bfloat16, stream)


def _moe_combine(entry, plan, D, weights, Y, dtype, stream):
    pd, ldd = _rows(D, "D", dtype)
    py, ldy = _rows(Y, "Y", dtype)
    N = D.shape[1]
    if D.shape[0] != plan.size or tuple(Y.shape) != (plan.tokens, N) or \
            tuple(weights.shape) != (plan.tokens, plan.topk):
        raise ValueError(f"shape mismatch plan {plan.size} rows D{tuple(D.shape)} "
                         f"weights{tuple(weights.shape)} Y{tuple(Y.shape)}")
    if not (plan.device == D.get_device() == weights.get_device() == Y.get_device()):
        raise _apart(entry, plan.device, D.get_device(), weights.get_device(), Y.get_device())
    _check(getattr(lib(), entry)(ctypes.byref(plan._struct), N, pd, ldd,
                                 _floats(weights, "weights"), py, ldy, _stream_handle(stream)), entry)


def moe_combine_f16(plan: MoePlan, D, weights, Y, stream=None) -> None:
    """Y[t] = sum_j weights[t, j] * D[pos(t, j)]."""
    import torch
    _moe_combine("moe_combine_f16", plan, D, weights, Y, torch.float16, stream)


def moe_combine_bf16(plan: MoePlan, D, weights, Y, stream=None) -> None:
    import torch
    _moe_combine("moe_combine_bf16", plan, D, weights, Y, torch.bfloat16, stream)


def moe_experts_workspace_size(tokens: int, topk: int, experts: int, N: int, K: int) -> int:
    """Workspace bytes of moe_experts_mx4."""
    v = int(lib().sdt_moe_experts_workspace_size(int(tokens), int(topk), int(experts), int(N),
                                                 int(K)))
    if v < 0:
        raise SdtError(SDT_ERR_INVALID_ARG, "sdt_moe_experts_workspace_size")
    return v


def moe_experts_mx4(layer: SdtMoeLayer, X, idx, weights, plan: MoePlan, Y, workspace,
                    stream=None) -> None:
    """A layer of gated MX4 experts in one call (moe.Mx4Experts keeps the layer);
    workspace: a uint8 device tensor of moe_experts_workspace_size bytes.  A layer
    made of plain addresses has to hold as many matrices as the plan has experts."""
    import torch
    entry = {torch.float16: "moe_experts_mx4_f16", torch.bfloat16: "moe_experts_mx4_bf16"}.get(X.dtype)
    if entry is None:
        raise TypeError(f"X must be float16 or bfloat16, got {X.dtype}")
    shape, chosen = (plan.tokens, layer.K), (plan.tokens, plan.topk)
    if X.shape != shape or Y.shape != shape or idx.shape != chosen or weights.shape != chosen:
        raise ValueError(f"shape mismatch X{tuple(X.shape)} Y{tuple(Y.shape)} idx{tuple(idx.shape)} "
                         f"weights{tuple(weights.shape)}")
    if layer.experts is not None and layer.experts != plan.experts:
        raise ValueError(f"a plan of {plan.experts} experts for a layer of {layer.experts}")
    px, ldx = _rows(X, "X", X.dtype)
    py, ldy = _rows(Y, "Y", X.dtype)
    if workspace.dtype is not torch.uint8 or not workspace.is_contiguous():
        raise TypeError("workspace must be contiguous uint8")
    where = X.get_device()
    if not (idx.get_device() == weights.get_device() == plan.device == Y.get_device() ==
            workspace.get_device() == where) or layer.device not in (None, where):
        raise _apart(entry, where, idx.get_device(), weights.get_device(), plan.device,
                     Y.get_device(), workspace.get_device(), layer.device)
    _check(getattr(lib(), entry)(ctypes.byref(layer), _ints(idx, "idx"),
                                 _floats(weights, "weights"), ctypes.byref(plan._struct), px, ldx,
                                 py, ldy, workspace.data_ptr(), workspace.numel(),
                                 _stream_handle(stream)), entry)


# ---- 8-bit matrices with a scale for each block of 128 ------------------------------

class Fp8:
    """An 8-bit matrix on the device (the format: include/sdt.h): float8_e4m3fn codes
    `q` [rows, K], rows a multiple of 16 bytes apart, and float32 scales `s`: of each
    row and block of 128 k, [ceil(K / 128), rows] (block 1, activations), or of each
    block of 128 rows x 128 k, [ceil(rows / 128), ceil(K / 128)] (block 128, weights).
    The two tensors are the matrix's for good; what they hold may change."""

    # device: its index, -1 the host; _at: the memory that _given and _bytes are made from
    __slots__ = ("_q", "_s", "rows", "K", "block", "device", "_at", "_given", "_bytes")

    @property
    def q(self):
        return self._q

    @property
    def s(self):
        return self._s

    def __init__(self, q, s, block: int = 1):
        import torch
        if block not in (1, 128):
            raise ValueError(f"Fp8: block must be 1 or 128, got {block}")
        if q.dtype is not torch.float8_e4m3fn or s.dtype is not torch.float32:
            raise TypeError(f"Fp8: codes must be float8_e4m3fn and scales float32, got {q.dtype} and "
                            f"{s.dtype}")
        where = q.get_device() if q.is_cuda else -1
        if where < 0 or not s.is_cuda or s.get_device() != where:
            raise TypeError("Fp8: codes and scales must be on one device")
        if q.dim() != 2:
            raise ValueError(f"Fp8: codes {tuple(q.shape)} must be 2-D")
        (self.rows, self.K), self.block, self.device = q.shape, block, where
        self._q, self._s, self._at = q, s, None
        self._args()

    @classmethod
    def empty(cls, rows: int, K: int, block: int = 1, device="cuda") -> "Fp8":
        import torch
        if block not in (1, 128):
            raise ValueError(f"Fp8: block must be 1 or 128, got {block}")
        m = cls.__new__(cls)                 # tensors that fit by construction: no checks
        kb, ld = -(-K // 128), -(-K // 16) * 16
        q = torch.empty(rows, ld, dtype=torch.float8_e4m3fn, device=device)
        m._q = q if ld == K else q[:, :K]
        m._s = torch.empty((kb, rows) if block == 1 else (-(-rows // 128), kb), dtype=torch.float32,
                          device=device)
        m.rows, m.K, m.block, m.device, m._at = rows, K, block, q.get_device(), None
        return m

    def _args(self):
        """Codes, bytes from row to row, scales, floats from row to row of them; made again
        where the tensors have been given other memory or strides."""
        q, s = self._q, self._s
        qs, ss = q.stride(), s.stride()
        at = q.data_ptr(), qs, s.data_ptr(), ss
        if at != self._at:
            rows, K, kb = self.rows, self.K, -(-self.K // 128)
            fits = (kb, rows) if self.block == 1 else (-(-rows // 128), kb)
            if q.shape != (rows, K) or s.shape != fits:
                raise ValueError(f"Fp8: a {rows} x {K} matrix of block {self.block} has scales {fits}, not "
                                 f"codes {tuple(q.shape)} and scales {tuple(s.shape)}")
            if (K > 1 and qs[1] != 1) or (fits[1] > 1 and ss[1] != 1):
                raise ValueError("Fp8: unit stride along rows of codes and of scales")
            # several rows of scales: their own stride, so that rows that overlap are refused
            given = (at[0], qs[0] if rows > 1 else max(qs[0], K), at[2], ss[0] if fits[0] > 1 else fits[1])
            # _at last: another thread that finds it finds the rest
            self._given, self._bytes, self._at = given, _pack_fp8(*given, self.block), at
        return self._given

    def _packed(self):
        """An sdt_fp8, as bytes."""
        self._args()
        return self._bytes


def _quantize8(entry, X, out, dtype, stream):
    px, ldx = _rows(X, "X", dtype)
    if X.shape != (out.rows, out.K):
        raise ValueError(f"shape mismatch X{tuple(X.shape)} out ({out.rows}, {out.K})")
    if out.device != X.get_device():
        raise _apart(entry, X.get_device(), out.device)
    _check(getattr(lib(), entry)(out.rows, out.K, px, ldx, out._packed(), _stream_handle(stream)), entry)


def fp8_quantize_f16(X, out: Fp8, stream=None) -> None:
    """out = X [rows, K] in 8 bits."""
    import torch
    _quantize8("fp8_quantize_f16", X, out, torch.float16, stream)


def fp8_quantize_bf16(X, out: Fp8, stream=None) -> None:
    import torch
    _quantize8("fp8_quantize_bf16", X, out, torch.bfloat16, stream)


def _dequantize8(entry, m, Y, dtype, stream):
    py, ldy = _rows(Y, "Y", dtype)
    if Y.shape != (m.rows, m.K):
        raise ValueError(f"shape mismatch matrix ({m.rows}, {m.K}) Y{tuple(Y.shape)}")
    if m.device != Y.get_device():
        raise _apart(entry, m.device, Y.get_device())
    _check(getattr(lib(), entry)(m.rows, m.K, m._packed(), py, ldy, _stream_handle(stream)), entry)


def fp8_dequantize_f16(m: Fp8, Y, stream=None) -> None:
    """Y [rows, K] = the values of an 8-bit matrix."""
    import torch
    _dequantize8("fp8_dequantize_f16", m, Y, torch.float16, stream)


def fp8_dequantize_bf16(m: Fp8, Y, stream=None) -> None:
    import torch
    _dequantize8("fp8_dequantize_bf16", m, Y, torch.bfloat16, stream)


def fp8_dequantize_f32(m: Fp8, Y, stream=None) -> None:
    import torch
    _dequantize8("fp8_dequantize_f32", m, Y, torch.float32, stream)


_split_sizes = {}          # (entry point, sizes): bytes that let the product be split


def _split_size(entry, M, N, K):
    key = (entry, M, N, K)
    need = _split_sizes.get(key)
    if need is None:
        need = int(getattr(lib(), entry)(M, N, K))
        if len(_split_sizes) >= 4096:
            _split_sizes.clear()
        _split_sizes[key] = need
    return need


def _split_buffer(need, workspace, where, stream):
    """A work buffer's address, its bytes and what keeps it: `workspace`, or `need` bytes made here, of
    the stream that runs the call (the allocator gives them to no other while they are in use)."""
    if workspace is not None or need <= 0:
        return (*_buffer(workspace, where), workspace)
    import torch
    if stream is None:
        t = torch.empty(need, dtype=torch.uint8, device=where)
    else:
        with torch.cuda.stream(stream):
            t = torch.empty(need, dtype=torch.uint8, device=where)
    return t.data_ptr(), need, t


def gemm_fp8_workspace_size(M: int, N: int, K: int) -> int:
    """Workspace bytes that let gemm_fp8 split a C [M, N] along K (0: no split)."""
    v = int(lib().sdt_gemm_fp8_workspace_size(int(M), int(N), int(K)))
    if v < 0:
        raise SdtError(SDT_ERR_INVALID_ARG, "sdt_gemm_fp8_workspace_size")
    return v


def _gemm_fp8(entry, A, B, C, dtype, workspace, stream):
    M, N, K = A.rows, B.rows, A.K
    if K != B.K or C.shape != (M, N):
        raise ValueError(f"shape mismatch A({M}, {K}) B({N}, {B.K}) C{tuple(C.shape)}")
    if A.block != 1 or B.block != 128:
        raise ValueError(f"A must have blocks of 1 x 128 and B of 128 x 128, not {A.block} and {B.block}")
    pc, ldc = _rows(C, "C", dtype)
    where = A.device
    if not (where == B.device == C.get_device()):
        raise _apart(entry, where, B.device, C.get_device())
    need = _split_size("sdt_gemm_fp8_workspace_size", M, N, K) if M > 16 else 0
    wp, wn, _kept = _split_buffer(need, workspace, where, stream)
    _check(getattr(lib(), entry)(M, N, K, A._packed(), B._packed(), pc, ldc, wp, wn,
                                 _stream_handle(stream)), entry)


def gemm_fp8_f16(A: Fp8, B: Fp8, C, workspace=None, stream=None) -> None:
    """C[M, N] = A[M, K] . B[N, K]^T for 8-bit matrices (A of block 1, B of block
    128), fp32 accumulate, fp16 out.  workspace: a uint8 device tensor of
    gemm_fp8_workspace_size bytes instead of one that the call makes."""
    import torch
    _gemm_fp8("gemm_fp8_f16", A, B, C, torch.float16, workspace, stream)


def gemm_fp8_bf16(A: Fp8, B: Fp8, C, workspace=None, stream=None) -> None:
    import torch
    _gemm_fp8("gemm_fp8_bf16", A, B, C, torch.bfloat16, workspace, stream)


# ---- the norm and the gated feed-forward block ------------------------------------------

def _kind16(t, name):
    """The suffix of the entry points for tensors of t's type."""
    import torch
    if t.dtype is torch.float16:
        return "f16"
    if t.dtype is torch.bfloat16:
        return "bf16"
    raise TypeError(f"{name} must be float16 or bfloat16, got {t.dtype}")


def _matrix(t, name, shape, dtype, where):
    """Address and row stride of a matrix that a call needs in this shape and place."""
    if t.shape != shape:
        raise ValueError(f"{name} must be {tuple(shape)}, got {tuple(t.shape)}")
    got = _rows(t, name, dtype)
    if t.get_device() != where:
        raise _apart(name, where, t.get_device())
    return got


def _vector(t, name, n, dtype, where):
    if tuple(t.shape) != (n,) or not t.is_contiguous():
        raise ValueError(f"{name} must be {n} contiguous values, got {tuple(t.shape)}")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.get_device() != where:
        raise _apart(name, where, t.get_device())
    return t.data_ptr()


def _buffer(t, where):
    """Address and bytes of a work buffer (None: none)."""
    import torch
    if t is None:
        return 0, 0
    if t.dtype is not torch.uint8 or not t.is_contiguous():
        raise TypeError("workspace must be contiguous uint8")
    if t.get_device() != where:
        raise _apart("workspace", where, t.get_device())
    return t.data_ptr(), t.numel()


def rms_norm(x, weight, y=None, q: Fp8 | None = None, residual=None, total=None, rstd=None,
             eps: float = 1e-6, stream=None) -> None:
    """y [rows, K] = t * rstd * weight with t = x + residual rounded to the type and
    rstd = 1 / sqrt(mean(t^2) + eps).  float16 or bfloat16 x, residual, weight [K]
    (None: ones), y and total (t); q: y in 8 bits; rstd [rows] float32, for the
    gradient.  At least one of y, q, total and rstd is given."""
    import torch
    kind = _kind16(x, "x")
    px, ldx = _rows(x, "x", x.dtype)
    shape, dtype, where = x.shape, x.dtype, x.get_device()
    rows, K = shape
    none = (0, 0)
    pr, ldr = none if residual is None else _matrix(residual, "residual", shape, dtype, where)
    pt, ldt = none if total is None else _matrix(total, "total", shape, dtype, where)
    py, ldy = none if y is None else _matrix(y, "y", shape, dtype, where)
    pw = 0 if weight is None else _vector(weight, "weight", K, dtype, where)
    ps = 0 if rstd is None else _vector(rstd, "rstd", rows, torch.float32, where)
    if q is None:
        codes = (0, 0, 0, 0)
    else:
        if (q.rows, q.K) != (rows, K) or q.block != 1:
            raise ValueError(f"q must be {rows} x {K} of block 1, got {q.rows} x {q.K} of {q.block}")
        if q.device != where:
            raise _apart("rms_norm", where, q.device)
        codes = q._args()
    entry = "rms_norm_" + kind
    args = _pack_norm(rows, K, px, ldx, pr, ldr, pw, eps, pt, ldt, py, ldy, *codes, ps)
    _check(getattr(lib(), entry)(args, _stream_handle(stream)), entry)


def rms_norm_workspace_size(rows: int, K: int) -> int:
    """Workspace bytes of rms_norm_backward with dweight."""
    v = int(lib().sdt_rms_norm_workspace_size(int(rows), int(K)))
    if v < 0:
        raise SdtError(SDT_ERR_INVALID_ARG, "sdt_rms_norm_workspace_size")
    return v


def rms_norm_backward(total, weight, rstd, dy, dx, dweight=None, workspace=None, dtotal=None,
                      stream=None) -> None:
    """dx [rows, K], the gradient of x (and of the residual), and dweight [K] float32,
    from dy and, where t has a gradient besides, dtotal.  workspace: a uint8 device
    tensor of rms_norm_workspace_size bytes, where dweight is given."""
    import torch
    kind = _kind16(total, "total")
    pt, ldt = _rows(total, "total", total.dtype)
    shape, dtype, where = total.shape, total.dtype, total.get_device()
    rows, K = shape
    py, ldy = _matrix(dy, "dy", shape, dtype, where)
    px, ldx = _matrix(dx, "dx", shape, dtype, where)
    pd, ldd = (0, 0) if dtotal is None else _matrix(dtotal, "dtotal", shape, dtype, where)
    pw = 0 if weight is None else _vector(weight, "weight", K, dtype, where)
    pg = 0 if dweight is None else _vector(dweight, "dweight", K, torch.float32, where)
    ps = _vector(rstd, "rstd", rows, torch.float32, where)
    wp, wn = _buffer(workspace, where)
    entry = "rms_norm_backward_" + kind
    args = _pack_norm_grad(rows, K, pt, ldt, pw, ps, py, ldy, pd, ldd, px, ldx, pg, wp, wn)
    _check(getattr(lib(), entry)(args, _stream_handle(stream)), entry)


_ACTS = {"silu": 0, "gelu": 1}


def _act(act):
    if act not in _ACTS:
        raise ValueError(f"act must be one of {sorted(_ACTS)}, got {act!r}")
    return _ACTS[act]


def _factors(g, u, shape, dtype, where):
    """The kept factors' addresses, strides and whether they are float32."""
    import torch
    if g is None and u is None:
        return 0, 0, 0, 0, 0
    if g is None or u is None:
        raise ValueError("g and u are given together")
    kept = torch.float32 if g.dtype is torch.float32 else dtype
    return (*_matrix(g, "g", shape, kept, where), *_matrix(u, "u", shape, kept, where),
            1 if kept is torch.float32 else 0)


def gated_ff_split_size(M: int, N: int, K: int) -> int:
    """Workspace bytes that let gated_ff split its products along K (0: no split)."""
    v = int(lib().sdt_gated_ff_split_size(int(M), int(N), int(K)))
    if v < 0:
        raise SdtError(SDT_ERR_INVALID_ARG, "sdt_gated_ff_split_size")
    return v


def gated_ff(x, gate, up, h, act: str = "silu", g=None, u=None, workspace=None, stream=None) -> None:
    """h [M, N] = a(x . gate^T) * (x . up^T) for x [M, K], gate and up [N, K], float16 or
    bfloat16; a: silu, or gelu in its tanh form.  g and u [M, N], float32 or the type:
    the two products, kept for gated_ff_backward.  workspace: a uint8 device tensor of
    gated_ff_split_size bytes instead of one that the call makes."""
    kind = _kind16(x, "x")
    px, ldx = _rows(x, "x", x.dtype)
    dtype, where = x.dtype, x.get_device()
    (M, K), N = x.shape, gate.shape[0]
    pg, ldg = _matrix(gate, "gate", (N, K), dtype, where)
    pu, ldu = _matrix(up, "up", (N, K), dtype, where)
    ph, ldh = _matrix(h, "h", (M, N), dtype, where)
    entry = "gated_ff_" + kind
    need = _split_size("sdt_gated_ff_split_size", M, N, K) if M > 16 else 0
    wp, wn, _kept = _split_buffer(need, workspace, where, stream)
    args = _pack_gated(M, N, K, px, ldx, pg, ldg, pu, ldu, _act(act), ph, ldh,
                      *_factors(g, u, (M, N), dtype, where), wp, wn)
    _check(getattr(lib(), entry)(args, _stream_handle(stream)), entry)


def gated_ff_workspace_size(M: int, N: int, K: int) -> int:
    """Workspace bytes of gated_ff_backward."""
    v = int(lib().sdt_gated_ff_workspace_size(int(M), int(N), int(K)))
    if v < 0:
        raise SdtError(SDT_ERR_INVALID_ARG, "sdt_gated_ff_workspace_size")
    return v


def gated_ff_backward(x, gate, up, g, u, dh, dx, dgate, dup, workspace, act: str = "silu",
                      stream=None) -> None:
    """dx [M, K], dgate and dup [N, K] from dh [M, N] and the kept g and u (dx, or
    dgate and dup together, None: not wanted).  workspace: a uint8 device tensor of
    gated_ff_workspace_size bytes."""
    kind = _kind16(x, "x")
    px, ldx = _rows(x, "x", x.dtype)
    dtype, where = x.dtype, x.get_device()
    (M, K), N = x.shape, gate.shape[0]
    pg, ldg = _matrix(gate, "gate", (N, K), dtype, where)
    pu, ldu = _matrix(up, "up", (N, K), dtype, where)
    pd, ldd = _matrix(dh, "dh", (M, N), dtype, where)
    if g is None:
        raise ValueError("g and u, as gated_ff kept them, are needed")
    factors = _factors(g, u, (M, N), dtype, where)
    none = (0, 0)
    ox = none if dx is None else _matrix(dx, "dx", (M, K), dtype, where)
    og = none if dgate is None else _matrix(dgate, "dgate", (N, K), dtype, where)
    ou = none if dup is None else _matrix(dup, "dup", (N, K), dtype, where)
    entry = "gated_ff_backward_" + kind
    args = _pack_gated_grad(M, N, K, px, ldx, pg, ldg, pu, ldu, _act(act), *factors, pd, ldd, *ox, *og,
                          *ou, *_buffer(workspace, where))
    _check(getattr(lib(), entry)(args, _stream_handle(stream)), entry)


# ---- products of operands stored along the other dimension ---------------------------------

def gemm_turned_workspace_size(M: int, N: int, K: int) -> int:
    """Workspace bytes that let gemm_*_nn and gemm_*_tn split a C [M, N] along K (0: no split)."""
    v = int(lib().sdt_gemm_turned_workspace_size(int(M), int(N), int(K)))
    if v < 0:
        raise SdtError(SDT_ERR_INVALID_ARG, "sdt_gemm_turned_workspace_size")
    return v


def _gemm_turned(entry, A, B, C, workspace, dtype, stream):
    M, K = A.shape if entry.endswith("nn") else A.shape[::-1]
    N = B.shape[1]
    if B.shape[0] != K or C.shape != (M, N):
        raise ValueError(f"shape mismatch A{tuple(A.shape)} B{tuple(B.shape)} C{tuple(C.shape)}")
    pa, lda = _rows(A, "A", dtype)
    pb, ldb = _rows(B, "B", dtype)
    pc, ldc = _rows(C, "C", dtype)
    where = A.get_device()
    if not (B.get_device() == C.get_device() == where):
        raise _apart(entry, where, B.get_device(), C.get_device())
    _check(getattr(lib(), entry)(M, N, K, pa, lda, pb, ldb, pc, ldc, *_buffer(workspace, where),
                                 _stream_handle(stream)), entry)


def gemm_f16_nn(A, B, C, workspace=None, stream=None) -> None:
    """C[M, N] = A[M, K] . B[K, N], fp32 accumulate, fp16 out (of a product a . b^T, the
    gradient of a: dC . b).  workspace: a uint8 device tensor, see
    gemm_turned_workspace_size."""
    import torch
    _gemm_turned("gemm_f16_nn", A, B, C, workspace, torch.float16, stream)


def gemm_bf16_nn(A, B, C, workspace=None, stream=None) -> None:
    import torch
    _gemm_turned("gemm_bf16_nn", A, B, C, workspace, torch.bfloat16, stream)


def gemm_f16_tn(A, B, C, workspace=None, stream=None) -> None:
    """C[M, N] = A[K, M]^T . B[K, N] (of a product a . b^T, the gradient of b: dC^T . a)."""
    import torch
    _gemm_turned("gemm_f16_tn", A, B, C, workspace, torch.float16, stream)


def gemm_bf16_tn(A, B, C, workspace=None, stream=None) -> None:
    import torch
    _gemm_turned("gemm_bf16_tn", A, B, C, workspace, torch.bfloat16, stream)

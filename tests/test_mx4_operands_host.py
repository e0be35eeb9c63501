"""What the binding of the MX4 and expert entry points refuses before the library
is called (no GPU): memory of the host or of another device, which the C ABI cannot
tell from its own, and a work buffer that is not plain bytes.  Tensors are stand-ins
that know their device; the library only notes that it was called."""
import math

import pytest

from shape_driven_tile_amd import binding as sdt


class Tensor:
    """As much of a tensor as the binding looks at."""

    def __init__(self, *shape, dtype, device=0, stride=None):
        self.shape, self.dtype, self.index = tuple(shape), dtype, device
        if stride is None:
            stride = tuple(math.prod(shape[i + 1:]) for i in range(len(shape)))
            self.dense = True
        else:
            self.dense = False
        self.strides = stride

    is_cuda = property(lambda t: t.index >= 0)

    def get_device(self):
        return self.index

    def stride(self, i=None):
        return self.strides if i is None else self.strides[i]

    def dim(self):
        return len(self.shape)

    def numel(self):
        return math.prod(self.shape)

    def is_contiguous(self):
        return self.dense

    def data_ptr(self):
        return 0x10000


class Library:
    """Notes the calls and accepts them; sizes are the library's own."""

    def __init__(self, real):
        self.real, self.calls = real, []

    def __getattr__(self, name):
        if name.startswith("sdt_"):
            return getattr(self.real, name)
        return lambda *args: self.calls.append(name) or sdt.SDT_OK


@pytest.fixture
def library(monkeypatch):
    fake = Library(sdt.lib())
    monkeypatch.setattr(sdt, "lib", lambda: fake)
    monkeypatch.setattr(sdt, "_stream_handle", lambda s: 0)
    return fake


T, TOPK, E, N, K = 5, 2, 4, 64, 96


def matrix(rows, cols, device, experts=None):
    import torch
    m = sdt.Mx4.empty(rows, cols, experts=experts, device="cpu")
    lead = () if experts is None else (experts,)
    u8 = torch.uint8
    on = sdt.Mx4.__new__(sdt.Mx4)
    for name in sdt.Mx4.__slots__:
        setattr(on, name, getattr(m, name))
    on.q = Tensor(*lead, *m.q.shape[len(lead):], dtype=u8, device=device)
    on.s = Tensor(*lead, *m.s.shape[len(lead):], dtype=u8, device=device)
    on.__init__(on.q, on.s, rows, cols) if device >= 0 else None
    return on


def plan(device):
    """A plan whose memory says that it is on the device."""
    import torch
    placed = type("Placed", (torch.Tensor,), {"get_device": lambda t: device,
                                              "is_cuda": property(lambda t: device >= 0)})
    with pytest.MonkeyPatch.context() as m:
        empty = torch.empty
        m.setattr(torch, "empty", lambda *a, **kw: empty(*a, **kw).as_subclass(placed))
        return sdt.MoePlan.empty(T, TOPK, E, device="cpu")


def entries():
    """Every entry point: its name, a call on tensors of the devices d(i), and how
    many operands it has."""
    import torch
    bf, i32, f32, u8 = torch.bfloat16, torch.int32, torch.float32, torch.uint8
    cfg = sdt.route_cfg(topk=TOPK)
    size = sdt.moe_plan_rows(T, TOPK, E)

    def t(*shape, dtype=bf, d):
        return Tensor(*shape, dtype=dtype, device=d)

    def layer(d):
        def experts():
            return sdt.SdtMx4Experts(0x10000, 64, 64 * 64, 0x10000, 512)
        return sdt.SdtMoeLayer(N, K, experts(), experts(), experts())

    need = sdt.moe_experts_workspace_size(T, TOPK, E, N, K)
    yield "mx4_quantize_bf16", 2, lambda d: sdt.mx4_quantize_bf16(t(T, K, d=d(0)), matrix(T, K, d(1)))
    yield "mx4_quantize_rows_bf16", 3, lambda d: sdt.mx4_quantize_rows_bf16(
        t(T, K, d=d(0)), t(9, dtype=i32, d=d(1)), 1, matrix(9, K, d(2)))
    yield "mx4_dequantize_f32", 2, lambda d: sdt.mx4_dequantize_f32(
        matrix(T, K, d(0)), t(T, K, dtype=f32, d=d(1)))
    yield "mx4_pack_scales", 2, lambda d: sdt.mx4_pack_scales(
        t(T, 3, dtype=u8, d=d(0)), matrix(T, K, d(1)))
    yield "gemm_mx4_bf16", 3, lambda d: sdt.gemm_mx4_bf16(
        matrix(T, K, d(0)), matrix(N, K, d(1)), t(T, N, d=d(2)))
    yield "gemv_mx4_m1_bf16", 3, lambda d: sdt.gemv_mx4_m1_bf16(
        t(K, d=d(0)), matrix(N, K, d(1)), t(N, d=d(2)))
    yield "moe_route_bf16", 4, lambda d: sdt.moe_route(
        t(T, E, d=d(0)), t(T, TOPK, dtype=i32, d=d(1)), t(T, TOPK, dtype=f32, d=d(2)), cfg,
        bias=t(E, dtype=f32, d=d(3)))
    yield "moe_route_backward_bf16", 4, lambda d: sdt.moe_route_backward(
        t(T, E, d=d(0)), t(T, TOPK, dtype=i32, d=d(1)), t(T, TOPK, dtype=f32, d=d(2)),
        t(T, E, d=d(3)), cfg)
    yield "moe_plan", 2, lambda d: sdt.moe_plan(t(T, TOPK, dtype=i32, d=d(0)), plan(d(1)))
    yield "moe_gemm_mx4_bf16", 5, lambda d: sdt.moe_gemm_mx4_bf16(
        plan(d(0)), matrix(size, K, d(1)), matrix(N, K, d(2), E), t(size, N, d=d(3)),
        up=matrix(N, K, d(4), E))
    yield "moe_combine_bf16", 4, lambda d: sdt.moe_combine_bf16(
        plan(d(0)), t(size, N, d=d(1)), t(T, TOPK, dtype=f32, d=d(2)), t(T, N, d=d(3)))
    yield "moe_experts_mx4_bf16", 6, lambda d: sdt.moe_experts_mx4(
        layer(0), t(T, K, d=d(0)), t(T, TOPK, dtype=i32, d=d(1)), t(T, TOPK, dtype=f32, d=d(2)),
        plan(d(3)), t(T, K, d=d(4)), t(need, dtype=u8, d=d(5)))


@pytest.mark.parametrize("name", [e[0] for e in entries()])
def test_operands_on_one_device(name, library):
    _, count, call = next(e for e in entries() if e[0] == name)
    for device in (0, 1):
        call(lambda i: device)
        assert library.calls.pop() == name
    for other in (-1, 1):                        # the host, another device
        for i in range(count):
            with pytest.raises(TypeError):
                call(lambda j: other if j == i else 0)
            assert not library.calls, (other, i)
    with pytest.raises(TypeError):
        call(lambda i: -1)
    assert not library.calls


def test_layer_workspace_is_plain_bytes(library):
    import torch
    need = sdt.moe_experts_workspace_size(T, TOPK, E, N, K)
    experts = sdt.SdtMx4Experts(0x10000, 64, 64 * 64, 0x10000, 512)
    given = sdt.SdtMoeLayer(N, K, experts, experts, experts)

    def call(workspace):
        sdt.moe_experts_mx4(given, Tensor(T, K, dtype=torch.bfloat16),
                            Tensor(T, TOPK, dtype=torch.int32), Tensor(T, TOPK, dtype=torch.float32),
                            plan(0), Tensor(T, K, dtype=torch.bfloat16), workspace)
    call(Tensor(need, dtype=torch.uint8))
    assert library.calls.pop() == "moe_experts_mx4_bf16"
    for bad in (Tensor(need, dtype=torch.float32), Tensor(need, dtype=torch.int8),
                Tensor(need, dtype=torch.uint8, stride=(0,)),     # numel() without the memory
                Tensor(2, need, dtype=torch.uint8, stride=(0, 1))):
        with pytest.raises((TypeError, ValueError)):
            call(bad)
        assert not library.calls


def test_layer_and_plan_are_of_the_same_experts(library):
    """A plan of more experts than the layer's matrices hold would send the products
    past the last one."""
    import torch

    from shape_driven_tile_amd import moe

    def matrices(experts, device=0):
        return (matrix(N, K, device, experts), matrix(N, K, device, experts),
                matrix(K, N, device, experts))

    def call(given, experts=E):
        need = sdt.moe_experts_workspace_size(T, TOPK, 8, N, K)
        sdt.moe_experts_mx4(given, Tensor(T, K, dtype=torch.bfloat16),
                            Tensor(T, TOPK, dtype=torch.int32), Tensor(T, TOPK, dtype=torch.float32),
                            plan(0), Tensor(T, K, dtype=torch.bfloat16),
                            Tensor(need, dtype=torch.uint8))
    call(moe.Mx4Experts(*matrices(E)).layer)
    assert library.calls.pop() == "moe_experts_mx4_bf16"
    for experts in (E - 1, E + 1):
        given = moe.Mx4Experts(*matrices(experts)).layer
        with pytest.raises(ValueError):
            call(given)
    given = moe.Mx4Experts(*matrices(E, 1)).layer
    with pytest.raises(TypeError):
        call(given)
    gate, up, down = matrices(E)
    for mixed in ((matrix(N, K, 1, E), up, down), (gate, matrix(N, K, 1, E), down),
                  (gate, up, matrix(K, N, 1, E))):
        with pytest.raises(TypeError):
            moe.Mx4Experts(*mixed)
    # a struct of addresses: its caller knows what they hold
    experts = sdt.SdtMx4Experts(0x10000, 64, 64 * 64, 0x10000, 512)
    assert not library.calls
    call(sdt.SdtMoeLayer(N, K, experts, experts, experts))
    assert library.calls.pop() == "moe_experts_mx4_bf16"


@pytest.mark.parametrize("missing", ["_cuda_getCurrentRawStream", "_cuda_getDevice"])
def test_stream_handle_without_torchs_own_call(monkeypatch, missing):
    """torch's unnamed call for the current stream's handle may go: the public one
    then serves."""
    import types

    import torch
    monkeypatch.delattr(torch._C, missing)
    monkeypatch.setattr(torch.cuda, "current_stream",
                        lambda *a: types.SimpleNamespace(cuda_stream=77))
    assert sdt._stream_handle(None) == 77
    assert sdt._stream_handle(types.SimpleNamespace(cuda_stream=5)) == 5

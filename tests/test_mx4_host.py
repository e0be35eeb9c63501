"""Host-side tests of the MX4 and expert entry points (no GPU): sizes, and the
refusals of every entry point.  No call here reaches a device: each is refused,
or is a no-op, before the HIP runtime is touched."""
import ctypes

import numpy as np
import pytest

import mx4_reference as ref
from shape_driven_tile_amd import binding as sdt

OK, INVALID, UNSUPPORTED = sdt.SDT_OK, sdt.SDT_ERR_INVALID_ARG, sdt.SDT_ERR_UNSUPPORTED
P = [0x10000 * (i + 1) for i in range(12)]   # fake, aligned addresses: never dereferenced


def test_sizes():
    L = sdt.lib()
    for rows, K in ((0, 0), (1, 1), (64, 256), (65, 257), (8191, 8170), (1, 32), (3, 33)):
        assert L.sdt_mx4_row_bytes(K) == ref.row_bytes(K) == sdt.mx4_row_bytes(K)
        assert L.sdt_mx4_scale_bytes(rows, K) == ref.scale_bytes(rows, K) == \
            sdt.mx4_scale_bytes(rows, K)
    assert L.sdt_mx4_row_bytes(-1) == -1
    assert L.sdt_mx4_scale_bytes(-1, 4) == -1 and L.sdt_mx4_scale_bytes(4, -1) == -1


@pytest.mark.parametrize("T,k,E", [(0, 1, 1), (1, 1, 1), (1, 8, 256), (64, 8, 256), (4096, 6, 64)])
def test_plan_rows_hold_any_choice(T, k, E):
    rows = sdt.moe_plan_rows(T, k, E)
    R = T * k
    assert rows % 64 == 0 and rows >= R
    # the worst spread: one slot to as many experts as there are, the rest to one
    m = min(E, R)
    worst = 64 * max(m - 1, 0) + -(-(R - max(m - 1, 0)) // 64) * 64
    assert rows >= worst
    assert sdt.lib().sdt_moe_plan_rows(-1, 1, 1) == -1
    assert sdt.lib().sdt_moe_plan_rows(1, 0, 1) == -1
    assert sdt.lib().sdt_moe_plan_rows(1, 1, 0) == -1
    assert sdt.lib().sdt_moe_plan_rows(2 ** 31 - 1, 4, 4) == -1


def test_reference_packs_and_reads_back():
    """The reference's own pieces agree (grid values survive quantisation)."""
    rng = np.random.default_rng(0)
    codes = rng.integers(0, 16, (5, 64), dtype=np.uint8)
    codes[:, 0], codes[:, 32] = 7, 7               # every block reaches 6
    scales = rng.integers(100, 150, (5, 2), dtype=np.uint8)
    v = ref.values(codes, scales, 64)
    c2, s2 = ref.quantize(v)
    assert np.array_equal(s2, scales)
    assert np.array_equal(ref.values(c2, s2, 64), v)
    assert np.array_equal(ref.unpack(ref.pack(codes)), codes)


@pytest.mark.parametrize("t", ["f16", "bf16"])
def test_quantize_refusals(t):
    f = getattr(sdt.lib(), f"mx4_quantize_{t}")
    x, q, s = P[:3]
    assert f(0, 64, None, 64, None, 32, None, None) == OK
    assert f(4, 0, None, 0, None, 0, None, None) == OK
    for args, want in [
            ((-1, 64, x, 64, q, 32, s), INVALID), ((4, -1, x, 64, q, 32, s), INVALID),
            ((4, 64, None, 64, q, 32, s), INVALID), ((4, 64, x, 63, q, 32, s), INVALID),
            ((4, 64, x, 64, None, 32, s), INVALID), ((4, 64, x, 64, q, 32, None), INVALID),
            ((4, 64, x, 64, q, 16, s), INVALID), ((4, 64, x, 64, q, 40, s), UNSUPPORTED),
            ((4, 64, x + 1, 64, q, 32, s), UNSUPPORTED), ((4, 64, x, 64, q + 8, 32, s), UNSUPPORTED),
            ((4, 64, x, 64, q, 32, s + 4), UNSUPPORTED),
            ((4, 2 ** 23 + 1, x, 2 ** 24, q, 2 ** 23, s), UNSUPPORTED),
            ((4, 64, x, 64, q, 2 ** 23, s), UNSUPPORTED), ((2 ** 31, 64, x, 64, q, 32, s), UNSUPPORTED)]:
        assert f(*args, None) == want, args
    g = getattr(sdt.lib(), f"mx4_quantize_rows_{t}")
    i = P[3]
    for args, want in [
            ((4, 64, x, 9, 64, None, 2, q, 32, s), INVALID), ((4, 64, x, -1, 64, i, 2, q, 32, s), INVALID),
            ((4, 64, x, 9, 64, i, -1, q, 32, s), INVALID), ((4, 64, x, 9, 63, i, 2, q, 32, s), INVALID),
            ((4, 64, x, 9, 64, i + 2, 2, q, 32, s), UNSUPPORTED), ((0, 64, x, 9, 64, None, 2, q, 32, s), OK)]:
        assert g(*args, None) == want, args


@pytest.mark.parametrize("t", ["f16", "bf16", "f32"])
def test_dequantize_and_pack_refusals(t):
    f = getattr(sdt.lib(), f"mx4_dequantize_{t}")
    y, q, s = P[:3]
    assert f(0, 64, None, 32, None, None, 64, None) == OK
    for args, want in [
            ((-1, 64, q, 32, s, y, 64), INVALID), ((4, 64, None, 32, s, y, 64), INVALID),
            ((4, 64, q, 32, None, y, 64), INVALID), ((4, 64, q, 32, s, None, 64), INVALID),
            ((4, 64, q, 32, s, y, 63), INVALID), ((4, 64, q, 16, s, y, 64), INVALID),
            ((4, 64, q, 32, s, y + 1, 64), UNSUPPORTED), ((4, 64, q + 1, 32, s, y, 64), UNSUPPORTED)]:
        assert f(*args, None) == want, args
    p = sdt.lib().mx4_pack_scales
    for args, want in [((0, 64, None, 2, None), OK), ((-1, 64, q, 2, s), INVALID),
                       ((4, 64, None, 2, s), INVALID), ((4, 64, q, 1, s), INVALID),
                       ((4, 64, q, 2, s + 8), UNSUPPORTED)]:
        assert p(*args, None) == want, args


@pytest.mark.parametrize("t", ["f16", "bf16"])
def test_gemm_and_gemv_refusals(t):
    f = getattr(sdt.lib(), f"gemm_mx4_{t}")
    a, sa, b, sb, c = P[:5]
    good = [4, 8, 64, a, 32, sa, b, 32, sb, c, 8]
    assert f(0, 8, 64, None, 32, None, None, 32, None, None, 8, None) == OK
    assert f(4, 0, 64, None, 32, None, None, 32, None, None, 8, None) == OK
    for at, v, want in [(0, -1, INVALID), (1, -1, INVALID), (2, -1, INVALID), (3, None, INVALID),
                        (4, 16, INVALID), (4, 33, UNSUPPORTED), (5, None, INVALID),
                        (6, None, INVALID), (7, 31, INVALID), (8, None, INVALID),
                        (8, sb + 8, UNSUPPORTED), (9, None, INVALID), (9, c + 2, UNSUPPORTED),
                        (10, 7, INVALID), (10, 12, UNSUPPORTED), (0, 2 ** 31, UNSUPPORTED),
                        (1, 2 ** 31, INVALID)]:
        args = list(good)
        args[at] = v
        assert f(*args, None) == want, (at, v)
    g = getattr(sdt.lib(), f"gemv_mx4_m1_{t}")
    x, y = P[5:7]
    good = [8, 64, x, b, 32, sb, y]
    assert g(0, 64, None, None, 32, None, None, None) == OK
    for at, v, want in [(0, -1, INVALID), (1, -1, INVALID), (2, None, INVALID), (2, x + 1, UNSUPPORTED),
                        (3, None, INVALID), (4, 16, INVALID), (4, 40, UNSUPPORTED), (5, None, INVALID),
                        (6, None, INVALID), (6, y + 1, UNSUPPORTED)]:
        args = list(good)
        args[at] = v
        assert g(*args, None) == want, (at, v)


ROUTE = dict(topk=4, groups=1, groups_kept=1, group_top=1)


@pytest.mark.parametrize("change,E,want", [
    (dict(topk=0), 16, INVALID), (dict(topk=17), 16, INVALID), (dict(topk=65), 128, INVALID),
    (dict(groups=3), 16, INVALID), (dict(groups=4, groups_kept=5), 16, INVALID),
    (dict(groups=4, groups_kept=0), 16, INVALID), (dict(groups=4, groups_kept=1, topk=5), 16, INVALID),
    (dict(group_top=3), 16, INVALID), (dict(groups=16, groups_kept=8, group_top=2), 16, INVALID),
    (dict(scale=float("nan")), 16, INVALID), (dict(scale=float("inf")), 16, INVALID),
    (dict(), 0, INVALID), (dict(), -4, INVALID), (dict(), 1025, UNSUPPORTED),
    (dict(groups=128, groups_kept=64), 512, UNSUPPORTED)])
@pytest.mark.parametrize("t", ["f32", "f16", "bf16"])
def test_route_refusals(change, E, want, t):
    c = sdt.route_cfg(**{**ROUTE, **change})
    f, g = getattr(sdt.lib(), f"moe_route_{t}"), getattr(sdt.lib(), f"moe_route_backward_{t}")
    x, b, i, w, d = P[:5]
    assert f(3, E, x, max(E, 1), b, ctypes.byref(c), i, w, None) == want
    assert g(3, E, x, max(E, 1), ctypes.byref(c), i, w, d, max(E, 1), None) == want
    assert f(0, E, x, max(E, 1), b, ctypes.byref(c), i, w, None) == want    # checked for no tokens too


def test_route_refusals_of_pointers():
    c = sdt.route_cfg(topk=2)
    L = sdt.lib()
    x, b, i, w, d = P[:5]
    r = ctypes.byref(c)
    assert L.moe_route_f32(0, 8, None, 8, None, r, None, None, None) == OK
    for args, want in [((-1, 8, x, 8, b, r, i, w), INVALID), ((3, 8, None, 8, b, r, i, w), INVALID),
                       ((3, 8, x, 7, b, r, i, w), INVALID), ((3, 8, x, 8, b, None, i, w), INVALID),
                       ((3, 8, x, 8, b, r, None, w), INVALID), ((3, 8, x, 8, b, r, i, None), INVALID),
                       ((3, 8, x + 2, 8, b, r, i, w), UNSUPPORTED), ((3, 8, x, 8, b + 1, r, i, w), UNSUPPORTED),
                       ((3, 8, x, 8, b, r, i + 2, w), UNSUPPORTED), ((2 ** 31, 8, x, 8, b, r, i, w), UNSUPPORTED)]:
        assert L.moe_route_f32(*args, None) == want, args
    for args, want in [((3, 8, x, 8, r, i, w, None, 8), INVALID), ((3, 8, x, 8, r, i, w, d, 7), INVALID),
                       ((3, 8, x, 8, r, i, None, d, 8), INVALID), ((3, 8, x, 8, r, i, w, d + 2, 8), UNSUPPORTED)]:
        assert L.moe_route_backward_f32(*args, None) == want, args
    with pytest.raises(ValueError):
        sdt.route_cfg(topk=2, score="relu")


def plan_struct(tokens=4, topk=2, experts=8, **over):
    v = dict(counts=P[0], offsets=P[1], rows=P[2], pos=P[3], tiles=P[4])
    v.update(over)
    return sdt.SdtMoePlan(tokens, topk, experts, v["counts"], v["offsets"], v["rows"], v["pos"],
                          v["tiles"])


def test_plan_gemm_and_combine_refusals():
    L = sdt.lib()
    by = ctypes.byref
    idx = P[5]
    bad = [(plan_struct(tokens=-1), INVALID), (plan_struct(topk=0), INVALID),
           (plan_struct(experts=0), INVALID), (plan_struct(experts=1025), UNSUPPORTED),
           (plan_struct(counts=None), INVALID), (plan_struct(offsets=None), INVALID),
           (plan_struct(rows=None), INVALID), (plan_struct(pos=None), INVALID),
           (plan_struct(tiles=None), INVALID), (plan_struct(rows=P[2] + 2), UNSUPPORTED)]
    assert L.moe_plan(idx, None, None) == INVALID
    assert L.moe_plan(None, by(plan_struct()), None) == INVALID
    assert L.moe_plan(idx + 1, by(plan_struct()), None) == UNSUPPORTED
    a, sa, c, w, y = P[6:11]
    B = sdt.SdtMx4Experts(P[5], 32, 8 * 32, P[11], 512)
    for p, want in bad:
        assert L.moe_plan(idx, by(p), None) == want
        assert L.moe_gemm_mx4_f16(by(p), 8, 64, a, 32, sa, by(B), None, c, 8, None) == want
        assert L.moe_combine_f16(by(p), 8, c, 8, w, y, 8, None) == want
    good = [by(plan_struct()), 8, 64, a, 32, sa, by(B), None, c, 8]
    odd = sdt.SdtMx4Experts(P[5], 32, 8, P[11], 512)
    neg = sdt.SdtMx4Experts(P[5], 32, -16, P[11], 512)
    nul = sdt.SdtMx4Experts(None, 32, 256, P[11], 512)
    for at, v, want in [(1, -1, INVALID), (2, -1, INVALID), (3, None, INVALID), (4, 16, INVALID),
                        (4, 40, UNSUPPORTED), (5, None, INVALID), (6, None, INVALID),
                        (6, by(odd), UNSUPPORTED), (6, by(neg), INVALID), (6, by(nul), INVALID),
                        (7, by(odd), UNSUPPORTED), (7, by(nul), INVALID), (8, None, INVALID),
                        (8, c + 2, UNSUPPORTED), (9, 7, INVALID), (9, 12, UNSUPPORTED)]:
        args = list(good)
        args[at] = v
        for t in ("f16", "bf16"):
            assert getattr(L, f"moe_gemm_mx4_{t}")(*args, None) == want, (at, want)
    none = plan_struct(tokens=0, rows=None, pos=None, tiles=None)
    assert L.moe_gemm_mx4_f16(by(none), 8, 64, None, 32, None, by(B), None, None, 8, None) == OK
    assert L.moe_combine_f16(by(none), 8, None, 8, None, None, 8, None) == OK
    good = [by(plan_struct()), 8, c, 8, w, y, 8]
    for at, v, want in [(1, -1, INVALID), (2, None, INVALID), (2, c + 2, UNSUPPORTED), (3, 7, INVALID),
                        (3, 12, UNSUPPORTED), (4, None, INVALID), (4, w + 1, UNSUPPORTED),
                        (5, None, INVALID), (6, 7, INVALID), (6, 12, UNSUPPORTED)]:
        args = list(good)
        args[at] = v
        assert L.moe_combine_f16(*args, None) == want, (at, want)


def test_layer_refusals():
    L = sdt.lib()
    by = ctypes.byref
    m = sdt.SdtMx4Experts(P[5], 32, 64 * 32, P[6], 512)
    layer = sdt.SdtMoeLayer(64, 64, m, m, m)
    need = sdt.moe_experts_workspace_size(4, 2, 8, 64, 64)
    assert need > 0
    assert L.sdt_moe_experts_workspace_size(-1, 2, 8, 64, 64) == -1
    assert L.sdt_moe_experts_workspace_size(4, 2, 8, 64, 2 ** 24) == -1
    good = [by(layer), P[7], P[8], by(plan_struct()), P[9], 64, P[10], 64, P[11], need]
    broken = sdt.SdtMoeLayer(64, 64, m, sdt.SdtMx4Experts(None, 32, 2048, P[6], 512), m)
    for at, v, want in [(0, None, INVALID), (0, by(broken), INVALID), (1, None, INVALID),
                        (2, None, INVALID), (3, None, INVALID), (3, by(plan_struct(pos=None)), INVALID),
                        (4, None, INVALID), (4, P[9] + 1, UNSUPPORTED), (5, 63, INVALID),
                        (6, None, INVALID), (6, P[10] + 2, UNSUPPORTED), (7, 60, INVALID),
                        (7, 68, UNSUPPORTED), (8, None, INVALID), (8, P[11] + 4, UNSUPPORTED),
                        (9, need - 1, INVALID), (1, P[7] + 1, UNSUPPORTED)]:
        args = list(good)
        args[at] = v
        for t in ("f16", "bf16"):
            assert getattr(L, f"moe_experts_mx4_{t}")(*args, None) == want, (at, want)


def test_binding_refusals():
    """The binding's own checks, on host tensors."""
    import torch
    u8 = torch.uint8
    with pytest.raises(TypeError):
        sdt.Mx4(torch.zeros(4, 32, dtype=torch.int8), torch.zeros(512, dtype=u8), 4, 64)
    with pytest.raises(TypeError):
        sdt.Mx4(torch.zeros(4, 32, dtype=u8), torch.zeros(512, dtype=u8), 4, 64)   # not on a device
    with pytest.raises(TypeError):
        sdt.moe_route(torch.zeros(2, 8, dtype=torch.float64), None, None, sdt.route_cfg(topk=2))
    with pytest.raises(ValueError):
        sdt.moe_plan(torch.zeros(3, 2, dtype=torch.int32), sdt.MoePlan.empty(2, 2, 8, device="cpu"))
    with pytest.raises(sdt.SdtError):
        sdt.MoePlan.empty(-1, 2, 8, device="cpu")

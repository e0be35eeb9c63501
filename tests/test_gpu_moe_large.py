"""Grouped products whose workgroups take several tiles in turn, as the layer of a
prompt does: the loads go on from one expert's tile to another's, some experts have
no rows at all, others many tiles.  Against the 64-bit definitions, and the layer
against its operators bit for bit."""
import numpy as np
import pytest

import mx4_reference as ref
from gpu_helpers import DEV, say
from test_gpu_moe import by_parts, dev, expert_matrices, make_layer
from test_gpu_mx4 import _sdt, _t, device_matrix, product_bound, random_matrix

pytestmark = pytest.mark.gpu


def uneven(T, topk, E, rng):
    """Experts of very different popularity, three of them never chosen, a slot dropped."""
    p = rng.standard_normal((T, E)) + 1.2 * rng.standard_normal(E)
    p[:, [0, E // 2, E - 1]] = -100
    idx = np.argsort(-p, axis=1)[:, :topk].astype(np.int32)
    idx[2, 0] = -1
    return idx


def check_turns(counts, rows, columns, N, nkt, stages):
    """More tiles than two a CU, and k-loops longer than the stages: what sends a
    workgroup from tile to tile."""
    import torch
    cu = torch.cuda.get_device_properties(0).multi_processor_count
    assert (-(-counts // rows)).sum() * -(-N // columns) > 2 * cu
    assert nkt > stages


# (tokens, topk, experts, N, K), rows of a tile, stages: 13 to 64 rows an expert and more
SIZES = [((1100, 4, 128, 520, 1030), 64, 3), ((1500, 6, 100, 648, 801), 128, 2)]


@pytest.mark.parametrize("size,rows,stages", SIZES, ids=["64 rows", "128 rows"])
@pytest.mark.parametrize("gated", [False, True])
def test_moe_gemm_in_turn(size, rows, stages, gated):
    import torch
    sdt = _sdt()
    T, topk, E, N, K = size
    dtype = "bf16" if gated == (rows == 64) else "f16"
    rng = np.random.default_rng(T)
    idx = uneven(T, topk, E, rng)
    plan = sdt.MoePlan.empty(T, topk, E, device=DEV)
    say(f"moe gemm in turn {dtype} gated {gated} {size}")
    sdt.moe_plan(dev(idx), plan)
    counts, offsets, slots, _, _ = ref.plan(idx, E)
    check_turns(counts, rows, 64 if gated else 128, N, -(-K // 256), stages)
    ca, sa = random_matrix(plan.size, K, rng, whole=not gated)
    if gated:
        sa = sa - 6
    A, a = device_matrix(ca, sa, plan.size, K), ref.values(ca, sa, K)
    B, b = expert_matrices(E, N, K, rng, not gated)
    up, u = expert_matrices(E, N, K, rng, False) if gated else (None, None)
    full = torch.full((plan.size, N + 8), float("nan"), dtype=_t(dtype), device=DEV)
    getattr(sdt, f"moe_gemm_mx4_{dtype}")(plan, A, B, full[:, :N], up=up)
    torch.cuda.synchronize()
    got = full.cpu()
    assert bool(torch.isnan(got[:, N:]).all()), "padding of C was written"
    assert bool(torch.isnan(got[torch.from_numpy(slots < 0)]).all()), "a row without a slot was written"
    step = torch.finfo(_t(dtype)).eps / 2
    for e in range(E):
        at = slice(offsets[e], offsets[e] + counts[e])
        if counts[e] == 0:
            continue
        g = a[at] @ b[e].T
        mine = got[at, :N]
        if not gated:
            assert torch.equal(mine, torch.from_numpy(g).float().to(_t(dtype))), e
            continue
        # d(silu(g) u) <= 1.1 |u| dg + |g| du; expf, the division and two products
        # are off by a few steps (2^-21 together, relative)
        v = a[at] @ u[e].T
        want = ref.silu_mul(g, v)
        eg = product_bound(a[at], b[e], np.zeros_like(g), "bf16")
        eu = product_bound(a[at], u[e], np.zeros_like(g), "bf16")
        tol = 1.1 * (np.abs(v) + eu) * eg + (np.abs(g) + eg) * eu + 2.0 ** -21 * np.abs(want)
        tol = tol * (1 + step) + step * np.abs(want) + 2.0 ** -25
        ok = np.abs(mine.double().numpy() - want) <= tol
        if dtype == "f16":
            ok |= np.abs(want) > 65500
        assert ok.all(), (e, np.argwhere(~ok)[:3])


@pytest.mark.parametrize("size,rows,stages", [((850, 4, 100, 808, 801), 64, 3),
                                              ((1500, 6, 100, 520, 801), 128, 2)],
                         ids=["64 rows", "128 rows"])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_layer_in_turn(size, rows, stages, dtype):
    import torch
    T, topk, E, N, K = size
    layer, parts = make_layer(E, N, K, dtype, T)
    rng = np.random.default_rng(N)
    idx = uneven(T, topk, E, rng)
    counts = ref.plan(idx, E)[0]
    check_turns(counts, rows, 64, N, -(-K // 256), stages)      # the gated product
    check_turns(counts, rows, 128, K, -(-N // 256), stages)     # the down product
    x = torch.from_numpy(rng.standard_normal((T, K))).to(_t(dtype)).to(DEV)
    w = dev(rng.random((T, topk)).astype(np.float32))
    say(f"layer in turn {dtype} {size}")
    y = layer(x, dev(idx), w)
    torch.cuda.synchronize()
    want = by_parts(parts, x, dev(idx), w, dtype)
    torch.cuda.synchronize()
    assert torch.isfinite(want).all()
    assert torch.equal(y, want)

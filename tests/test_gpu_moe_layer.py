"""The experts' layer in one call against its operators one by one, bit for bit:
sizes that end inside a block, a scale tile and an output tile, every number of
rows an expert, dropped slots, tokens that hold NaN or infinity, any stride of x."""
import numpy as np
import pytest

from gpu_helpers import DEV, say
from test_gpu_moe import by_parts, choose, dev, make_layer
from test_gpu_mx4 import _sdt, _t

pytestmark = pytest.mark.gpu


def same(got, want):
    import torch
    nan = torch.isnan(want)
    assert torch.equal(torch.isnan(got), nan)
    assert torch.equal(got[~nan], want[~nan])


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("T,topk,E,N,K", [
    (1, 1, 1, 1, 1), (2, 1, 3, 31, 33), (17, 4, 4, 40, 65),          # up to 16 rows an expert, 17
    (40, 2, 4, 33, 65), (64, 4, 4, 100, 256), (100, 1, 3, 64, 520), (90, 3, 5, 257, 129),
    (300, 2, 4, 100, 300), (257, 3, 5, 321, 1000), (1000, 6, 9, 192, 264), (130, 1, 1, 65, 31)])
def test_layer_is_its_parts(T, topk, E, N, K, dtype):
    import torch
    layer, parts = make_layer(E, N, K, dtype, T + N)
    rng = np.random.default_rng(T + K)
    ld = K + 3                                       # rows at any alignment
    x = torch.from_numpy(rng.standard_normal((T, ld))).to(_t(dtype)).to(DEV)[:, :K]
    idx = dev(choose(T, topk, E, rng))
    w = dev(rng.random((T, topk)).astype(np.float32))
    say(f"layer parts {dtype} T {T} topk {topk} E {E} N {N} K {K}")
    y = layer(x, idx, w)
    torch.cuda.synchronize()
    want = by_parts(parts, x, idx, w, dtype)
    torch.cuda.synchronize()
    assert torch.isfinite(want).all()
    assert torch.equal(y, want)


@pytest.mark.parametrize("T", [6, 70, 400])
def test_layer_of_odd_tokens(T):
    """A NaN or an infinity stays in its token; slots outside the experts take no part."""
    import torch
    E, topk, N, K = 4, 2, 96, 160
    layer, parts = make_layer(E, N, K, "bf16", 9)
    rng = np.random.default_rng(T)
    x = torch.from_numpy(rng.standard_normal((T, K))).bfloat16()
    x[1, 40] = float("nan")
    x[T - 2, 0] = float("inf")
    ids = choose(T, topk, E, rng)
    ids[1] = [0, 2]
    ids[T - 2] = [3, 1]
    ids[0] = -1
    ids[2, 1] = E
    w = dev(rng.random((T, topk)).astype(np.float32))
    say(f"layer of odd tokens {T}")
    y = layer(x.to(DEV), dev(ids), w)
    torch.cuda.synchronize()
    same(y, by_parts(parts, x.to(DEV), dev(ids), w, "bf16"))
    torch.cuda.synchronize()
    bad = torch.isnan(y).any(dim=1).cpu().numpy()
    assert list(np.nonzero(bad)[0]) == [1, T - 2]
    assert bool((y[0] == 0).all())


@pytest.mark.parametrize("name,make", [
    ("one expert takes all", lambda T, k, E: np.tile(np.arange(k, dtype=np.int32), (T, 1))),
    ("none", lambda T, k, E: np.full((T, k), -1, dtype=np.int32)),
    ("an expert twice", lambda T, k, E: np.full((T, k), 3, dtype=np.int32))])
def test_layer_of_uneven_choices(name, make):
    import torch
    T, topk, E, N, K = 200, 3, 16, 72, 288
    layer, parts = make_layer(E, N, K, "f16", 4)
    x = torch.randn(T, K, generator=torch.Generator().manual_seed(1)).half().to(DEV)
    idx = dev(make(T, topk, E))
    w = torch.rand(T, topk, generator=torch.Generator().manual_seed(2)).to(DEV)
    say(f"layer: {name}")
    y = layer(x, idx, w)
    torch.cuda.synchronize()
    want = by_parts(parts, x, idx, w, "f16")
    torch.cuda.synchronize()
    assert torch.equal(y, want)


@pytest.mark.parametrize("E,R", [(1, 1), (3, 5), (64, 4097), (7, 33000), (1024, 66001)])
def test_plan_of_ragged_slots(E, R):
    """Numbers of slots that are not whole quads or waves' shares, at any alignment."""
    import torch

    import mx4_reference as ref
    sdt = _sdt()
    rng = np.random.default_rng(R)
    flat = rng.integers(-1, E + 1, R).astype(np.int32)
    full = torch.zeros(R + 1, dtype=torch.int32, device=DEV)
    full[1:] = dev(flat)
    p = sdt.MoePlan.empty(R, 1, E, device=DEV)
    for a in (p.counts, p.offsets, p.rows, p.pos, p.tiles):
        a.fill_(-77)
    say(f"plan of {R} slots, {E} experts")
    sdt.moe_plan(full[1:].view(R, 1), p)
    torch.cuda.synchronize()
    for got, want, what in zip((p.counts, p.offsets, p.rows, p.pos, p.tiles),
                               ref.plan(flat[:, None], E),
                               ("counts", "offsets", "rows", "pos", "tiles")):
        assert np.array_equal(got.cpu().numpy(), want), what


def test_layer_of_many_slots_a_token():
    """More slots a token than the router chooses: the layer takes any plan."""
    import torch
    T, topk, E, N, K = 20, 70, 8, 64, 96
    layer, parts = make_layer(E, N, K, "bf16", 3)
    rng = np.random.default_rng(8)
    x = torch.from_numpy(rng.standard_normal((T, K))).bfloat16().to(DEV)
    idx = dev(rng.integers(-1, E, (T, topk)).astype(np.int32))
    w = dev(rng.random((T, topk)).astype(np.float32))
    say("layer of 70 slots a token")
    y = layer(x, idx, w)
    torch.cuda.synchronize()
    want = by_parts(parts, x, idx, w, "bf16")
    torch.cuda.synchronize()
    assert torch.equal(y, want)


@pytest.mark.parametrize("T,topk,E", [(1, 1, 1), (1, 8, 64), (3, 5, 7), (17, 15, 33), (64, 4, 32),
                                      (4, 64, 1024), (128, 2, 60), (129, 2, 60), (2, 100, 9),
                                      (1, 64, 1024), (16, 4, 33), (64, 1, 1024), (21, 3, 5), (13, 5, 64)])
def test_layer_fills_its_plan(T, topk, E):
    """The plan that the layer leaves is moe_plan's, with few slots and many."""
    import torch

    import mx4_reference as ref
    sdt = _sdt()
    N, K = 32, 288
    layer, parts = make_layer(E, N, K, "bf16", 6)
    rng = np.random.default_rng(T * topk)
    ids = rng.integers(-1, E + 1, (T, topk)).astype(np.int32)
    x = torch.from_numpy(rng.standard_normal((T, K))).bfloat16().to(DEV)
    w = dev(rng.random((T, topk)).astype(np.float32))
    p = sdt.MoePlan.empty(T, topk, E, device=DEV)
    for a in (p.counts, p.offsets, p.rows, p.pos, p.tiles):
        a.fill_(-77)
    say(f"layer's plan T {T} topk {topk} E {E}")
    y = layer(x, dev(ids), w, plan=p)
    torch.cuda.synchronize()
    for got, want, what in zip((p.counts, p.offsets, p.rows, p.pos, p.tiles), ref.plan(ids, E),
                               ("counts", "offsets", "rows", "pos", "tiles")):
        assert np.array_equal(got.cpu().numpy(), want), what
    want = by_parts(parts, x, dev(ids), w, "bf16")
    torch.cuda.synchronize()
    assert torch.equal(y, want)

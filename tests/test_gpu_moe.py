"""Expert routing, its gradient, the plan, the experts' products, their weighted
sum and the whole layer on the GPU, against the 64-bit definitions of
mx4_reference.  Choices and plans are compared exactly."""
import numpy as np
import pytest

import mx4_reference as ref
from gpu_helpers import DEV, say
from test_gpu_mx4 import _sdt, _t, device_matrix, product_bound, random_matrix

pytestmark = pytest.mark.gpu


def dev(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def logits_of(T, E, dtype, seed, spread=2.0):
    import torch
    g = torch.Generator().manual_seed(seed)
    return (spread * torch.randn(T, E, generator=g)).to(_t(dtype))


def run_route(logits, cfg_args, bias=None, pad=0):
    import torch
    sdt = _sdt()
    T, E = logits.shape
    cfg = sdt.route_cfg(**cfg_args)
    full = torch.zeros(T, E + pad, dtype=logits.dtype, device=DEV)
    full[:, :E] = logits.to(DEV)
    idx = torch.full((T, cfg.topk), -9, dtype=torch.int32, device=DEV)
    w = torch.full((T, cfg.topk), float("nan"), device=DEV)
    sdt.moe_route(full[:, :E], idx, w, cfg, bias=None if bias is None else dev(bias))
    torch.cuda.synchronize()
    return idx.cpu().numpy(), w.cpu().numpy()


def check_weights(got, want, E):
    """fp32 scores: an exponential and its argument's rounding, E additions of the
    sum, topk of the renormalisation and a few multiplications, each half a step
    relative to a positive quantity; the logits reach 20, whose difference is
    rounded to 2^-24 * 32."""
    tol = (E + 64 + 64) * 2.0 ** -24
    assert np.all(np.abs(got - want) <= tol * np.abs(want) + 1e-37)


ROUTES = [
    dict(T=1, E=1, topk=1), dict(T=3, E=7, topk=7), dict(T=5, E=64, topk=6),
    dict(T=130, E=65, topk=4, renormalize=False), dict(T=33, E=128, topk=8, scale=2.5),
    dict(T=9, E=256, topk=8, score="sigmoid", bias=True, groups=8, groups_kept=4, group_top=2,
         scale=2.5),
    dict(T=9, E=256, topk=8, score="sigmoid", groups=8, groups_kept=3, group_top=2),
    dict(T=17, E=60, topk=5, score="softmax", bias=True, groups=4, groups_kept=2, group_top=1),
    dict(T=17, E=160, topk=6, score="softmax", groups=8, groups_kept=3, group_top=1,
         renormalize=False, scale=16.0),
    dict(T=4, E=300, topk=16, score="sigmoid"), dict(T=4, E=1024, topk=64, score="softmax", bias=True),
    dict(T=6, E=640, topk=10, score="sigmoid", bias=True, groups=64, groups_kept=64, group_top=2)]


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("i", range(len(ROUTES)))
def test_route(i, dtype):
    r = dict(ROUTES[i])
    T, E, biased = r.pop("T"), r.pop("E"), r.pop("bias", False)
    x = logits_of(T, E, dtype, 100 + i)
    bias = (0.1 * np.random.default_rng(i).standard_normal(E)).astype(np.float32) if biased else None
    say(f"route {i} {dtype} T {T} E {E} {r}")
    idx, w = run_route(x, r, bias, pad=3)
    want_i, want_w = ref.route(x.double().numpy(), bias=bias, **r)
    assert np.array_equal(idx, want_i)
    check_weights(w, want_w, E)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True])
def test_route_ties_and_masks(score, biased):
    """Equal logits (also 0 and -0), rows masked by the type's lowest value, by
    -inf or NaN in part and whole, +inf, and saturated scores."""
    inf = np.inf
    low = np.finfo(np.float32).min
    E = 70
    rng = np.random.default_rng(4)
    rows = [np.zeros(E), np.where(np.arange(E) % 2, -0.0, 0.0), rng.integers(-2, 3, E).astype(float),
            np.full(E, -inf), np.full(E, low), np.where(np.arange(E) == 50, 1.0, -inf),
            np.where(np.arange(E) > 40, np.nan, -1.0), np.full(E, np.nan),
            np.where(np.isin(np.arange(E), [3, 69]), inf, 0.5),
            np.where(np.arange(E) == 9, inf, -inf), np.arange(E) * 2.0 - 60, np.arange(E) * -3.0,
            np.where(np.arange(E) < 66, low, 0.0)]
    x = np.array(rows, dtype=np.float32)
    bias = None
    if biased:
        bias = np.zeros(E, dtype=np.float32)
        bias[5], bias[6], bias[7] = 0.25, -inf, np.nan
    for groups, kept, top in ((1, 1, 1), (7, 3, 1), (7, 3, 2)):
        args = dict(topk=6, score=score, groups=groups, groups_kept=kept, group_top=top)
        say(f"route ties {score} biased {biased} groups {groups} top {top}")
        import torch
        idx, w = run_route(torch.from_numpy(x), args, bias)
        want_i, want_w = ref.route(x, bias=bias, **args)
        assert np.array_equal(idx, want_i), np.argwhere(idx != want_i)[:4]
        assert np.isfinite(w).all()
        check_weights(w, want_w, E)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("i", range(len(ROUTES)))
def test_route_backward(i, dtype):
    import torch
    sdt = _sdt()
    r = dict(ROUTES[i])
    T, E, biased = r.pop("T"), r.pop("E"), r.pop("bias", False)
    x = logits_of(T, E, dtype, 200 + i)
    bias = (0.1 * np.random.default_rng(i).standard_normal(E)).astype(np.float32) if biased else None
    x64 = x.double().numpy()
    idx, _ = ref.route(x64, bias=bias, **r)
    dw = np.random.default_rng(i + 50).standard_normal(idx.shape).astype(np.float32)
    cfg = sdt.route_cfg(**r)
    full = torch.full((T, E + 5), -7.0, dtype=_t(dtype), device=DEV)
    say(f"route backward {i} {dtype}")
    sdt.moe_route_backward(x.to(DEV), dev(idx), dev(dw), full[:, :E], cfg)
    torch.cuda.synchronize()
    assert bool((full[:, E:] == -7.0).all())
    got = full[:, :E].double().cpu().numpy()
    score, renorm, scale = r.get("score", "softmax"), r.get("renormalize", True), r.get("scale", 1.0)
    want = ref.route_backward(x64, idx, dw, score, renorm, scale)
    # fp32 throughout: every term is a product of scores and weights' gradients,
    # the differences between them cancel, so the error is relative to their
    # largest; then half a step of the output
    size = scale * np.abs(dw).max(axis=1, keepdims=True) * 2.0 * \
        (np.ones((T, E)) if renorm else ref.scores(x64, score))
    tol = (E + 128) * 2.0 ** -24 * size + torch.finfo(_t(dtype)).eps / 2 * np.abs(want) + 2.0 ** -25
    assert np.all(np.abs(got - want) <= tol)
    # and against differences of the weights
    h = 1e-5
    for t in range(min(T, 3)):
        for e in list(idx[t][:2]) + [E - 1]:
            hi, lo = x64[t:t + 1].copy(), x64[t:t + 1].copy()
            hi[0, e] += h
            lo[0, e] -= h
            d = (ref.route_weights(hi, idx[t:t + 1], score, renorm, scale) -
                 ref.route_weights(lo, idx[t:t + 1], score, renorm, scale)) / (2 * h)
            diff = float((d[0] * dw[t]).sum())
            assert abs(got[t, e] - diff) <= tol[t, e] + 1e-6 * (1 + abs(diff)) * scale


def test_route_backward_masked():
    """A row with nothing but masks, slots outside the experts, a repeated expert."""
    import torch
    sdt = _sdt()
    x = np.random.default_rng(8).standard_normal((4, 10)).astype(np.float32)
    x[0] = -np.inf
    x[1, 3:] = -np.inf
    idx = np.array([[0, 1, 2], [0, 1, 5], [4, -1, 10], [7, 7, 2]], dtype=np.int32)
    dw = np.random.default_rng(9).standard_normal(idx.shape).astype(np.float32)
    for score in ("softmax", "sigmoid"):
        for renorm in (True, False):
            out = torch.full((4, 10), float("nan"), device=DEV)
            say(f"route backward masked {score} {renorm}")
            sdt.moe_route_backward(dev(x), dev(idx), dev(dw), out,
                                   sdt.route_cfg(topk=3, score=score, renormalize=renorm))
            torch.cuda.synchronize()
            want = ref.route_backward(x, idx, dw, score, renorm, 1.0)
            assert np.all(np.abs(out.double().cpu().numpy() - want) <= 200 * 2.0 ** -24 *
                          np.abs(dw).max(axis=1, keepdims=True) * 2)


# ---- plan ------------------------------------------------------------------------------


def plan_cases():
    rng = np.random.default_rng(6)
    yield "one", np.zeros((1, 1), dtype=np.int32), 1
    yield "all to the last", np.full((300, 1), 15, dtype=np.int32), 16
    yield "few", rng.integers(0, 64, (3, 4)), 64
    yield "uneven", np.minimum(rng.exponential(6, (700, 6)).astype(np.int64), 59), 60
    yield "dropped", rng.integers(-3, 20, (200, 3)), 16
    yield "all dropped", np.full((5, 2), -1), 8
    yield "many experts", rng.integers(0, 1024, (500, 8)), 1024
    yield "exact tiles", np.repeat(np.arange(4), 64).reshape(64, 4), 4
    yield "large", rng.integers(0, 128, (9000, 8)), 128


@pytest.mark.parametrize("case", list(plan_cases()), ids=lambda c: c[0])
def test_plan(case):
    import torch
    sdt = _sdt()
    name, idx, E = case
    idx = np.asarray(idx, dtype=np.int32)
    p = sdt.MoePlan.empty(*idx.shape, E, device=DEV)
    for a in (p.counts, p.offsets, p.rows, p.pos, p.tiles):
        a.fill_(-77)
    say(f"plan {name}")
    sdt.moe_plan(dev(idx), p)
    torch.cuda.synchronize()
    for got, want, what in zip((p.counts, p.offsets, p.rows, p.pos, p.tiles), ref.plan(idx, E),
                               ("counts", "offsets", "rows", "pos", "tiles")):
        assert np.array_equal(got.cpu().numpy(), want), what


def test_plan_of_no_tokens():
    import torch
    sdt = _sdt()
    p = sdt.MoePlan.empty(0, 2, 5, device=DEV)
    p.counts.fill_(9)
    p.offsets.fill_(9)
    say("plan of no tokens")
    sdt.moe_plan(torch.empty(0, 2, dtype=torch.int32, device=DEV), p)
    torch.cuda.synchronize()
    assert bool((p.counts == 0).all()) and bool((p.offsets == 0).all())


# ---- products and the weighted sum -------------------------------------------------------


def expert_matrices(E, rows, K, rng, whole):
    """One matrix per expert on the device, and their values."""
    import torch
    sdt = _sdt()
    parts = [random_matrix(rows, K, rng, whole) for _ in range(E)]
    if not whole:
        parts = [(c, s - 4) for c, s in parts]
    q = torch.from_numpy(np.stack([ref.pack(c) for c, _ in parts])).to(DEV)
    s = torch.from_numpy(np.stack([ref.tile_scales(sc, rows, K) for _, sc in parts])).to(DEV)
    return sdt.Mx4(q, s, rows, K), [ref.values(c, sc, K) for c, sc in parts]


# (tokens, topk, experts, N, K): single tokens, few rows an expert, segments that
# cross and end inside 64- and 128-row tiles, one expert with nearly all
GROUPED = [(1, 1, 1, 1, 1), (1, 4, 16, 40, 64), (5, 2, 8, 100, 300), (64, 4, 8, 72, 513),
           (90, 2, 4, 130, 256), (200, 3, 5, 200, 700), (400, 2, 3, 65, 1030), (700, 1, 2, 264, 288)]


def choose(T, topk, E, rng):
    p = rng.standard_normal((T, E)) + 1.5 * rng.standard_normal(E)
    idx = np.argsort(-p, axis=1)[:, :topk].astype(np.int32)
    if T > 4:
        idx[2, 0] = -1
    return idx


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("T,topk,E,N,K", GROUPED)
def test_moe_gemm(T, topk, E, N, K, gated, dtype):
    import torch
    sdt = _sdt()
    rng = np.random.default_rng(T + N + K)
    idx = choose(T, topk, E, rng)
    plan = sdt.MoePlan.empty(T, topk, E, device=DEV)
    say(f"moe gemm {dtype} gated {gated} T {T} topk {topk} E {E} N {N} K {K}")
    sdt.moe_plan(dev(idx), plan)
    counts, offsets, rows, pos, tiles = ref.plan(idx, E)
    ca, sa = random_matrix(plan.size, K, rng, whole=not gated)
    if gated:
        sa = sa - 6
    A, a = device_matrix(ca, sa, plan.size, K), ref.values(ca, sa, K)
    B, b = expert_matrices(E, N, K, rng, not gated)
    up, u = expert_matrices(E, N, K, rng, False) if gated else (None, None)
    full = torch.full((plan.size, -(-N // 8) * 8 + 8), float("nan"), dtype=_t(dtype), device=DEV)
    getattr(sdt, f"moe_gemm_mx4_{dtype}")(plan, A, B, full[:, :N], up=up)
    torch.cuda.synchronize()
    got = full.cpu()
    assert bool(torch.isnan(got[:, N:]).all()), "padding of C was written"
    assert bool(torch.isnan(got[torch.from_numpy(rows < 0)]).all()), "a row without a slot was written"
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
        v = a[at] @ u[e].T
        want = ref.silu_mul(g, v)
        # d(silu(g) u) <= 1.1 |u| dg + |g| du; expf, the division and two products
        # are off by a few steps (2^-21 together, relative)
        eg = product_bound(a[at], b[e], np.zeros_like(g), "bf16")
        eu = product_bound(a[at], u[e], np.zeros_like(g), "bf16")
        tol = 1.1 * (np.abs(v) + eu) * eg + (np.abs(g) + eg) * eu + 2.0 ** -21 * np.abs(want)
        tol = tol * (1 + step) + step * np.abs(want) + 2.0 ** -25
        ok = np.abs(mine.double().numpy() - want) <= tol
        if dtype == "f16":
            ok |= np.abs(want) > 65500
        assert ok.all(), (e, np.argwhere(~ok)[:3])


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("T,topk,N", [(1, 1, 1), (3, 4, 9), (70, 6, 264), (5, 2, 2049)])
def test_combine(T, topk, N, dtype):
    import torch
    sdt = _sdt()
    rng = np.random.default_rng(T * N)
    E = 8
    idx = rng.integers(-1, E, (T, topk)).astype(np.int32)
    plan = sdt.MoePlan.empty(T, topk, E, device=DEV)
    sdt.moe_plan(dev(idx), plan)
    pos = ref.plan(idx, E)[3].reshape(T, topk)
    ld = -(-N // 8) * 8
    d = torch.full((plan.size, ld), float("nan"), dtype=_t(dtype))
    rows = np.unique(pos[pos >= 0])
    d[rows, :N] = torch.from_numpy(rng.standard_normal((len(rows), N))).to(_t(dtype))
    w = rng.standard_normal((T, topk)).astype(np.float32)
    y = torch.full((T, ld + 8), -7.0, dtype=_t(dtype), device=DEV)
    say(f"combine {dtype} T {T} topk {topk} N {N}")
    getattr(sdt, f"moe_combine_{dtype}")(plan, d.to(DEV)[:, :N], dev(w), y[:, :N])
    torch.cuda.synchronize()
    terms = np.where((pos >= 0)[:, :, None],
                     w.astype(np.float64)[:, :, None] * d[np.maximum(pos, 0), :N].double().numpy(), 0.0)
    want = np.nansum(terms, axis=1)
    tol = topk * 2.0 ** -24 * np.abs(np.nan_to_num(terms)).sum(axis=1)
    tol = tol + torch.finfo(_t(dtype)).eps / 2 * (np.abs(want) + tol) + 2.0 ** -25
    assert np.all(np.abs(y[:, :N].double().cpu().numpy() - want) <= tol)
    assert bool((y[:, N:] == -7.0).all())


# ---- the layer -----------------------------------------------------------------------------


def make_layer(E, N, K, dtype, seed):
    import torch
    from shape_driven_tile_amd import moe
    sdt = _sdt()
    g = torch.Generator(device=DEV).manual_seed(seed)

    def matrices(rows, cols):
        m = sdt.Mx4.empty(rows, cols, experts=E, device=DEV)
        for e in range(E):
            w = (torch.randn(rows, cols, device=DEV, generator=g) * cols ** -0.5).to(_t(dtype))
            getattr(sdt, f"mx4_quantize_{dtype}")(w, sdt.Mx4(m.q[e], m.s[e], rows, cols))
        return m
    gate, up, down = matrices(N, K), matrices(N, K), matrices(K, N)
    return moe.Mx4Experts(gate, up, down), (gate, up, down)


def by_parts(parts, x, idx, w, dtype):
    """The layer through its operators one by one."""
    import torch
    sdt = _sdt()
    gate, up, down = parts
    T, topk = idx.shape
    plan = sdt.MoePlan.empty(T, topk, gate.q.shape[0], device=DEV)
    sdt.moe_plan(idx, plan)
    N, K = gate.rows, gate.K
    xq = sdt.Mx4.empty(plan.size, K, device=DEV)
    getattr(sdt, f"mx4_quantize_rows_{dtype}")(x, plan.rows, topk, xq)
    h = torch.zeros(plan.size, -(-N // 8) * 8, dtype=x.dtype, device=DEV)[:, :N]
    getattr(sdt, f"moe_gemm_mx4_{dtype}")(plan, xq, gate, h, up=up)
    hq = sdt.Mx4.empty(plan.size, N, device=DEV)
    getattr(sdt, f"mx4_quantize_rows_{dtype}")(h, plan.rows, 0, hq)
    d = torch.zeros(plan.size, -(-K // 8) * 8, dtype=x.dtype, device=DEV)[:, :K]
    getattr(sdt, f"moe_gemm_mx4_{dtype}")(plan, hq, down, d)
    y = torch.zeros(T, -(-K // 8) * 8, dtype=x.dtype, device=DEV)[:, :K]
    getattr(sdt, f"moe_combine_{dtype}")(plan, d, w, y)
    return y


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("T,topk,E,N,K", [(1, 2, 4, 64, 128), (9, 3, 8, 136, 200), (150, 2, 4, 96, 257),
                                          (600, 2, 4, 128, 192)])
def test_layer(T, topk, E, N, K, dtype):
    """One call equals the operators one by one, bit for bit, and the layer's
    definition within its roundings; on a side stream, and in a graph."""
    import torch
    sdt = _sdt()
    layer, parts = make_layer(E, N, K, dtype, 5)
    rng = np.random.default_rng(T)
    x = torch.from_numpy(rng.standard_normal((T, -(-K // 8) * 8))).to(_t(dtype)).to(DEV)[:, :K]
    idx = dev(choose(T, topk, E, rng))
    w = dev(rng.random((T, topk)).astype(np.float32))
    say(f"layer {dtype} T {T} topk {topk} E {E} N {N} K {K}")
    y = layer(x, idx, w)
    torch.cuda.synchronize()
    want = by_parts(parts, x, idx, w, dtype)
    torch.cuda.synchronize()
    assert torch.equal(y, want)
    # the definition: the roundings of h and d (half a step of the type each), and
    # where h lies next to a border of the 4-bit grid the neighbouring code
    dense = []
    for m in parts:
        v = torch.empty(E, m.rows, m.K, device=DEV)
        for e in range(E):
            sdt.mx4_dequantize_f32(sdt.Mx4(m.q[e], m.s[e], m.rows, m.K), v[e])
        dense.append(v.double().cpu().numpy())
    xs = ref.values(*ref.quantize(x.double().cpu().numpy()), K)
    ids = idx.cpu().numpy()
    ys = np.zeros((T, K))
    for t in range(T):
        for j in range(topk):
            e = ids[t, j]
            if e < 0:
                continue
            h = ref.silu_mul(dense[0][e] @ xs[t], dense[1][e] @ xs[t])
            h = torch.from_numpy(h).to(_t(dtype)).double().numpy()
            hq = ref.values(*ref.quantize(h[None]), N)[0]
            ys[t] += float(w[t, j]) * (dense[2][e] @ hq)
    got = y.double().cpu().numpy()
    rel = np.linalg.norm(got - ys) / np.linalg.norm(ys)
    assert rel <= 4 * torch.finfo(_t(dtype)).eps, rel
    say("layer on a side stream")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y2 = torch.zeros(T, -(-K // 8) * 8, dtype=x.dtype, device=DEV)[:, :K]
    layer(x, idx, w, out=y2, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(y2, y)
    say("layer in a graph")
    plan = sdt.MoePlan.empty(T, topk, E, device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer(x, idx, w, plan=plan, out=y2)
    for _ in range(3):
        y2.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y2, y)
        assert torch.equal(layer(x, idx, w), y)


def test_example_command():
    from shape_driven_tile_amd import moe
    say("moe example")
    moe.main(["--tokens", "5", "--experts", "8", "--topk", "2", "--hidden", "256", "--inter", "128",
              "--steps", "2"])

"""Routing where scores lie far from 1: sigmoids of very negative logits, softmax
scores far below the row's largest, and sigmoids next to 1, against the definitions
in extended precision (64 fraction bits), with bounds relative to each value."""
import numpy as np
import pytest

import mx4_reference as ref
from gpu_helpers import DEV, say
from test_gpu_moe import dev, run_route
from test_gpu_mx4 import _sdt, _t

pytestmark = pytest.mark.gpu

E, TOPK = 96, 6
STEP = 2.0 ** -24                                # half a step of fp32, relative


def rows(dtype):
    """Finite rows: about a level each, two levels, a wide spread, ordinary ones."""
    import torch
    rng = np.random.default_rng(17)
    levels = [-95.0, -88.5, -104.0, -200.0, -600.0, -20.0, 0.0, 12.0, 16.0, 20.0, 60.0]
    x = [level + 2 * rng.standard_normal(E) for level in levels]
    x += [np.where(np.arange(E) % 20 == 0, -95.0, -130.0) + rng.standard_normal(E),
          np.where(np.arange(E) == 40, 15.0, -95.0) + rng.standard_normal(E),
          -300 * rng.random(E), 40 * rng.standard_normal(E)]
    return torch.from_numpy(np.array(x)).to(_t(dtype))


def scores(x, score):
    """In extended precision, and the complement 1 - score without a subtraction."""
    x = x.astype(np.longdouble)
    if score == "sigmoid":
        return 1 / (1 + np.exp(-x)), 1 / (1 + np.exp(x))
    z = np.exp(x - x.max(axis=1, keepdims=True))
    total = z.sum(axis=1, keepdims=True)
    return z / total, (total - z) / total


def far(x, idx, score, renormalize):
    """A row's largest difference of two logits that an exponential is taken of."""
    chosen = np.take_along_axis(x, idx.astype(np.int64), axis=1)
    top = (chosen if renormalize else x).max(axis=1, keepdims=True)
    d = np.abs(chosen - top).max(axis=1, keepdims=True)
    return d + np.abs(chosen).max(axis=1, keepdims=True) if score == "sigmoid" else d


# The steps of a weight: the difference of two logits (half a step of it, which is as
# much relative to its exponential), the exponentials (a step each), 1 + e, a
# division, topk (or E) additions, a division, the scale; twice, for the sum's terms
# are off by as much as the term itself.
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("renormalize", [True, False])
@pytest.mark.parametrize("score", ["sigmoid", "softmax", "softmax, the largest barred"])
def test_route_far_scores(score, renormalize, dtype):
    x = rows(dtype)
    x64 = x.double().numpy()
    bias = None
    if score.endswith("barred"):                 # all the chosen lie far below the largest
        score = "softmax"
        x64[:, ::3] += 90.0 if dtype != "f32" else 100.0
        import torch
        x = torch.from_numpy(x64).to(_t(dtype))
        x64 = x.double().numpy()
        bias = np.where(np.arange(E) % 3 == 0, -5.0, 0.0).astype(np.float32)
    args = dict(topk=TOPK, score=score, renormalize=renormalize, scale=2.5)
    say(f"route far scores {score} biased {bias is not None} {renormalize} {dtype}")
    idx, w = run_route(x, args, bias)
    want_i, _ = ref.route(x64, bias=bias, **args)
    assert np.array_equal(idx, want_i)
    s, _ = scores(x64, score)
    want = np.take_along_axis(s, idx.astype(np.int64), axis=1)
    if renormalize:
        want = want / want.sum(axis=1, keepdims=True)
    want = (2.5 * want).astype(np.float64)
    steps = 2 * (far(x64, idx, score, renormalize) + (TOPK if renormalize else E) + 12)
    # the smallest scores: fp32 holds them to 2^-149, which the scale multiplies
    tol = steps * STEP * want + 2.5 * 4 * 2.0 ** -149
    bad = np.argwhere(np.abs(w - want) > tol)
    assert bad.size == 0, (bad[:4], w[tuple(bad[0])], want[tuple(bad[0])])
    if renormalize:
        assert np.all(np.abs(w.sum(axis=1, keepdims=True) - 2.5) <= 2.5 * steps * STEP)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_masks_stay_masks(score):
    """Chosen logits of a type's lowest value have a score of zero in 64 bits: zero
    weights, also where nothing else is left to choose."""
    import torch
    for dtype in ("f32", "f16", "bf16"):
        low = torch.finfo(_t(dtype)).min
        x = torch.full((3, 10), low, dtype=_t(dtype))
        x[1, 4] = -95.0
        x[2, 7] = 3.0
        say(f"route masks {score} {dtype}")
        idx, w = run_route(x, dict(topk=4, score=score))
        assert np.isfinite(w).all()
        assert idx[1, 0] == 4 and idx[2, 0] == 7
        assert np.array_equal(w[1:], [[1, 0, 0, 0]] * 2)
        assert np.array_equal(w[0], [0.25] * 4 if score == "softmax" else [0.0] * 4)


def mean_difference(p, ds):
    """ds_j - sum_i p_i ds_i where the p add up to 1, as sum_i p_i (ds_j - ds_i): the
    first form loses to cancellation what lies 2^-64 below ds where a p is next to 1."""
    return (p[:, None, :] * (ds[:, :, None] - ds[:, None, :])).sum(axis=2)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("renormalize", [True, False])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_backward_far_scores(score, renormalize, dtype):
    """Every gradient relative to its own score (and complement).  The differences of
    the weights' gradients are taken from that of the row's largest score, so a
    bound counts |dw_j - dw_top| and their mean, each off by the steps of a score."""
    import torch
    sdt = _sdt()
    x = rows(dtype)
    x64 = x.double().numpy()
    T = x64.shape[0]
    scale = 2.5
    rng = np.random.default_rng(3)
    cases = {"chosen": ref.route(x64, topk=TOPK, score=score)[0],
             "others": np.argsort(x64, axis=1)[:, :TOPK].astype(np.int32)[:, ::-1].copy(),
             "any": np.stack([rng.permutation(E)[:TOPK] for _ in range(T)]).astype(np.int32)}
    for name, idx in cases.items():
        dw = rng.standard_normal(idx.shape).astype(np.float32)
        out = torch.full((T, E), float("nan"), dtype=_t(dtype), device=DEV)
        say(f"route backward far scores {score} {renormalize} {dtype} {name}")
        sdt.moe_route_backward(x.to(DEV), dev(idx), dev(dw), out,
                               sdt.route_cfg(topk=TOPK, score=score, renormalize=renormalize,
                                             scale=scale))
        torch.cuda.synchronize()
        got = out.double().cpu().numpy()
        s, c = scores(x64, score)
        at = np.arange(T)[:, None], idx
        chosen = np.zeros((T, E), dtype=bool)
        chosen[at] = True
        ds = np.zeros((T, E), dtype=np.longdouble)
        ds[at] = dw
        # exponentials of differences as large as these (a softmax of less than 2^-160
        # is left to the bound's last term)
        reach = 2 * (far(x64, idx, score, renormalize) if renormalize or score == "sigmoid"
                     else 160.0)
        if renormalize:
            p = np.where(chosen, s, 0)
            p = p / p.sum(axis=1, keepdims=True)
            pivot = np.take_along_axis(ds, p.argmax(axis=1)[:, None], axis=1)
            off = np.where(chosen, np.abs(ds - pivot), 0)
            want = scale * p * mean_difference(p, ds)
            size = scale * p * (off + (p * off).sum(axis=1, keepdims=True))
            if score == "sigmoid":
                want, size = want * c, size * c
            steps = reach + 2 * TOPK + 32
            assert not np.any(got[~chosen]), "a gradient where nothing was chosen"
        elif score == "sigmoid":
            want = scale * ds * s * c
            size = np.abs(want)
            steps = reach + 32
        else:
            pivot = np.take_along_axis(ds, s.argmax(axis=1)[:, None], axis=1)
            off = np.abs(ds - pivot)
            want = scale * s * mean_difference(s, ds)
            size = scale * s * (off + (s * off).sum(axis=1, keepdims=True))
            steps = reach + 2 * E + 32
        want, size = want.astype(np.float64), size.astype(np.float64)
        # the smallest scores: fp32 holds them to 2^-149, which dw and the scale multiply
        least = scale * np.abs(dw).max() * 8 * 2.0 ** -149
        least = least + {"f32": 2.0 ** -150, "f16": 2.0 ** -25, "bf16": 2.0 ** -134}[dtype]
        tol = steps * STEP * size
        tol = tol + torch.finfo(_t(dtype)).eps / 2 * (np.abs(want) + tol) + least
        bad = np.argwhere(np.abs(got - want) > tol)
        assert bad.size == 0, (name, len(bad), bad[:4], got[tuple(bad[0])], want[tuple(bad[0])])

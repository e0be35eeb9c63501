"""The MX4 format, the products and the experts' operators in 64 bits on the
CPU, written from their definitions in include/sdt.h with numpy alone."""
from __future__ import annotations

import numpy as np

GRID = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=np.float64)
NEG_INF = -np.inf


def row_bytes(K):
    return -(-K // 32) * 16


def scale_bytes(rows, K):
    return -(-rows // 64) * -(-K // 256) * 512


def quantize(x):
    """codes (rows, blocks * 32) and scale bytes (rows, blocks) of float64 x."""
    rows, K = x.shape
    nb = -(-K // 32)
    v = np.zeros((rows, nb * 32))
    v[:, :K] = x
    v = v.reshape(rows, nb, 32)
    special = ~np.isfinite(v).all(axis=2)
    safe = np.where(special[:, :, None], 0.0, v)
    top = np.abs(safe).max(axis=2)
    with np.errstate(divide="ignore"):
        p = np.frexp(top)[1]                      # top = m 2^p, m in [0.5, 1)
    e = np.where(top > 0, np.clip(p - 3 + 127, 0, 254), 0)
    a = np.abs(safe) / np.ldexp(1.0, e - 127)[:, :, None]
    mid = (GRID[1:] + GRID[:-1]) / 2
    low = np.searchsorted(mid, a, side="left")    # a tie stays at the lower code
    high = np.searchsorted(mid, a, side="right")  # a tie goes to the upper code
    code = np.where(low % 2 == 0, low, high)
    code = code + 8 * np.signbit(safe)
    code = np.where(special[:, :, None], 0, code)
    return (code.reshape(rows, nb * 32).astype(np.uint8),
            np.where(special, 255, e).astype(np.uint8))


def pack(codes):
    return codes[:, 0::2] | (codes[:, 1::2] << 4)


def unpack(q):
    out = np.empty((q.shape[0], q.shape[1] * 2), dtype=np.uint8)
    out[:, 0::2] = q & 15
    out[:, 1::2] = q >> 4
    return out


def tile_scales(scales, rows, K):
    """Row-major scale bytes into the tiled layout, byte by byte."""
    nkt = -(-K // 256)
    out = np.zeros(scale_bytes(rows, K), dtype=np.uint8)
    r, b = np.meshgrid(np.arange(rows), np.arange(scales.shape[1]), indexing="ij")
    at = ((r // 64) * nkt + b // 8) * 512 + ((b % 8 // 2) * 16 + r % 16) * 8 + \
        (r % 64 // 16) * 2 + b % 2
    out[at] = scales
    return out


def values(codes, scales, K):
    s = np.ldexp(1.0, scales.astype(np.int64) - 127)
    s = np.where(scales == 255, np.nan, s)
    v = np.where(codes >= 8, -1.0, 1.0) * GRID[codes & 7]
    v = v.reshape(codes.shape[0], -1, 32) * s[:, :, None]
    return v.reshape(codes.shape[0], -1)[:, :K]


def scores(logits, score):
    x = np.where(np.isnan(logits), NEG_INF, logits.astype(np.float64))
    with np.errstate(invalid="ignore", over="ignore", divide="ignore"):
        if score == "sigmoid":
            return np.where(x == NEG_INF, 0.0, 1.0 / (1.0 + np.exp(-x)))
        top = x.max(axis=1, keepdims=True)
        z = np.where(x == NEG_INF, 0.0, np.where(x == top, 1.0, np.exp(x - top)))
        total = z.sum(axis=1, keepdims=True)
        return np.where(total > 0, z / np.where(total > 0, total, 1.0), 0.0)


def route(logits, topk, score="softmax", bias=None, groups=1, groups_kept=1, group_top=1,
          renormalize=True, scale=1.0):
    x = np.where(np.isnan(logits), NEG_INF, logits.astype(np.float64))
    T, E = x.shape
    s = scores(logits, score)
    choice = x if bias is None else s + bias.astype(np.float64)
    choice = np.where(np.isnan(choice), NEG_INF, choice)
    idx = np.empty((T, topk), dtype=np.int32)
    per = E // groups
    for t in range(T):
        allowed = np.ones(E, dtype=bool)
        if groups > 1:
            by = choice[t] if bias is not None or group_top == 1 else s[t]
            best = -np.sort(-by.reshape(groups, per), axis=1)[:, :group_top]
            worth = best[:, 0] if group_top == 1 else best[:, 0] + best[:, 1]
            kept = sorted(range(groups), key=lambda g: (-worth[g], g))[:groups_kept]
            allowed = np.isin(np.arange(E) // per, kept)
        order = sorted(np.nonzero(allowed)[0], key=lambda e: (-choice[t, e], e))
        idx[t] = order[:topk]
    w = np.take_along_axis(s, idx.astype(np.int64), axis=1)
    if renormalize:
        total = w.sum(axis=1, keepdims=True)
        w = np.where(total > 0, w / np.where(total > 0, total, 1.0), 0.0)
    return idx, w * scale


def route_weights(logits, idx, score, renormalize, scale):
    """The weights of a fixed choice (finite differences go through this)."""
    w = np.take_along_axis(scores(logits, score), idx.astype(np.int64), axis=1)
    if renormalize:
        w = w / w.sum(axis=1, keepdims=True)
    return w * scale


def route_backward(logits, idx, dw, score, renormalize, scale):
    """The Jacobian of route_weights, contracted with dw, term by term."""
    s = scores(logits, score)
    T, E = s.shape
    out = np.zeros((T, E))
    for t in range(T):
        sel = idx[t].astype(np.int64)
        ok = (sel >= 0) & (sel < E)
        sel, d = sel[ok], dw[t][ok].astype(np.float64)
        w = s[t, sel]
        total = w.sum()
        ds = np.zeros(E)
        for j in range(len(sel)):
            if renormalize:
                g = 0.0 if total <= 0 else scale / total * (d[j] - (d * w).sum() / total)
            else:
                g = scale * d[j]
            ds[sel[j]] += g
        if score == "sigmoid":
            out[t] = ds * s[t] * (1.0 - s[t])
        else:
            out[t] = s[t] * (ds - (ds * s[t]).sum())
    return out


def plan(idx, E):
    """counts, offsets, rows, pos, tiles of a plan."""
    T, k = idx.shape
    R = T * k
    cap = (R + 63 * min(E, R)) // 64 * 64
    counts = np.zeros(E, dtype=np.int32)
    flat = idx.reshape(-1)
    for v in flat:
        if 0 <= v < E:
            counts[v] += 1
    offsets = np.zeros(E + 1, dtype=np.int32)
    offsets[1:] = np.cumsum((counts + 63) // 64 * 64)
    rows = np.full(cap, -1, dtype=np.int32)
    pos = np.full(R, -1, dtype=np.int32)
    tiles = np.full(cap // 64, -1, dtype=np.int32)
    at = offsets[:-1].copy()
    for i, v in enumerate(flat):
        if 0 <= v < E:
            rows[at[v]] = i
            pos[i] = at[v]
            at[v] += 1
    for e in range(E):
        tiles[offsets[e] // 64:offsets[e + 1] // 64] = e
    return counts, offsets, rows, pos, tiles


def silu_mul(g, u):
    with np.errstate(over="ignore"):
        return g / (1.0 + np.exp(-g)) * u

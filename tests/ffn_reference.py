"""64-bit definitions of the 8-bit, norm and gated feed-forward operators, on
numpy arrays and (where named) torch tensors of float64."""
import math

import numpy as np

E4M3_MAX = 448.0
SMALLEST_SCALE = np.float32(2.0 ** -126)


def e4m3(v):
    """The nearest e4m3 value of each v (ties to even), |v| <= 448 (1 + 2^-5)."""
    v = np.asarray(v, dtype=np.float64)
    _, e = np.frexp(v)
    step = np.ldexp(1.0, np.maximum(e - 1, -6) - 3)
    return np.clip(np.round(v / step) * step, -E4M3_MAX, E4M3_MAX)


def _block(x):
    """Codes and scale of a block of float64 values that fp32 holds."""
    top = np.abs(x).max(initial=0.0)
    if not np.isfinite(top):
        return np.zeros_like(x), np.float32(np.nan)
    scale = max(np.float32(top) / np.float32(E4M3_MAX), SMALLEST_SCALE)
    return e4m3(x.astype(np.float32) / scale), scale


def quantize(x, block):
    """Code values and scales (as the library lays them out) of x [rows, K]."""
    rows, K = x.shape
    kb = -(-K // 128)
    codes = np.zeros((rows, K))
    height = 1 if block == 1 else 128
    scales = np.zeros((-(-rows // height), kb), dtype=np.float32)
    for i in range(scales.shape[0]):
        for j in range(kb):
            at = np.s_[i * height:(i + 1) * height, j * 128:(j + 1) * 128]
            codes[at], scales[i, j] = _block(x[at])
    return codes, np.ascontiguousarray(scales.T) if block == 1 else scales


def scale_map(scales, block, rows, K):
    """The scale of every element."""
    if block == 1:
        return np.repeat(scales.T, 128, axis=1)[:, :K]
    return np.repeat(np.repeat(scales, 128, axis=0)[:rows], 128, axis=1)[:, :K]


def act(g, kind):
    """a(g) and a'(g) of float64 torch tensors."""
    import torch
    if kind == "silu":
        s = torch.sigmoid(g)
        return g * s, s + g * s * (1 - s)
    c = math.sqrt(2 / math.pi)
    t = torch.tanh(c * (g + 0.044715 * g ** 3))
    return 0.5 * g * (1 + t), 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * c * (1 + 3 * 0.044715 * g * g)

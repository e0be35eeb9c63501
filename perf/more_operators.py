"""Measured cases of the feed-forward operators: root-mean-square norms, 8-bit
products with a scale for each block of 128, the gated block of two projections,
and the products that a product's gradients are.

Each case is one pass through an operator as a serving or training program calls
it.  `run` makes the library's calls where `own` is true and computes the same
operators from elementary torch operations, in 32 bits, where it is not.  `exact`
computes them in 64 bits, from the definitions.

The 8-bit format: codes are e4m3 (largest value 448).  Activations have a scale
for each row and block of 128 k, [ceil(K / 128), rows]; weights one for each block
of 128 rows x 128 k, [ceil(rows / 128), ceil(K / 128)].  A block's scale is its
largest magnitude / 448 in 32 bits (at least 2^-126), a code is the 32-bit quotient
x / scale rounded to nearest even.
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"f16": torch.float16, "bf16": torch.bfloat16}
EPS = 1e-6


# ---- the cases -----------------------------------------------------------------


def listed():
    return [
        # one token: the residual is added, the norm leaves in 8 bits for the next product
        {"name": "norm 1 x 4096, 8 bits", "op": "norm", "dtype": "f16", "rows": 1, "K": 4096,
         "backward": False},
        # a prefill batch, rows that end inside a block of 128
        {"name": "norm 4097 x 8170, 8 bits", "op": "norm", "dtype": "bf16", "rows": 4097,
         "K": 8170, "backward": False},
        # a training batch: the norm in 16 bits, then its gradients
        {"name": "norm 8192 x 4096, training", "op": "norm", "dtype": "bf16", "rows": 8192,
         "K": 4096, "backward": True},
        # one token against one projection's 8-bit weights
        {"name": "linear 1 x 12288 x 4096", "op": "linear", "dtype": "f16", "M": 1, "N": 12288,
         "K": 4096},
        # a decode batch
        {"name": "linear 64 x 4096 x 12288", "op": "linear", "dtype": "bf16", "M": 64, "N": 4096,
         "K": 12288},
        # ragged in every direction
        {"name": "linear 3000 x 2000 x 2000", "op": "linear", "dtype": "bf16", "M": 3000,
         "N": 2000, "K": 2000},
        # the library's largest square
        {"name": "linear 8192", "op": "linear", "dtype": "f16", "M": 8192, "N": 8192, "K": 8192},
        # one token through both projections and their product
        {"name": "gated 1 x 12288 x 4096", "op": "gated", "dtype": "f16", "M": 1, "N": 12288,
         "K": 4096, "act": "silu", "backward": False},
        # a small training batch, ragged in every direction
        {"name": "gated 500 x 1400 x 1000, training", "op": "gated", "dtype": "f16", "M": 500,
         "N": 1400, "K": 1000, "act": "gelu", "backward": True},
        # a training batch of a full-sized layer
        {"name": "gated 4096 x 12288 x 4096, training", "op": "gated", "dtype": "bf16",
         "M": 4096, "N": 12288, "K": 4096, "act": "silu", "backward": True},
        # gradients of a small, ragged product
        {"name": "gradients 1023 x 1000 x 520", "op": "gradients", "dtype": "f16", "M": 1023,
         "N": 1000, "K": 520},
        # of a full-sized projection in a training batch
        {"name": "gradients 8192 x 4096 x 4096", "op": "gradients", "dtype": "bf16", "M": 8192,
         "N": 4096, "K": 4096},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "norm", "linear", "linear", "gated", "gated", "gradients"])
    case = {"op": op, "dtype": rng.choice(["f16", "bf16"])}
    if op == "norm":
        case.update(rows=_log_int(rng, 1, 8192), K=_log_int(rng, 65, 8192),
                    backward=rng.random() < 0.5)
    elif op == "linear":
        case.update(M=_log_int(rng, 1, 8192), N=_log_int(rng, 64, 8192), K=_log_int(rng, 64, 8192))
    elif op == "gated":
        backward = rng.random() < 0.5
        case.update(M=_log_int(rng, 32 if backward else 1, 4096), N=_log_int(rng, 64, 12288),
                    K=_log_int(rng, 64, 4096), act=rng.choice(["silu", "gelu"]),
                    backward=backward)
    else:
        case.update(M=_log_int(rng, 32, 8192), N=_log_int(rng, 64, 4096), K=_log_int(rng, 64, 4096))
    return case


# ---- inputs ----------------------------------------------------------------------


def _generator(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _normal(rows, K, dtype, g, std=1.0):
    """Normal rows that start 16-byte aligned."""
    ld = -(-K // 8) * 8
    return (torch.randn(rows, ld, device=DEV, generator=g) * std).to(dtype)[:, :K]


def _activations(rows, K, dtype, g):
    """Rows of a hidden state: normal, with a few channels much larger than the rest."""
    ld = -(-K // 8) * 8
    x = torch.randn(rows, ld, device=DEV, generator=g)
    big = torch.rand(ld, device=DEV, generator=g) < 0.01
    return (x * torch.where(big, 12.0, 1.0)).to(dtype)[:, :K]


def _weights8(rows, K, g):
    """An 8-bit matrix of normal weights: codes (rows start 16-byte aligned) and scales."""
    nb, kb = -(-rows // 128), -(-K // 128)
    w = torch.zeros(nb * 128, kb * 128, device=DEV)
    w[:rows, :K] = torch.randn(rows, K, device=DEV, generator=g) * K ** -0.5
    t = w.view(nb, 128, kb, 128)
    scale = t.abs().amax(dim=(1, 3)) / 448.0
    t = (t / scale[:, None, :, None]).view(nb * 128, kb * 128)
    ld = -(-K // 16) * 16
    return t[:rows, :ld].to(torch.float8_e4m3fn)[:, :K], scale


def prepare(case, seed):
    g = _generator(seed)
    op, dtype = case["op"], TYPES[case["dtype"]]
    s = dict(case)
    if op == "norm":
        rows, K = case["rows"], case["K"]
        s["x"] = _normal(rows, K, dtype, g)
        s["residual"] = _activations(rows, K, dtype, g)
        s["weight"] = (1.0 + 0.1 * torch.randn(K, device=DEV, generator=g)).to(dtype)
        if case["backward"]:
            s["dy"] = _normal(rows, K, dtype, g)
            s["dtotal"] = _normal(rows, K, dtype, g)
    elif op == "linear":
        s["x"] = _activations(case["M"], case["K"], dtype, g)
        s["w"] = _weights8(case["N"], case["K"], g)
    elif op == "gated":
        M, N, K = case["M"], case["N"], case["K"]
        s["x"] = _normal(M, K, dtype, g)
        s["gate"] = _normal(N, K, dtype, g, K ** -0.5)
        s["up"] = _normal(N, K, dtype, g, K ** -0.5)
        if case["backward"]:
            s["dh"] = _normal(M, N, dtype, g)
    else:
        M, N, K = case["M"], case["N"], case["K"]
        s["a"] = _normal(M, K, dtype, g)                     # the product was a . b^T
        s["b"] = _normal(N, K, dtype, g, K ** -0.5)
        s["dc"] = _normal(M, N, dtype, g)
    return s


# ---- the plain form ----------------------------------------------------------------


def _rows8(y):
    """The values that rows y (32 bits) have after 8 bits with a scale for each 128."""
    rows, K = y.shape
    kb = -(-K // 128)
    t = torch.zeros(rows, kb * 128, device=y.device)
    t[:, :K] = y
    t = t.view(rows, kb, 128)
    # by a tensor: a number's reciprocal would be multiplied by, a rounding more
    top = torch.full((), 448.0, device=y.device)
    scale = (t.abs().amax(dim=2, keepdim=True) / top).clamp(min=2.0 ** -126)
    codes = (t / scale).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
    return (codes.float() * scale).view(rows, kb * 128)[:, :K]


def _dense8(w, rows, K):
    codes, scale = w
    full = scale.repeat_interleave(128, dim=0)[:rows].repeat_interleave(128, dim=1)[:, :K]
    return codes.float() * full


def _act(g, act):
    """An activation and its derivative."""
    if act == "silu":
        sig = 1.0 / (1.0 + torch.exp(-g))
        return g * sig, sig * (1.0 + g * (1.0 - sig))
    c = math.sqrt(2.0 / math.pi)
    t = torch.tanh(c * (g + 0.044715 * g * g * g))
    return 0.5 * g * (1.0 + t), \
        0.5 * (1.0 + t) + 0.5 * g * (1.0 - t * t) * c * (1.0 + 3 * 0.044715 * g * g)


def _run_plain(s):
    op, dtype = s["op"], TYPES[s["dtype"]]
    if op == "norm":
        total = (s["x"].float() + s["residual"].float()).to(dtype)
        v = total.float()
        rstd = torch.rsqrt((v * v).mean(dim=1, keepdim=True) + EPS)
        w = s["weight"].float()
        n = v * rstd
        if not s["backward"]:
            return total, _rows8(n * w).to(dtype)
        dy = s["dy"].float()
        dn = dy * w
        dx = rstd * (dn - n * (dn * n).mean(dim=1, keepdim=True)) + s["dtotal"].float()
        return total, (n * w).to(dtype), dx.to(dtype), (dy * n).sum(dim=0)
    if op == "linear":
        x = _rows8(s["x"].float())
        return torch.mm(x, _dense8(s["w"], s["N"], s["K"]).t()).to(dtype)
    if op == "gated":
        x, gate, up = s["x"].float(), s["gate"].float(), s["up"].float()
        g, u = torch.mm(x, gate.t()), torch.mm(x, up.t())
        a, da = _act(g, s["act"])
        h = (a * u).to(dtype)
        if not s["backward"]:
            return h
        dh = s["dh"].float()
        dg, du = dh * u * da, dh * a
        dx = torch.mm(dg, gate) + torch.mm(du, up)
        return h, dx.to(dtype), torch.mm(dg.t(), x).to(dtype), torch.mm(du.t(), x).to(dtype)
    a, b, dc = s["a"].float(), s["b"].float(), s["dc"].float()
    return torch.mm(dc, b).to(dtype), torch.mm(dc.t(), a).to(dtype)


# ---- the library's calls -----------------------------------------------------------


def _like(t):
    """Memory for a result of t's shape and type, rows 16-byte aligned."""
    rows, K = t.shape
    return torch.empty(rows, -(-K // 8) * 8, dtype=t.dtype, device=t.device)[:, :K]


def _work_buffer(s, size):
    """A work buffer, kept with the state as a program keeps it with its layer."""
    if "buffer" not in s:
        s["buffer"] = torch.empty(max(size(), 16), dtype=torch.uint8, device=DEV)
    return s["buffer"]


def _run_own(s):
    from shape_driven_tile_amd import binding as sdt
    op, f16 = s["op"], s["dtype"] == "f16"
    if op == "norm":
        x = s["x"]
        rows, K = x.shape
        total, y = _like(x), _like(x)
        if not s["backward"]:
            q = sdt.Fp8.empty(rows, K, device=x.device)
            sdt.rms_norm(x, s["weight"], q=q, residual=s["residual"], total=total, eps=EPS)
            (sdt.fp8_dequantize_f16 if f16 else sdt.fp8_dequantize_bf16)(q, y)
            return total, y
        rstd = torch.empty(rows, device=x.device)
        sdt.rms_norm(x, s["weight"], y=y, residual=s["residual"], total=total, rstd=rstd, eps=EPS)
        dx, dweight = _like(x), torch.empty(K, device=x.device)
        sdt.rms_norm_backward(total, s["weight"], rstd, s["dy"], dx, dweight,
                              _work_buffer(s, lambda: sdt.rms_norm_workspace_size(rows, K)),
                              dtotal=s["dtotal"])
        return total, y, dx, dweight
    if op == "linear":
        x = s["x"]
        M, N, K = s["M"], s["N"], s["K"]
        a = sdt.Fp8.empty(M, K, device=x.device)
        w = sdt.Fp8(*s["w"], block=128)
        c = torch.empty(M, -(-N // 8) * 8, dtype=x.dtype, device=x.device)[:, :N]
        if f16:
            sdt.fp8_quantize_f16(x, a)
            sdt.gemm_fp8_f16(a, w, c)
        else:
            sdt.fp8_quantize_bf16(x, a)
            sdt.gemm_fp8_bf16(a, w, c)
        return c
    if op == "gated":
        x, gate, up = s["x"], s["gate"], s["up"]
        M, N, K = s["M"], s["N"], s["K"]
        h = torch.empty(M, -(-N // 8) * 8, dtype=x.dtype, device=x.device)[:, :N]
        if not s["backward"]:
            sdt.gated_ff(x, gate, up, h, act=s["act"])
            return h
        # both projections in 32 bits, kept for the gradients
        g, u = (torch.empty(M, -(-N // 8) * 8, device=x.device)[:, :N] for _ in range(2))
        sdt.gated_ff(x, gate, up, h, act=s["act"], g=g, u=u)
        dx, dgate, dup = _like(x), _like(gate), _like(up)
        sdt.gated_ff_backward(x, gate, up, g, u, s["dh"], dx, dgate, dup,
                              _work_buffer(s, lambda: sdt.gated_ff_workspace_size(M, N, K)),
                              act=s["act"])
        return h, dx, dgate, dup
    da, db = _like(s["a"]), _like(s["b"])
    M, N, K = s["M"], s["N"], s["K"]
    buffer = _work_buffer(s, lambda: max(sdt.gemm_turned_workspace_size(M, K, N),
                                         sdt.gemm_turned_workspace_size(N, K, M)))
    if f16:
        sdt.gemm_f16_nn(s["dc"], s["b"], da, buffer)
        sdt.gemm_f16_tn(s["dc"], s["a"], db, buffer)
    else:
        sdt.gemm_bf16_nn(s["dc"], s["b"], da, buffer)
        sdt.gemm_bf16_tn(s["dc"], s["a"], db, buffer)
    return da, db


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ---- what a pass cannot do without ----------------------------------------------------


def work(case):
    op = case["op"]
    if op == "norm":
        n, K = case["rows"] * case["K"], case["K"]
        if case["backward"]:
            # x, residual, dy, dtotal in; total, y, dx out
            return {"bytes": 14 * n + 6 * K, "flops": 16 * n}
        # x, residual in; total, the 8-bit rows and the values they stand for out
        return {"bytes": 9 * n + 4 * case["rows"] * -(-K // 128) + 2 * K, "flops": 8 * n}
    M, N, K = case["M"], case["N"], case["K"]
    if op == "linear":
        blocks = -(-N // 128) * -(-K // 128)
        return {"bytes": 2 * M * K + N * K + 4 * blocks + 2 * M * N, "flops": 2 * M * N * K}
    if op == "gated":
        forward = 2 * (M * K + 2 * N * K + M * N)
        if not case["backward"]:
            return {"bytes": forward, "flops": 4 * M * N * K}
        return {"bytes": forward + 2 * (M * N + M * K + 2 * N * K), "flops": 12 * M * N * K}
    return {"bytes": 2 * (M * N + 2 * M * K + 2 * N * K), "flops": 4 * M * N * K}


# ---- the definitions in 64 bits ---------------------------------------------------------


def _e4m3(v):
    """The nearest values of e4m3 (ties to even): steps of 2^(e - 3), e >= -6."""
    e = torch.frexp(v).exponent.long() - 1
    step = ((e.clamp(min=-6) - 3 + 1023) << 52).view(torch.float64)
    return (torch.round(v / step) * step).clamp(-448.0, 448.0)


def _rows8_exact(y):
    out = torch.empty_like(y)
    for k in range(0, y.shape[1], 128):
        part = y[:, k:k + 128]
        scale = (part.abs().amax(dim=1, keepdim=True) / 448.0).clamp(min=2.0 ** -126)
        scale = scale.float().double()
        # 16-bit values are often next to a tie: the quotient's own rounding decides them
        out[:, k:k + 128] = _e4m3((part / scale).float().double()) * scale
    return out


def exact(case, seed):
    s = prepare(case, seed)
    op, dtype = case["op"], TYPES[case["dtype"]]
    if op == "norm":
        total = (s["x"].double() + s["residual"].double()).to(dtype).double()
        K = case["K"]
        r = 1.0 / torch.sqrt(total.square().sum(dim=1) / K + EPS)
        y = total * r[:, None] * s["weight"].double()
        if not case["backward"]:
            return total, _rows8_exact(y)
        dy, w = s["dy"].double(), s["weight"].double()
        # y_i = t_i r w_i and dr / dt_j = -r^3 t_j / K
        inner = (dy * w * total).sum(dim=1)
        dx = r[:, None] * dy * w - (r ** 3 * inner / K)[:, None] * total + s["dtotal"].double()
        return total, y, dx, torch.mv((dy * total).t(), r)
    if op == "linear":
        x = _rows8_exact(s["x"].double())
        codes, scale = s["w"]
        n = torch.arange(case["N"], device=DEV) // 128
        k = torch.arange(case["K"], device=DEV) // 128
        w = codes.double() * scale.double()[n][:, k]
        return torch.mm(x, w.t())
    if op == "gated":
        x, gate, up = s["x"].double(), s["gate"].double(), s["up"].double()
        g, u = torch.mm(x, gate.t()), torch.mm(x, up.t())
        if case["act"] == "silu":
            sig = torch.sigmoid(g)
            a, da = g * sig, sig + g * sig * (1.0 - sig)
        else:
            c = math.sqrt(2.0 / math.pi)
            z = c * (g + 0.044715 * g ** 3)
            sig = torch.sigmoid(2.0 * z)                     # (1 + tanh z) / 2
            a, da = g * sig, sig + 2.0 * g * sig * (1.0 - sig) * c * (1.0 + 0.134145 * g ** 2)
        if not case["backward"]:
            return a * u
        dh = s["dh"].double()
        both = torch.cat([dh * u * da, dh * a], dim=1)
        dx = torch.mm(both, torch.cat([gate, up], dim=0))
        dw = torch.mm(both.t().contiguous(), x)
        return a * u, dx, dw[:case["N"]], dw[case["N"]:]
    dc = s["dc"].double()
    return torch.mm(dc, s["b"].double()), torch.mm(dc.t().contiguous(), s["a"].double())

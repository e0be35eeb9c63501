"""Measured cases of the MX4 (microscaled 4-bit) and expert-routing operators.

Each case is one pass through an operator as a serving or training program
calls it: quantisation of activations, products of MX4 matrices, the M = 1
product of 16-bit activations with MX4 weights, the router (with its gradient)
and a whole layer of MX4 experts.  `run` makes the library's calls where `own`
is true and computes the same operators from elementary torch operations, in
32 bits (64 where scores are compared), where it is not.  `exact` computes them
in 64 bits, from the definitions.

The MX4 format: blocks of 32 consecutive k of a row share the scale 2^(e - 127)
with e = floor(log2(max |x|)) - 2 + 127, clamped to [0, 254]; an element is x /
scale rounded to the nearest of 0, 0.5, 1, 1.5, 2, 3, 4, 6 (ties to the even
code, saturated), two a byte with the even k in the low nibble.  The scales of
64 rows x 256 k are one tile of 512 bytes: the byte of row r, block b is at
((b / 2) * 16 + r % 16) * 8 + (r / 16) * 2 + b % 2; the tiles of a matrix lie
row by row.
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"f16": torch.float16, "bf16": torch.bfloat16}
LOGITS = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


# ---- the cases -----------------------------------------------------------------


def listed():
    return [
        # one token's activations before a 4-bit product: latency
        {"name": "quantize 1 x 4096", "op": "quantize", "dtype": "f16", "rows": 1, "K": 4096},
        # a prefill batch's activations, with a row that ends inside a block
        {"name": "quantize 8191 x 8170", "op": "quantize", "dtype": "bf16", "rows": 8191,
         "K": 8170},
        # a small decode batch against one projection's weights
        {"name": "gemm 16 x 12288 x 4096", "op": "gemm", "dtype": "f16", "M": 16, "N": 12288,
         "K": 4096},
        # ragged in every direction: partial tiles, a partial last block of k
        {"name": "gemm 3000 x 2000 x 2000", "op": "gemm", "dtype": "bf16", "M": 3000, "N": 2000,
         "K": 2000},
        # the library's largest square
        {"name": "gemm 8192", "op": "gemm", "dtype": "f16", "M": 8192, "N": 8192, "K": 8192},
        # one token against one projection's weights, activations kept in 16 bits
        {"name": "gemv 12288 x 4096", "op": "gemv", "dtype": "f16", "N": 12288, "K": 4096},
        # the same, small and ragged: latency
        {"name": "gemv 4099 x 1000", "op": "gemv", "dtype": "bf16", "N": 4099, "K": 1000},
        # routing four decode tokens: sigmoid scores, a balancing bias, groups
        {"name": "route 4 of 256", "op": "route", "dtype": "f32", "T": 4, "E": 256, "topk": 8,
         "score": "sigmoid", "bias": True, "groups": 8, "groups_kept": 4, "group_top": 2,
         "renormalize": True, "scale": 2.5, "backward": False},
        # a training batch: softmax scores, and the gradient of the logits
        {"name": "route 16384 of 128, training", "op": "route", "dtype": "bf16", "T": 16384,
         "E": 128, "topk": 8, "score": "softmax", "bias": False, "groups": 1, "groups_kept": 1,
         "group_top": 1, "renormalize": True, "scale": 1.0, "backward": True},
        # a layer of experts for one token: the chosen experts' weights stream
        {"name": "experts 1 token", "op": "experts", "dtype": "bf16", "T": 1, "E": 64, "topk": 8,
         "K": 2048, "N": 1024},
        # for a decode batch: nearly every expert has a few rows
        {"name": "experts 64 tokens", "op": "experts", "dtype": "f16", "T": 64, "E": 32, "topk": 4,
         "K": 4096, "N": 1536},
        # for a prefill batch: hundreds of rows an expert
        {"name": "experts 4096 tokens", "op": "experts", "dtype": "bf16", "T": 4096, "E": 64,
         "topk": 6, "K": 2048, "N": 1024},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["quantize", "gemm", "gemm", "gemv", "route", "experts", "experts"])
    dtype = rng.choice(["f16", "bf16"])
    if op == "quantize":
        rows = _log_int(rng, 1, 8191)
        return {"op": op, "dtype": dtype, "rows": rows, "K": _log_int(rng, 33, 8170)}
    if op == "gemm":
        M = _log_int(rng, 2, 8192)
        return {"op": op, "dtype": dtype, "M": M, "N": _log_int(rng, 64, 8192),
                "K": _log_int(rng, 64, 8192)}
    if op == "gemv":
        return {"op": op, "dtype": dtype, "N": _log_int(rng, 64, 12288),
                "K": _log_int(rng, 64, 12288)}
    if op == "route":
        groups = rng.choice([1, 1, 4, 8])
        E = groups * rng.randint(8, 256 // groups)
        kept = 1 if groups == 1 else rng.randint(2, groups)
        bias = rng.random() < 0.5
        backward = rng.random() < 0.5
        return {"op": op, "dtype": rng.choice(["f32", "f16", "bf16"]),
                "T": _log_int(rng, 1, 16384 if E <= 128 else 8192), "E": E,
                # one renormalised weight is constant: its gradient is zero
                "topk": rng.randint(2 if backward else 1, min(8, kept * (E // groups))),
                "score": rng.choice(["softmax", "sigmoid"]), "bias": bias, "groups": groups,
                "groups_kept": kept, "group_top": 1 if groups == 1 else rng.choice([1, 2]),
                "renormalize": rng.random() < 0.7, "scale": rng.choice([1.0, 2.5]),
                "backward": backward}
    E = rng.choice([8, 16, 32, 60, 64])
    return {"op": op, "dtype": dtype, "T": _log_int(rng, 1, 4096), "E": E,
            "topk": rng.randint(1, min(6, E)), "K": _log_int(rng, 256, 2048),
            "N": _log_int(rng, 128, 1024)}


# ---- inputs ----------------------------------------------------------------------


def _generator(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _activations(rows, K, dtype, g):
    """Rows of a hidden state: normal, with a few channels much larger than the
    rest; rows start 16-byte aligned."""
    ld = -(-K // 8) * 8
    x = torch.randn(rows, ld, device=DEV, generator=g)
    big = torch.rand(ld, device=DEV, generator=g) < 0.01
    x = x * torch.where(big, 12.0, 1.0)
    return x.to(dtype)[:, :K]


def _weights(rows, K, g):
    """An MX4 matrix of normal weights, packed."""
    w = torch.randn(rows, K, device=DEV, generator=g) * (K ** -0.5)
    code, scale = _to_mx4(w)
    return _pack(code), _tile_scales(scale, rows)


def _expert_weights(E, rows, K, g):
    parts = [_weights(rows, K, g) for _ in range(E)]
    return torch.stack([p[0] for p in parts]), torch.stack([p[1] for p in parts])


def prepare(case, seed):
    g = _generator(seed)
    op = case["op"]
    s = dict(case)
    if op == "quantize":
        s["x"] = _activations(case["rows"], case["K"], TYPES[case["dtype"]], g)
    elif op == "gemm":
        M, N, K = case["M"], case["N"], case["K"]
        code, scale = _to_mx4(_activations(M, K, torch.float32, g))
        s["a"] = (_pack(code), _tile_scales(scale, M))
        s["b"] = _weights(N, K, g)
        s["c"] = torch.empty(M, -(-N // 8) * 8, dtype=TYPES[case["dtype"]], device=DEV)[:, :N]
    elif op == "gemv":
        N, K = case["N"], case["K"]
        s["x"] = _activations(1, K, TYPES[case["dtype"]], g)[0]
        s["b"] = _weights(N, K, g)
        s["y"] = torch.empty(N, dtype=TYPES[case["dtype"]], device=DEV)
    elif op == "route":
        T, E, k = case["T"], case["E"], case["topk"]
        s["logits"] = (2.0 * torch.randn(T, E, device=DEV, generator=g)).to(LOGITS[case["dtype"]])
        s["bias_v"] = 0.1 * torch.randn(E, device=DEV, generator=g) if case["bias"] else None
        s["dweights"] = torch.randn(T, k, device=DEV, generator=g) if case["backward"] else None
    else:
        T, E, k, K, N = (case[n] for n in ("T", "E", "topk", "K", "N"))
        s["x"] = _activations(T, K, TYPES[case["dtype"]], g)
        # experts of uneven popularity, as a router picks them
        p = torch.randn(T, E, device=DEV, generator=g) + 0.5 * torch.randn(E, device=DEV,
                                                                          generator=g)
        top = torch.topk(p, k, dim=1)
        s["idx"] = top.indices.to(torch.int32)
        s["weights"] = torch.softmax(top.values, dim=1)
        s["gate"] = _expert_weights(E, N, K, g)
        s["up"] = _expert_weights(E, N, K, g)
        s["down"] = _expert_weights(E, K, N, g)
    return s


# ---- the plain form ----------------------------------------------------------------


def _to_mx4(x):
    """Codes (rows, blocks * 32) in 0..15 and scale bytes (rows, blocks) of x."""
    rows, K = x.shape
    nb = -(-K // 32)
    v = torch.zeros(rows, nb * 32, dtype=torch.float32, device=x.device)
    v[:, :K] = x
    v = v.view(rows, nb, 32)
    amax = v.abs().amax(dim=2)
    # floor(log2) from the exponent field; a subnormal amax ends at byte 0 as 0 does
    e = (amax.view(torch.int32) >> 23) - 2
    e = e.clamp(0, 254)
    inv = ((254 - e) << 23).view(torch.float32)            # 2^(127 - e), e <= 252
    a = v.abs() * inv[:, :, None]
    code = (a > 0.25).to(torch.uint8)
    code += a >= 0.75
    code += a > 1.25
    code += a >= 1.75
    code += a > 2.5
    code += a >= 3.5
    code += a > 5.0
    code += torch.signbit(v).to(torch.uint8) * 8
    return code.view(rows, nb * 32), e.to(torch.uint8)


def _pack(code):
    return code[:, 0::2] | (code[:, 1::2] << 4)


def _tile_scales(scale, rows):
    nb = scale.shape[1]
    nr, nk = -(-rows // 64), -(-nb // 8)
    full = torch.zeros(nr * 64, nk * 8, dtype=torch.uint8, device=scale.device)
    full[:rows, :nb] = scale
    # (row tile, 16-row part, row) x (k tile, quarter, block of the quarter)
    t = full.view(nr, 4, 16, nk, 4, 2).permute(0, 3, 4, 2, 1, 5)
    return t.reshape(-1)


def _row_scales(tiled, rows, nb):
    nr, nk = -(-rows // 64), -(-nb // 8)
    t = tiled.view(nr, nk, 4, 16, 4, 2).permute(0, 4, 3, 1, 2, 5)
    return t.reshape(nr * 64, nk * 8)[:rows, :nb]


def _values(code, scale, K, dtype=torch.float32):
    """The values that codes (..., rows, blocks * 32) and scale bytes stand for."""
    grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=dtype, device=code.device)
    grid = torch.cat([grid, -grid])
    s = scale.to(torch.int32)
    f = torch.where(s == 0, 0x00400000, s << 23).view(torch.float32).to(dtype)
    v = grid[code.to(torch.int32)]
    v = v.view(*scale.shape, 32) * f[..., None]
    return v.reshape(*code.shape)[..., :K]


def _unpack(q):
    return torch.stack([q & 15, q >> 4], dim=-1).reshape(*q.shape[:-1], q.shape[-1] * 2)


def _dense(m, rows, K, dtype=torch.float32):
    q, s = m
    return _values(_unpack(q), _row_scales(s, rows, q.shape[1] * 2 // 32), K, dtype)


def _fake_quant(x):
    code, scale = _to_mx4(x.float())
    return _values(code, scale, x.shape[1])


def _scores(case, logits):
    return torch.softmax(logits, dim=1) if case["score"] == "softmax" else torch.sigmoid(logits)


def _select(s):
    """Indices: in 64 bits, so that a tie is a tie; ties go to the lower index."""
    logits, k = s["logits"].double(), s["topk"]
    T, E = logits.shape
    G = s["groups"]
    scored = _scores(s, logits)
    choice = logits if s["bias_v"] is None else scored + s["bias_v"].double()
    if G > 1:
        by = choice if s["group_top"] == 1 or s["bias_v"] is not None else scored
        best = by.view(T, G, E // G).sort(dim=2, descending=True).values
        total = best[:, :, :s["group_top"]].sum(dim=2)
        kept = total.sort(dim=1, descending=True, stable=True).indices[:, :s["groups_kept"]]
        out = torch.ones(T, G, dtype=torch.bool, device=logits.device)
        out.scatter_(1, kept, False)
        choice = choice.masked_fill(out.repeat_interleave(E // G, dim=1), float("-inf"))
    return choice.sort(dim=1, descending=True, stable=True).indices[:, :k]


def _route(s):
    idx = _select(s)
    score = _scores(s, s["logits"].float())
    w = score.gather(1, idx)
    total = w.sum(dim=1, keepdim=True) if s["renormalize"] else None
    weights = w * s["scale"] if total is None else w / total * s["scale"]
    out = [idx.to(torch.int32), weights]
    if s["backward"]:
        dw = s["dweights"]
        if total is None:
            dsel = dw * s["scale"]
        else:
            p = w / total
            dsel = (dw - (dw * p).sum(dim=1, keepdim=True)) * (s["scale"] / total)
        ds = torch.zeros_like(score).scatter(1, idx, dsel)
        if s["score"] == "sigmoid":
            dl = ds * score * (1.0 - score)
        else:
            dl = score * (ds - (ds * score).sum(dim=1, keepdim=True))
        out.append(dl.to(s["logits"].dtype))
    return out


def _plan(idx, E):
    """Slots sorted by expert, every expert's rows padded to a multiple of 64."""
    flat = idx.reshape(-1).long()
    R = flat.numel()
    counts = torch.bincount(flat, minlength=E)
    padded = (counts + 63) // 64 * 64
    ends = torch.cumsum(padded, 0)
    offsets = torch.cat([torch.zeros_like(ends[:1]), ends])
    order = torch.sort(flat, stable=True).indices
    first = torch.cumsum(counts, 0) - counts
    e = flat[order]
    place = offsets[e] + torch.arange(R, device=idx.device) - first[e]
    cap = (R + 63 * min(E, R)) // 64 * 64
    rows = torch.full((cap,), -1, dtype=torch.int64, device=idx.device)
    rows[place] = order
    pos = torch.empty(R, dtype=torch.int64, device=idx.device)
    pos[order] = place
    return [v.to(torch.int32) for v in (counts, offsets, rows, pos)]


def _experts(s, real=torch.float32, quantized=_fake_quant, dense=_dense):
    T, E, k, K, N = (s[n] for n in ("T", "E", "topk", "K", "N"))
    dtype = TYPES[s["dtype"]]
    counts, offsets, rows, pos = _plan(s["idx"], E)
    flat = s["idx"].reshape(-1).long()
    used, which = torch.unique(flat, return_inverse=True)
    U, cap = used.numel(), int(counts.max())
    at = pos.long() - offsets[flat].long()               # a slot's row among its expert's

    def weights(m, r, c):
        q, t = m[0][used], m[1][used]
        nb = q.shape[2] * 2 // 32
        nr, nk = -(-r // 64), -(-nb // 8)
        t = t.view(U, nr, nk, 4, 16, 4, 2).permute(0, 1, 5, 4, 2, 3, 6)
        t = t.reshape(U, nr * 64, nk * 8)[:, :r, :nb]
        return dense(q, t, c)

    def product(rows_in, w):
        a = torch.zeros(U, cap, rows_in.shape[1], dtype=real, device=rows_in.device)
        a[which, at] = rows_in
        return torch.bmm(a, w.transpose(1, 2).contiguous())[which, at]

    slots = torch.arange(T * k, device=flat.device)
    x = quantized(s["x"])[slots // k]
    g = product(x, weights(s["gate"], N, K))
    u = product(x, weights(s["up"], N, K))
    h = (g / (1.0 + torch.exp(-g)) * u).to(dtype)
    d = product(quantized(h), weights(s["down"], K, N)).to(dtype)
    y = (d.to(real).view(T, k, K) * s["weights"].to(real)[:, :, None]).sum(dim=1)
    return counts, offsets, rows, pos, y


def _dense_batch(q, scale, K):
    return _values(_unpack(q), scale, K)


def _run_plain(s):
    op = s["op"]
    if op == "quantize":
        return _fake_quant(s["x"]).to(s["x"].dtype)
    if op == "gemm":
        a = _dense(s["a"], s["M"], s["K"])
        b = _dense(s["b"], s["N"], s["K"])
        return torch.mm(a, b.t()).to(s["c"].dtype)
    if op == "gemv":
        return torch.mv(_dense(s["b"], s["N"], s["K"]), s["x"].float()).to(s["y"].dtype)
    if op == "route":
        return _route(s)
    counts, offsets, rows, pos, y = _experts(s, dense=_dense_batch)
    return counts, offsets, rows, pos, y.to(s["x"].dtype)


# ---- the library's calls -----------------------------------------------------------


def _run_own(s):
    from shape_driven_tile_amd import binding as sdt
    op = s["op"]
    f16 = s["dtype"] == "f16"
    if op == "quantize":
        x = s["x"]
        m = sdt.Mx4.empty(x.shape[0], x.shape[1], device=x.device)
        y = torch.empty_like(x, memory_format=torch.contiguous_format)
        if f16:
            sdt.mx4_quantize_f16(x, m)
            sdt.mx4_dequantize_f16(m, y)
        else:
            sdt.mx4_quantize_bf16(x, m)
            sdt.mx4_dequantize_bf16(m, y)
        return y
    if op == "gemm":
        a = sdt.Mx4(*s["a"], s["M"], s["K"])
        b = sdt.Mx4(*s["b"], s["N"], s["K"])
        (sdt.gemm_mx4_f16 if f16 else sdt.gemm_mx4_bf16)(a, b, s["c"])
        return s["c"]
    if op == "gemv":
        b = sdt.Mx4(*s["b"], s["N"], s["K"])
        (sdt.gemv_mx4_m1_f16 if f16 else sdt.gemv_mx4_m1_bf16)(s["x"], b, s["y"])
        return s["y"]
    if op == "route":
        logits = s["logits"]
        cfg = sdt.route_cfg(topk=s["topk"], score=s["score"], groups=s["groups"],
                            groups_kept=s["groups_kept"], group_top=s["group_top"],
                            renormalize=s["renormalize"], scale=s["scale"])
        idx = torch.empty(s["T"], s["topk"], dtype=torch.int32, device=logits.device)
        weights = torch.empty(s["T"], s["topk"], device=logits.device)
        sdt.moe_route(logits, idx, weights, cfg, bias=s["bias_v"])
        if not s["backward"]:
            return [idx, weights]
        dlogits = torch.empty_like(logits)
        sdt.moe_route_backward(logits, idx, s["dweights"], dlogits, cfg)
        return [idx, weights, dlogits]
    from shape_driven_tile_amd import moe
    if "layer" not in s:     # the layer's weights and work buffers, as a server keeps them
        E, K, N = s["E"], s["K"], s["N"]
        s["layer"] = moe.Mx4Experts(sdt.Mx4(*s["gate"], N, K), sdt.Mx4(*s["up"], N, K),
                                    sdt.Mx4(*s["down"], K, N))
    plan = sdt.MoePlan.empty(s["T"], s["topk"], s["E"], device=s["x"].device)
    y = s["layer"](s["x"], s["idx"], s["weights"], plan=plan)
    return plan.counts, plan.offsets, plan.rows, plan.pos, y


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ---- what a pass cannot do without ----------------------------------------------------


def _mx4_bytes(rows, K):
    nb = -(-K // 32)
    return rows * nb * 17


def work(case):
    op = case["op"]
    if op == "quantize":
        n = case["rows"] * case["K"]
        # the rows in; the 4-bit matrix and the values it stands for out
        return {"bytes": 4 * n + _mx4_bytes(case["rows"], case["K"]), "flops": 2 * n}
    if op == "gemm":
        M, N, K = case["M"], case["N"], case["K"]
        return {"bytes": _mx4_bytes(M, K) + _mx4_bytes(N, K) + 2 * M * N, "flops": 2 * M * N * K}
    if op == "gemv":
        N, K = case["N"], case["K"]
        return {"bytes": _mx4_bytes(N, K) + 2 * (N + K), "flops": 2 * N * K}
    if op == "route":
        T, E, k = case["T"], case["E"], case["topk"]
        z = 4 if case["dtype"] == "f32" else 2
        n = T * E * z + T * k * 8
        if case["backward"]:
            n += T * E * z + T * k * 4
        return {"bytes": n, "flops": T * E * (8 if case["backward"] else 4)}
    T, E, k, K, N = (case[n] for n in ("T", "E", "topk", "K", "N"))
    R = T * k
    # experts that T tokens of k distinct experts each reach, evenly spread
    used = E * (1.0 - (1.0 - k / E) ** T)
    weights = used * (2 * _mx4_bytes(N, K) + _mx4_bytes(K, N))
    return {"bytes": weights + 4 * T * K + 8 * R, "flops": 6 * R * K * N}


# ---- the definitions in 64 bits ---------------------------------------------------------


def _mx4_exact(x):
    """The values x stands for after quantisation, from the definition."""
    rows, K = x.shape
    nb = -(-K // 32)
    v = torch.zeros(rows, nb * 32, dtype=torch.float64, device=x.device)
    v[:, :K] = x.double()
    v = v.view(rows, nb, 32)
    top = v.abs().amax(dim=2, keepdim=True)
    # top = m * 2^p with m in [0.5, 1): floor(log2 top) = p - 1
    p = torch.frexp(top).exponent.long()
    e = torch.where(top > 0, p - 3, -127).clamp(-127, 127)
    scale = ((e + 1023) << 52).view(torch.float64)
    grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=x.device)
    mid = (grid[1:] + grid[:-1]) / 2
    a = (v / scale).abs()
    low = torch.bucketize(a, mid, right=False)     # a tie stays at the lower code
    high = torch.bucketize(a, mid, right=True)     # a tie goes to the upper code
    code = torch.where(low % 2 == 0, low, high)
    return (torch.sign(v) * grid[code] * scale).view(rows, nb * 32)[:, :K]


def _mx4_read(q, tiled, rows, K):
    """The values of a packed matrix, byte by byte from the format's definition."""
    nb, nk = q.shape[-1] // 16, -(-K // 256)
    dev = q.device
    r = torch.arange(rows, device=dev)[:, None]
    b = torch.arange(nb, device=dev)[None, :]
    tile = (r // 64) * nk + b // 8
    rr, bb = r % 64, b % 8
    e = tiled[tile * 512 + ((bb // 2) * 16 + rr % 16) * 8 + (rr // 16) * 2 + bb % 2].long()
    scale = ((e - 127 + 1023) << 52).view(torch.float64)
    k = torch.arange(K, device=dev)
    nibble = (q[:, k // 2].long() >> (4 * (k % 2))) & 15
    mant, exp = nibble & 1, (nibble >> 1) & 3
    mag = torch.where(exp == 0, mant * 0.5, (1 + 0.5 * mant.double()) * (1 << exp) * 0.5)
    mag = torch.where(nibble >= 8, -mag, mag).double()
    return mag * scale[:, k // 32]


def _exact_route(s):
    l = s["logits"].double()
    T, E = l.shape
    if s["score"] == "softmax":
        z = torch.exp(l - l.amax(dim=1, keepdim=True))
        score = z / z.sum(dim=1, keepdim=True)
    else:
        score = 1.0 / (1.0 + torch.exp(-l))
    idx = _select(s)                       # whole numbers: held to the plain form's
    w = torch.gather(score, 1, idx)
    S = w.sum(dim=1, keepdim=True) if s["renormalize"] else torch.ones_like(w[:, :1])
    out = [None, s["scale"] * w / S]
    if s["backward"]:
        # the Jacobian of the chosen weights, contracted with their gradient
        dw = s["dweights"].double() * s["scale"]
        inner = (dw * w).sum(dim=1, keepdim=True) / S if s["renormalize"] else 0.0
        dsel = (dw - inner) / S
        chosen = torch.zeros_like(score).scatter(1, idx, dsel)
        if s["score"] == "sigmoid":
            out.append(chosen * score * (1.0 - score))
        else:
            out.append(chosen * score - score * (dsel * w).sum(dim=1, keepdim=True))
    return out


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "quantize":
        return _mx4_exact(s["x"])
    if op == "gemm":
        a = _mx4_read(*s["a"], s["M"], s["K"])
        b = _mx4_read(*s["b"], s["N"], s["K"])
        return torch.mm(a, b.t())
    if op == "gemv":
        return torch.mv(_mx4_read(*s["b"], s["N"], s["K"]), s["x"].double())
    if op == "route":
        return _exact_route(s)
    T, E, k, K, N = (s[n] for n in ("T", "E", "topk", "K", "N"))
    dtype = TYPES[s["dtype"]]
    flat = s["idx"].reshape(-1).long()
    x = _mx4_exact(s["x"])
    d = torch.zeros(T * k, K, dtype=torch.float64, device=x.device)
    for e in flat.unique().tolist():
        at = (flat == e).nonzero().flatten()
        g = x[at // k] @ _mx4_read(s["gate"][0][e], s["gate"][1][e], N, K).t()
        u = x[at // k] @ _mx4_read(s["up"][0][e], s["up"][1][e], N, K).t()
        h = (g * torch.sigmoid(g) * u).to(dtype)
        o = _mx4_exact(h) @ _mx4_read(s["down"][0][e], s["down"][1][e], K, N).t()
        d[at] = o
    y = (d.view(T, k, K) * s["weights"].double()[:, :, None]).sum(dim=1)
    return None, None, None, None, y

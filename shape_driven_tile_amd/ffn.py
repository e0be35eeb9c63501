"""The feed-forward half of a transformer layer, in training and in serving.

    python -m shape_driven_tile_amd.ffn [--tokens T]

runs a training step of a random layer (norm, gated block, down projection, and their
gradients) and an 8-bit projection as a server runs it (norm to 8 bits, product), through
the library's operators, printing their times.
"""
from __future__ import annotations

from . import binding as sdt


def _rows(n: int, width: int, like, dtype=None):
    """Memory for n rows of `width`, from multiples of 8 elements, as products take them."""
    import torch
    ld = -(-width // 8) * 8
    t = torch.empty(n, ld, dtype=dtype or like.dtype, device=like.device)
    return t if ld == width else t[:, :width]


def _by_type(name: str, t):
    """The entry point of t's type, name_f16 or name_bf16 (and name_f16_nn ...)."""
    head, _, layout = name.partition(":")
    return getattr(sdt, f"{head}_{sdt._kind16(t, 'x')}" + (f"_{layout}" if layout else ""))


def _buffer(size: int, like):
    """A work buffer for calls that follow one another on the current stream; the
    allocator keeps it from others until they are done."""
    import torch
    return torch.empty(max(size, 16), dtype=torch.uint8, device=like.device)


class FeedForward:
    """y = down(a(gate(n)) * up(n)) with n the norm of the residual stream.  norm [K], gate
    and up [N, K], down [K, N], float16 or bfloat16, rows a multiple of 8 elements apart;
    act: silu or gelu.  Calls run on the current stream, make their memory there and keep
    nothing between them."""

    def __init__(self, norm, gate, up, down, act: str = "silu", eps: float = 1e-6):
        N, K = gate.shape
        if tuple(up.shape) != (N, K) or tuple(down.shape) != (K, N) or tuple(norm.shape) != (K,):
            raise ValueError(f"FeedForward: norm {tuple(norm.shape)}, gate {tuple(gate.shape)}, up "
                             f"{tuple(up.shape)} and down {tuple(down.shape)} do not fit one layer")
        sdt._act(act)
        self.norm, self.gate, self.up, self.down, self.act, self.eps = norm, gate, up, down, act, eps
        self.N, self.K = N, K

    def forward(self, x, residual=None, train: bool = True):
        """(y, total, saved) of x [T, K]: total = x + residual, the residual stream that y is
        added to next; saved: what backward needs (None where train is false)."""
        import torch
        T, K = x.shape
        n, h, y = _rows(T, K, x), _rows(T, self.N, x), _rows(T, K, x)
        total = x if residual is None else _rows(T, K, x)
        g = u = rstd = None
        if train:
            # both factors in fp32: rounded to 16 bits they would cost the gradients as
            # much precision as everything after them
            g, u = (_rows(T, self.N, x, torch.float32) for _ in range(2))
            rstd = torch.empty(T, device=x.device)
        sdt.rms_norm(x, self.norm, y=n, residual=residual, total=None if residual is None else total,
                     rstd=rstd, eps=self.eps)
        sdt.gated_ff(n, self.gate, self.up, h, act=self.act, g=g, u=u)
        _by_type("gemm", x)(h, self.down, y)
        return y, total, (total, rstd, n, g, u, h) if train else None

    def backward(self, saved, dy, dtotal=None):
        """(dx, gradients) from dy [T, K] and the gradient dtotal that total has besides;
        dx is the residual's gradient too.  gradients: norm (float32), gate, up, down."""
        import torch
        total, rstd, n, g, u, h = saved
        T, K = total.shape
        N = self.N
        dh, dn, dx = _rows(T, N, dy), _rows(T, K, dy), _rows(T, K, dy)
        dgate, dup, ddown = _rows(N, K, dy), _rows(N, K, dy), _rows(K, N, dy)
        dnorm = torch.empty(K, device=dy.device)
        ws = _buffer(max(sdt.gemm_turned_workspace_size(T, N, K), sdt.gemm_turned_workspace_size(K, N, T),
                         sdt.gated_ff_workspace_size(T, N, K), sdt.rms_norm_workspace_size(T, K)), dy)
        _by_type("gemm:nn", dy)(dy, self.down, dh, ws)
        _by_type("gemm:tn", dy)(dy, h, ddown, ws)
        sdt.gated_ff_backward(n, self.gate, self.up, g, u, dh, dn, dgate, dup, ws, act=self.act)
        sdt.rms_norm_backward(total, self.norm, rstd, dn, dx, dnorm, ws, dtotal=dtotal)
        return dx, {"norm": dnorm, "gate": dgate, "up": dup, "down": ddown}


class Fp8Projection:
    """y = norm(x + residual) . weight^T in 8 bits, as a server runs a layer's projections:
    the norm leaves in 8 bits, so that nothing is rounded to 16 in between.  norm [K] in
    16 bits; weight: an Fp8 of block 128 [N, K], or 16-bit [N, K], which is quantised."""

    def __init__(self, norm, weight, eps: float = 1e-6):
        if not isinstance(weight, sdt.Fp8):
            w16, weight = weight, sdt.Fp8.empty(*weight.shape, block=128, device=weight.device)
            _by_type("fp8_quantize", w16)(w16, weight)
        if weight.block != 128 or tuple(norm.shape) != (weight.K,):
            raise ValueError(f"Fp8Projection: norm {tuple(norm.shape)} and a weight ({weight.rows}, "
                             f"{weight.K}) of block {weight.block} do not fit")
        self.norm, self.weight, self.eps = norm, weight, eps

    def __call__(self, x, residual=None):
        """(y, total) of x [T, K]; total = x + residual."""
        T, K = x.shape
        q, y = sdt.Fp8.empty(T, K, device=x.device), _rows(T, self.weight.rows, x)
        total = x if residual is None else _rows(T, K, x)
        sdt.rms_norm(x, self.norm, q=q, residual=residual, total=None if residual is None else total,
                     eps=self.eps)
        _by_type("gemm_fp8", x)(q, self.weight, y)
        return y, total


def main(argv=None) -> None:
    import argparse

    import torch
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--tokens", type=int, default=2048)
    ap.add_argument("--hidden", type=int, default=2048)
    ap.add_argument("--inter", type=int, default=4096)
    ap.add_argument("--act", choices=sorted(sdt._ACTS), default="silu")
    ap.add_argument("--steps", type=int, default=20)
    a = ap.parse_args(argv)
    dev = torch.device("cuda:0")
    g = torch.Generator(device=dev)
    g.manual_seed(0)

    def normal(rows, width, std=1.0):
        t = _rows(rows, width, torch.empty(0, dtype=torch.bfloat16, device=dev))
        t.copy_(torch.randn(rows, width, device=dev, generator=g) * std)
        return t

    def timed(step):
        step()
        torch.cuda.synchronize()
        begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        begin.record()
        for _ in range(a.steps):
            step()
        end.record()
        torch.cuda.synchronize()
        return begin.elapsed_time(end) / a.steps * 1e3

    K, N, T = a.hidden, a.inter, a.tokens
    norm = torch.ones(K, dtype=torch.bfloat16, device=dev)
    layer = FeedForward(norm, normal(N, K, K ** -0.5), normal(N, K, K ** -0.5), normal(K, N, N ** -0.5),
                        act=a.act)
    x, residual, dy = normal(T, K), normal(T, K), normal(T, K)
    got = {}

    def train():
        y, total, saved = layer.forward(x, residual)
        got["y"] = y
        got["dx"], got["gradients"] = layer.backward(saved, dy, dtotal=dy)

    us = timed(train)
    print(f"{T} tokens, {K} -> {N}: a training step {us:.1f} us ({18 * T * K * N / us / 1e6:.0f} TFLOP/s), "
          f"|y| {got['y'].float().abs().mean().item():.3g}, |dx| {got['dx'].float().abs().mean().item():.3g}, "
          f"|dgate| {got['gradients']['gate'].float().abs().mean().item():.3g}", flush=True)
    project = Fp8Projection(norm, layer.gate)
    us = timed(lambda: got.update(q=project(x, residual)[0]))
    print(f"8-bit projection {us:.1f} us ({2 * T * K * N / us / 1e6:.0f} TFLOP/s), "
          f"|y| {got['q'].float().abs().mean().item():.3g}", flush=True)


if __name__ == "__main__":
    main()

"""A layer of gated experts with MX4 weights, as a server runs it.

    python -m shape_driven_tile_amd.moe [--tokens T]

quantises random weights, routes random tokens (by a 16-bit product: ranking experts
is where a 4-bit one's error shows first) and runs the layer through the library's
operators (route, plan, quantise, the experts' products, combine), printing its time.
"""
from __future__ import annotations

from . import binding as sdt


class Mx4Experts:
    """The experts' weights (gate and up: N x K, down: K x N, one matrix per
    expert) and the layer's work buffer, which grows to the largest call's need
    and is used by one stream at a time: work of the layer on another stream is
    ordered after it by the caller.  What a call allocates it allocates on the
    stream that runs it, and the buffer is recorded on every stream that uses it,
    so the allocator gives none of it away before that work is done.  A buffer
    that a graph was captured with is kept as long as the layer, also when a
    larger one replaces it for later calls."""

    def __init__(self, gate: sdt.Mx4, up: sdt.Mx4, down: sdt.Mx4):
        if gate.q.dim() != 3 or (up.rows, up.K) != (gate.rows, gate.K) or \
                (down.rows, down.K) != (gate.K, gate.rows):
            raise ValueError(f"Mx4Experts: gate ({gate.rows}, {gate.K}), up ({up.rows}, {up.K}) and "
                             f"down ({down.rows}, {down.K}) do not fit one layer")
        self.experts = gate.q.shape[0]
        self.N, self.K = gate.rows, gate.K
        self.weights = (gate, up, down)          # kept alive: the struct holds their addresses
        self.layer = sdt.SdtMoeLayer(self.N, self.K, gate._experts(self.experts, "gate"),
                                     up._experts(self.experts, "up"),
                                     down._experts(self.experts, "down"))
        self._workspace = None
        self._captured = False                   # a graph holds the buffer's address
        self._kept = []                          # replaced buffers that graphs hold
        self._streams = set()                    # that the allocator knows to use the buffer
        self._holds = None                       # the sizes and stream it was last checked for

    def workspace(self, tokens: int, topk: int):
        """The buffer for a call on the current stream."""
        import torch
        handle = sdt._stream_handle(None)
        if self._holds != (tokens, topk, handle):
            self._hold(tokens, topk, handle)
        # (the default stream, 0, cannot be captured)
        if handle != 0 and not self._captured and torch.cuda.is_current_stream_capturing():
            self._captured = True
        return self._workspace

    def _hold(self, tokens: int, topk: int, handle: int) -> None:
        import torch
        need = sdt.moe_experts_workspace_size(tokens, topk, self.experts, self.N, self.K)
        if self._workspace is None or self._workspace.numel() < need:
            if self._captured:
                self._kept.append(self._workspace)
                self._captured = False
            self._workspace = torch.empty(max(need, 16), dtype=torch.uint8,
                                          device=self.weights[0].q.device)
            self._streams = {handle}
        elif handle not in self._streams:
            self._workspace.record_stream(torch.cuda.current_stream())
            self._streams.add(handle)
        self._holds = (tokens, topk, handle)

    def __call__(self, x, idx, weights, plan: sdt.MoePlan | None = None, out=None, stream=None):
        """y [T, K] of x [T, K] (float16 or bfloat16), the experts idx [T, topk]
        (int32) of each token and their weights [T, topk] (float32).  `plan`: a
        MoePlan of these sizes to fill (made here if absent); `out`: y's memory,
        rows a multiple of 8 elements apart; `stream`: instead of the current
        one, ordered with it by the caller."""
        import torch
        if stream is not None and stream.cuda_stream != sdt._stream_handle(None):
            current = torch.cuda.current_stream()
            with torch.cuda.stream(stream):
                y = self(x, idx, weights, plan, out)
            if out is None:
                y.record_stream(current)         # where the caller goes on with it
            return y
        T, topk = idx.shape
        if plan is None:
            plan = sdt.MoePlan.empty(T, topk, self.experts, device=x.device)
        elif (plan.tokens, plan.topk, plan.experts) != (T, topk, self.experts):
            raise ValueError(f"plan is of {plan.tokens} tokens, {plan.topk} of {plan.experts} experts")
        if out is None:
            ld = -(-self.K // 8) * 8
            out = torch.empty(T, ld, dtype=x.dtype, device=x.device)
            if ld != self.K:
                out = out[:, :self.K]
        sdt.moe_experts_mx4(self.layer, x, idx, weights, plan, out, self.workspace(T, topk))
        return out


def main(argv=None) -> None:
    import argparse

    import torch
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--tokens", type=int, default=64)
    ap.add_argument("--experts", type=int, default=32)
    ap.add_argument("--topk", type=int, default=4)
    ap.add_argument("--hidden", type=int, default=2048)
    ap.add_argument("--inter", type=int, default=1024)
    ap.add_argument("--steps", type=int, default=50)
    a = ap.parse_args(argv)
    dev = torch.device("cuda:0")
    g = torch.Generator(device=dev)
    g.manual_seed(0)

    def matrices(rows, K):
        m = sdt.Mx4.empty(rows, K, experts=a.experts, device=dev)
        for e in range(a.experts):
            w = torch.randn(rows, K, device=dev, generator=g) * K ** -0.5
            sdt.mx4_quantize_bf16(w.bfloat16(), sdt.Mx4(m.q[e], m.s[e], rows, K))
        return m

    def rows(n, width):                          # from multiples of 8 elements, as products take them
        return torch.empty(n, -(-width // 8) * 8, dtype=torch.bfloat16, device=dev)[:, :width]

    layer = Mx4Experts(matrices(a.inter, a.hidden), matrices(a.inter, a.hidden),
                       matrices(a.hidden, a.inter))
    x, router = rows(a.tokens, a.hidden), rows(a.experts, a.hidden)
    x.copy_(torch.randn(x.shape, device=dev, generator=g))
    router.copy_(torch.randn(router.shape, device=dev, generator=g) * a.hidden ** -0.5)
    logits = rows(a.tokens, a.experts)
    cfg = sdt.route_cfg(topk=a.topk)
    idx = torch.empty(a.tokens, a.topk, dtype=torch.int32, device=dev)
    weights = torch.empty(a.tokens, a.topk, device=dev)
    plan = sdt.MoePlan.empty(a.tokens, a.topk, a.experts, device=dev)
    y = rows(a.tokens, a.hidden)

    def step():
        sdt.gemm_bf16(x, router, logits)
        sdt.moe_route(logits, idx, weights, cfg)
        layer(x, idx, weights, plan=plan, out=y)

    step()
    torch.cuda.synchronize()
    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    begin.record()
    for _ in range(a.steps):
        step()
    end.record()
    torch.cuda.synchronize()
    print(f"{a.tokens} tokens, {a.topk} of {a.experts} experts, {a.hidden} -> {a.inter}: "
          f"{begin.elapsed_time(end) / a.steps * 1e3:.1f} us a step, "
          f"rows per expert {plan.counts.min().item()}..{plan.counts.max().item()}, "
          f"|y| {y.float().abs().mean().item():.3g}", flush=True)


if __name__ == "__main__":
    main()

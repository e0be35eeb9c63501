"""The feed-forward layer built from the library's operators: its outputs and gradients
against autograd of the same layer in 64 bits, the 8-bit projection against its
definition, the example command.

Bounds: every tensor that the layer keeps in 16 bits (t, n, h, dy's products dh, dg and
du, dn) is rounded by at most half a step of its size.  A norm of such errors over a
tensor is at most the sum of their relative sizes through each product, as each is a
linear map of independent terms: six roundings at most lie on a path from an input to an
output, and none of the maps between them (norm, products with unit-variance weights,
activations with slopes below 1.13) raises a relative error by more than 2."""
import pytest

import ffn_reference as ref
from gpu_helpers import DEV, say

pytestmark = pytest.mark.gpu


def _off(got, want):
    return ((got.double() - want).norm() / want.norm()).item()


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("T, K, N", [(3, 64, 96), (200, 136, 300), (700, 512, 1024)])
def test_layer_against_autograd(dtype, act, T, K, N):
    import torch
    from shape_driven_tile_amd import ffn
    say(f"layer {dtype} {act} {T} {K} {N}")
    t = {"f16": torch.float16, "bf16": torch.bfloat16}[dtype]
    g = torch.Generator(device=DEV).manual_seed(3)

    def normal(rows, width, std=1.0):
        out = torch.zeros(rows, -(-width // 8) * 8, dtype=t, device=DEV)[:, :width]
        out.copy_(torch.randn(rows, width, device=DEV, generator=g) * std)
        return out
    norm = (1 + 0.1 * torch.randn(K, device=DEV, generator=g)).to(t)
    layer = ffn.FeedForward(norm, normal(N, K, K ** -0.5), normal(N, K, K ** -0.5), normal(K, N, N ** -0.5),
                            act=act, eps=1e-5)
    x, r, dy, dt = normal(T, K), normal(T, K), normal(T, K), normal(T, K)
    y, total, saved = layer.forward(x, r)
    dx, grads = layer.backward(saved, dy, dtotal=dt)
    served, total2, nothing = layer.forward(x, r, train=False)
    assert nothing is None and torch.equal(served, y) and torch.equal(total2, total)

    p = {n: getattr(layer, n).double().requires_grad_() for n in ("norm", "gate", "up", "down")}
    tot = total.double().requires_grad_()
    n = tot / (tot.square().mean(dim=1, keepdim=True) + 1e-5).sqrt() * p["norm"]
    h = ref.act(n @ p["gate"].t(), act)[0] * (n @ p["up"].t())
    want = h @ p["down"].t()
    ((want * dy.double()).sum() + (tot * dt.double()).sum()).backward()
    lim = 6 * 2 * torch.finfo(t).eps / 2
    assert torch.equal(total, (x.float() + r.float()).to(t))
    assert _off(y, want.detach()) <= lim
    assert _off(dx, tot.grad) <= lim
    for name, got in grads.items():
        assert _off(got, p[name].grad) <= lim, name


def test_layer_without_residual():
    import torch
    from shape_driven_tile_amd import ffn
    w = torch.randn(64, 32, device=DEV).half()
    layer = ffn.FeedForward(torch.ones(32, device=DEV).half(), w, w, torch.randn(32, 64, device=DEV).half())
    x = torch.randn(5, 32, device=DEV).half()
    y, total, saved = layer.forward(x)
    assert total is x
    zero = torch.zeros_like(x)
    y0, total0, _ = layer.forward(x, zero)
    assert torch.equal(y, y0) and torch.equal(total0, x)
    with pytest.raises(ValueError):
        ffn.FeedForward(torch.ones(32, device=DEV).half(), w, w, w)
    with pytest.raises(ValueError):
        ffn.FeedForward(torch.ones(32, device=DEV).half(), w, w, w.t().contiguous(), act="relu")


def test_layer_without_tokens():
    """An empty batch: empty outputs, gradients of the weights of zero."""
    import torch
    from shape_driven_tile_amd import ffn
    w = torch.randn(64, 32, device=DEV).half()
    layer = ffn.FeedForward(torch.ones(32, device=DEV).half(), w, w, torch.randn(32, 64, device=DEV).half())
    x = torch.empty(0, 32, device=DEV, dtype=torch.float16)
    y, total, saved = layer.forward(x, x)
    dx, grads = layer.backward(saved, y, dtotal=y)
    assert y.shape == total.shape == dx.shape == (0, 32)
    for name, shape in (("norm", (32,)), ("gate", (64, 32)), ("up", (64, 32)), ("down", (32, 64))):
        assert grads[name].shape == shape and not grads[name].any(), name


@pytest.mark.parametrize("T", [1, 40, 300])
def test_fp8_projection(T):
    """The product of the 8-bit rows that the norm makes with the 8-bit weights."""
    import torch
    from shape_driven_tile_amd import binding as sdt
    from shape_driven_tile_amd import ffn
    K, N = 700, 264
    w = torch.randn(N, 704, device=DEV).bfloat16()[:, :K] * K ** -0.5
    norm = torch.rand(K, device=DEV).bfloat16() + 0.5
    x, r = (torch.randn(T, 704, device=DEV).bfloat16()[:, :K] for _ in range(2))
    project = ffn.Fp8Projection(norm, w)
    y, total = project(x, r)
    q = sdt.Fp8.empty(T, K, device=DEV)
    sdt.rms_norm(x, norm, q=q, residual=r)
    a, b = torch.empty(T, K, device=DEV), torch.empty(N, K, device=DEV)
    sdt.fp8_dequantize_f32(q, a)
    sdt.fp8_dequantize_f32(project.weight, b)
    want = a.double() @ b.double().t()
    lim = (K + 4) * 2.0 ** -24 * (a.abs() @ b.abs().t()).double()
    n = -(-K // 8) * 8

    def tops(v):                 # what the MFMA drops of eight products: 2^-10 of the largest
        return torch.nn.functional.pad(v.abs().double(), (0, n - K)).view(v.shape[0], -1, 8).amax(dim=2)
    lim += 2.0 ** -10 * (tops(a) @ tops(b).t())
    assert bool(((y.double() - want).abs() <= lim + 2.0 ** -8 * (want.abs() + lim)).all())
    assert torch.equal(total, (x.float() + r.float()).bfloat16())
    again = ffn.Fp8Projection(norm, project.weight)
    assert torch.equal(again(x, r)[0], y)


def test_layer_in_a_graph():
    """A training step captured, and replayed among eager steps of the same layer."""
    import torch
    from shape_driven_tile_amd import ffn
    T, K, N = 90, 128, 264
    w = [torch.randn(s, device=DEV).bfloat16() * 0.1 for s in ((N, K), (N, K), (K, N))]
    layer = ffn.FeedForward(torch.ones(K, device=DEV).bfloat16(), *w)
    x, r, dy = (torch.randn(T, K, device=DEV).bfloat16() for _ in range(3))

    def step():
        y, total, saved = layer.forward(x, r)
        dx, grads = layer.backward(saved, dy, dtotal=dy)
        return [y, total, dx, *grads.values()]
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        captured = step()
    for _ in range(4):
        for t in (x, r, dy):
            t.copy_(torch.randn(T, K, device=DEV))
        graph.replay()
        eager = step()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(captured, eager))


def test_example(capsys):
    from shape_driven_tile_amd import ffn
    ffn.main(["--tokens", "100", "--hidden", "264", "--inter", "520", "--steps", "2", "--act", "gelu"])
    out = capsys.readouterr().out
    assert "a training step" in out and "8-bit projection" in out and "nan" not in out

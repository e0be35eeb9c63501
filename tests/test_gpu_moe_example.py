"""The example command routes by logits of 16-bit products: ranking experts is where
a 4-bit product's error shows first."""
import pytest

from gpu_helpers import say

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("experts,hidden", [(8, 512), (13, 512), (13, 301)])
def test_example_routes_by_16_bit_products(monkeypatch, experts, hidden):
    import torch

    from shape_driven_tile_amd import binding as sdt
    from shape_driven_tile_amd import moe
    products, routed = [], []
    gemm, route = sdt.gemm_bf16, sdt.moe_route
    monkeypatch.setattr(sdt, "gemm_bf16", lambda A, B, C, **kw: (products.append((A, B, C)),
                                                                 gemm(A, B, C, **kw)))
    monkeypatch.setattr(sdt, "moe_route", lambda logits, *a, **kw: (routed.append(logits),
                                                                    route(logits, *a, **kw)))
    say(f"moe example's router, {experts} experts, {hidden}")
    moe.main(["--tokens", "37", "--experts", str(experts), "--topk", "3", "--hidden", str(hidden),
              "--inter", "128", "--steps", "1"])
    torch.cuda.synchronize()
    assert products and len(products) == len(routed)
    x, w, c = products[-1]
    logits = routed[-1]
    assert logits.data_ptr() == c.data_ptr() and logits.shape == (37, experts)
    want = x.double().cpu() @ w.double().cpu().T
    size = x.double().abs().cpu() @ w.double().abs().cpu().T
    # up to 512 additions in fp32 and half a step of bf16
    tol = 513 * 2.0 ** -24 * size * (1 + 2.0 ** -8) + 2.0 ** -8 * want.abs() + 2.0 ** -134
    assert bool(((logits.double().cpu() - want).abs() <= tol).all())
    assert 0.5 < logits.float().std().item() < 2.0       # a softmax that is not saturated

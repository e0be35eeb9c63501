"""Outputs of the norm and of its gradients over the inputs that they may replace: bit for
bit what they are with memory of their own.  More rows than workgroups that keep the
weight's gradient, so that the next row is on its way while one is stored; rows of every
number of lanes and chunks, most of them ending inside a chunk, which is then read as the
row's last eight elements, those of the lane before among them."""
import pytest

from gpu_helpers import DEV, say
from test_gpu_ffn import normal, rows_of

pytestmark = pytest.mark.gpu

SIZES = [(2100, 300), (1100, 520), (1100, 1000), (1050, 2041), (1050, 4097), (700, 8170), (530, 16390), (520, 32761)]


def _sdt():
    from shape_driven_tile_amd import binding
    return binding


def copy(t, pad):
    return rows_of(t, pad, align=1)[0]


@pytest.mark.parametrize("rows, K", SIZES)
@pytest.mark.parametrize("pad", [0, 3])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_norm(dtype, rows, K, pad):
    import torch
    say(f"norm in place {dtype} {rows}x{K}+{pad}")
    sdt, t = _sdt(), torch.float16 if dtype == "f16" else torch.bfloat16
    x, r, w = (normal(s, t, i) for i, s in enumerate([(rows, K), (rows, K), (K,)]))
    y, total = torch.empty_like(x), torch.empty_like(x)
    q = sdt.Fp8.empty(rows, K, device=DEV)
    sdt.rms_norm(x, w, y=y, q=q, residual=r, total=total)
    codes = q.q.view(torch.uint8).clone()
    # which of total and y replaces x, and which the residual (None: memory of its own)
    for over_x, over_r in (("total", None), (None, "total"), ("y", None), (None, "y"), ("total", "y"), ("y", "total")):
        x2, r2 = copy(x, pad), copy(r, pad)
        got = {n: copy(torch.full_like(x, float("nan")), pad) for n in ("total", "y")}
        for name, over in ((over_x, x2), (over_r, r2)):
            if name:
                got[name] = over
        q.q.view(torch.uint8).fill_(0x55)
        sdt.rms_norm(x2, w, y=got["y"], q=q, residual=r2, total=got["total"])
        assert torch.equal(got["y"], y) and torch.equal(got["total"], total), (over_x, over_r)
        assert torch.equal(q.q.view(torch.uint8), codes), (over_x, over_r)
    alone = torch.empty_like(x)
    sdt.rms_norm(x, w, y=alone)
    x2 = copy(x, pad)
    sdt.rms_norm(x2, w, y=x2)
    assert torch.equal(x2, alone)


@pytest.mark.parametrize("rows, K", SIZES)
@pytest.mark.parametrize("pad", [0, 3])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_norm_backward(dtype, rows, K, pad):
    import torch
    say(f"norm gradients in place {dtype} {rows}x{K}+{pad}")
    sdt, t = _sdt(), torch.float16 if dtype == "f16" else torch.bfloat16
    x, dy, dt, w = (normal(s, t, i) for i, s in enumerate([(rows, K)] * 3 + [(K,)]))
    rstd = torch.empty(rows, device=DEV)
    sdt.rms_norm(x, w, rstd=rstd)
    ws = torch.empty(sdt.rms_norm_workspace_size(rows, K), dtype=torch.uint8, device=DEV)
    dx, dw = torch.empty_like(x), torch.empty(K, device=DEV)
    for extra in (None, dt):
        sdt.rms_norm_backward(x, w, rstd, dy, dx, dw, ws, dtotal=extra)
        for over in ("dy",) if extra is None else ("dy", "dtotal"):
            mine = {"dy": copy(dy, pad), "dtotal": None if extra is None else copy(extra, pad)}
            dw2 = torch.full((K,), float("nan"), device=DEV)
            ws.fill_(0xFF)
            sdt.rms_norm_backward(x, w, rstd, mine["dy"], mine[over], dw2, ws, dtotal=mine["dtotal"])
            assert torch.equal(mine[over], dx) and torch.equal(dw2, dw), (over, extra is None)

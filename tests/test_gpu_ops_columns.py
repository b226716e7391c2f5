"""Inputs and outputs in different columns of one buffer, against the same calls on buffers of
their own (equal inputs give equal bits), and what lies between the columns stays."""
import pytest
import torch

import nvfp4_expert_layer_amd as nv
from tests.gpu_helpers import log, require_gpu

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def columns(rows, *widths, gap=8, dtype=BF):
    """One buffer of 77s, its row pitch a multiple of 8, and views of its columns, `gap` elements
    between and at least as many behind them."""
    pitch = (sum(widths) + gap * len(widths) + 7) // 8 * 8
    buf = torch.full((rows, pitch), 77.0, dtype=dtype, device="cuda")
    views, at = [], 0
    for w in widths:
        views.append(buf[:, at:at + w])
        at += w + gap
    return buf, views


def gaps_untouched(buf, views):
    keep = torch.ones(buf.shape[1], dtype=torch.bool, device="cuda")
    for v in views:
        at = v.storage_offset()
        keep[at:at + v.shape[1]] = False
    return bool((buf[:, keep] == 77).all())


@pytest.mark.parametrize("T,d", [(3, 16), (700, 24), (50, 4096)])
def test_dispatch_and_combine(T, d):
    require_gpu()
    log(f"columns dispatch / combine T={T} d={d}")
    k, E = 4, 12
    gen = torch.Generator(device="cuda").manual_seed(T)
    ids = torch.rand(T, E, generator=gen, device="cuda").topk(k, 1).indices.int()
    p = nv.make_dispatch_problem(T, d, E, k, 0, E)
    ws = nv.alloc_dispatch_workspace(p)
    w = torch.rand(T, k, generator=gen, device="cuda")
    x0 = torch.randn(T, d, generator=gen, device="cuda").to(BF)
    inv = torch.empty(T, k, dtype=torch.int32, device="cuda")
    rows0, out0 = torch.empty(T * k, d, dtype=BF, device="cuda"), torch.empty(T, d, dtype=BF, device="cuda")
    drows0, dw0 = torch.empty_like(rows0), torch.empty_like(w)
    nv.moe_dispatch(p, ids, x0, None, None, None, inv, rows0, ws)
    nv.moe_combine(p, inv, w, rows0, out0)
    nv.moe_combine_backward(p, inv, w, rows0, x0, drows0, dw0)

    buf, (xv, rows, drows) = columns(T * k, d, d, d)
    x, out = xv[::k], xv[1::k]                                     # every k-th row; the rows after them
    x.copy_(x0)
    inv2, dw = torch.empty_like(inv), torch.empty_like(w)
    nv.moe_dispatch(p, ids, x, None, None, None, inv2, rows, ws)
    assert torch.equal(inv2, inv) and torch.equal(rows, rows0)
    nv.moe_combine(p, inv, w, rows, out)
    assert torch.equal(out, out0)
    nv.moe_combine_backward(p, inv, w, rows, x, drows, dw)
    assert torch.equal(drows, drows0) and torch.equal(dw, dw0)
    assert torch.equal(x, x0) and torch.equal(rows, rows0) and gaps_untouched(buf, (xv, rows, drows))
    assert (xv[2::k] == 77).all()


@pytest.mark.parametrize("M,G", [(5, 1), (100, 8), (2300, 8)])
@pytest.mark.parametrize("N,K", [(64, 96), (250, 512)])
def test_product_and_its_gradient(M, G, N, K):
    require_gpu()
    log(f"columns product M={M} G={G} N={N} K={K}")
    gen = torch.Generator(device="cuda").manual_seed(M + N)
    w = nv.quantize_mxfp4_weights(torch.randn(G, N, K, generator=gen, device="cuda"))
    off = torch.linspace(0, M, G + 1).int().cuda()
    p = nv.make_product_problem(M, N, K, G)
    a0 = torch.randn(M, K, generator=gen, device="cuda").to(BF)
    out0, da0 = torch.empty(M, N, dtype=BF, device="cuda"), torch.empty(M, K, dtype=BF, device="cuda")
    nv.moe_mxfp4_product(p, a0, w, off, out0)
    nv.moe_mxfp4_product_backward(p, out0, w, off, da0)
    buf, (a, out, da) = columns(M, K, N, K)
    a.copy_(a0)
    nv.moe_mxfp4_product(p, a, w, off, out)
    assert torch.equal(out, out0)
    nv.moe_mxfp4_product_backward(p, out, w, off, da)
    assert torch.equal(da, da0)
    assert torch.equal(a, a0) and gaps_untouched(buf, (a, out, da))

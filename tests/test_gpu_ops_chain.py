"""The operators together, as a layer uses them: the fused layer's router, dispatch,
MXFP4 products with a SwiGLU between them, combine; and the way back to the token
rows and the routing weights.  Against the same formulas in fp64 torch autograd on
the bf16 tensors that the chain itself holds (each step's rounding is then that
step's alone, so each is bounded by its own arithmetic)."""
import numpy as np
import pytest
import torch

import nvfp4_expert_layer_amd as nv
from oracle import mxfp4
from tests.gpu_helpers import log, require_gpu

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def close(got, ref, mag, terms, what):
    """terms fp32 operations on magnitudes mag, then one bf16 rounding."""
    err = (got.double() - ref).abs()
    lim = terms * 2.0 ** -23 * mag + 2.0 ** -8 * 1.01 * ref.abs() + 1e-30
    assert (err <= lim).all(), (what, float((err / lim).max()))


@pytest.mark.parametrize("T,E,k,offset,L", [(1, 16, 2, 0, 16), (50, 24, 4, 6, 12), (700, 8, 3, 0, 8)])
@pytest.mark.parametrize("w4a4", [False, True])
def test_layer_and_its_gradient(T, E, k, offset, L, w4a4):
    require_gpu()
    log(f"chain T={T} E={E} k={k} shard [{offset}, {offset + L}) w4a4={w4a4}")
    d, F = 256, 128
    gen = torch.Generator(device="cuda").manual_seed(T)
    x = torch.randn(T, d, generator=gen, device="cuda").to(BF)
    gate = (torch.randn(E, d, generator=gen, device="cuda") * 0.1).to(BF)
    w13 = nv.quantize_mxfp4_weights((torch.randn(L, 2 * F, d, generator=gen, device="cuda") / 16).to(BF))
    w2 = nv.quantize_mxfp4_weights((torch.randn(L, d, F, generator=gen, device="cuda") / 11).to(BF))
    val = lambda w: torch.from_numpy(mxfp4.dequantize(w.codes.cpu().numpy(), w.scales.cpu().numpy())).cuda()  # noqa: E731
    v13, v2 = val(w13), val(w2)
    i32, M = dict(dtype=torch.int32, device="cuda"), T * k
    rows_of = lambda n: torch.zeros(M, n, dtype=BF, device="cuda")                                           # noqa: E731

    # the fused layer's own router gives ids and weights; its plan must agree
    pr = nv.make_problem(T, d, F, E, k, offset, L, False, nv.W4A16)
    ids, w = torch.empty(T, k, **i32), torch.empty(T, k, device="cuda")
    rc, ro, rp = torch.empty(L, **i32), torch.empty(L + 1, **i32), torch.zeros(M, **i32)
    nv.moe_nvfp4_route(pr, x, gate, nv.alloc_workspace(pr), ids, w, rc, ro, rp)
    p = nv.make_dispatch_problem(T, d, E, k, offset, L)
    counts, offsets, perm, inv = torch.empty(L, **i32), torch.empty(L + 1, **i32), torch.zeros(M, **i32), torch.empty(T, k, **i32)
    xs = rows_of(d)
    nv.moe_dispatch(p, ids, x, counts, offsets, perm, inv, xs, nv.alloc_dispatch_workspace(p))
    P = int(offsets[-1])
    assert torch.equal(counts, rc) and torch.equal(offsets, ro) and torch.equal(perm[:P], rp[:P])

    def product(a, wt, N, K):
        out = rows_of(N)
        if w4a4:
            q = nv.MXFP4Rows.empty(M, K)
            nv.moe_mxfp4_quantize(a, q.codes, q.scales)
            nv.moe_mxfp4_product(nv.make_product_problem(M, N, K, L), q, wt, offsets, out)
            a = torch.empty(M, K, dtype=BF, device="cuda")
            nv.moe_mxfp4_dequantize(q.codes, q.scales, a)
        else:
            nv.moe_mxfp4_product(nv.make_product_problem(M, N, K, L), a, wt, offsets, out)
        return out, a

    def ref_product(a, v, trans):
        out = torch.zeros(M, v.shape[1] if trans else v.shape[2], dtype=torch.float64, device="cuda")
        o = offsets.tolist()
        for g in range(L):
            m = v[g].t().contiguous() if trans else v[g]
            out[o[g]:o[g + 1]] = a[o[g]:o[g + 1]].double() @ m
        return out

    h, hx = product(xs, w13, 2 * F, d)
    close(h, ref_product(hx, v13, True), ref_product(hx.abs(), v13.abs(), True), d, "gate/up")
    hf = h.float()
    act = (torch.nn.functional.silu(hf[:, :F]) * hf[:, F:]).to(BF)
    y, ya = product(act, w2, d, F)
    close(y, ref_product(ya, v2, True), ref_product(ya.abs(), v2.abs(), True), F, "down")
    out = torch.empty(T, d, dtype=BF, device="cuda")
    nv.moe_combine(p, inv, w, y, out)
    kept = (inv >= 0).double().unsqueeze(2)
    at = inv.clamp(min=0).long()
    terms = w.double().unsqueeze(2) * y.double()[at] * kept
    close(out, terms.sum(1), terms.abs().sum(1), k + 1, "combine")

    # backward from a gradient of the output
    dout = (torch.randn(T, d, generator=gen, device="cuda") * 0.1).to(BF)
    dy, dw = rows_of(d), torch.empty(T, k, device="cuda")
    nv.moe_combine_backward(p, inv, w, y, dout, dy, dw)
    dact, dh, dxs = rows_of(F), rows_of(2 * F), rows_of(d)
    nv.moe_mxfp4_product_backward(nv.make_product_problem(M, d, F, L), dy, w2, offsets, dact)
    close(dact, ref_product(dy, v2, False), ref_product(dy.abs(), v2.abs(), False), d, "down gradient")
    g64 = h.double().requires_grad_()
    (torch.nn.functional.silu(g64[:, :F]) * g64[:, F:] * dact.double()).sum().backward()
    dh.copy_(g64.grad)
    nv.moe_mxfp4_product_backward(nv.make_product_problem(M, 2 * F, d, L), dh, w13, offsets, dxs)
    close(dxs, ref_product(dh, v13, False), ref_product(dh.abs(), v13.abs(), False), 2 * F, "gate/up gradient")
    dx = torch.empty(T, d, dtype=BF, device="cuda")
    nv.moe_dispatch_backward(p, inv, dxs, dx)
    terms = dxs.double()[at] * kept
    close(dx, terms.sum(1), terms.abs().sum(1), k + 1, "dispatch gradient")

    # the routing weights' gradient against autograd of the combine in fp64
    w64 = w.double().requires_grad_()
    ((w64.unsqueeze(2) * y.double()[at] * kept).sum(1) * dout.double()).sum().backward()
    mag = (y.double()[at].abs() * dout.double().abs().unsqueeze(1) * kept).sum(2)
    assert ((dw.double() - w64.grad).abs() <= d * 2.0 ** -23 * mag).all()
    assert np.isfinite(out.float().cpu().numpy()).all()

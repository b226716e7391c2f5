"""Buffers past 2^32 bytes, neighbours in one buffer, and long axes of the operators in
include/moe_block.h."""
import pytest
import torch

import nvfp4_expert_layer_amd as nv
from tests.gpu_helpers import log, require_gpu

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def tail_equal(a, b, n=3):
    return torch.equal(a[-n:], b[-n:]) and torch.equal(a[:n], b[:n])


def test_rows_past_four_gigabytes():
    """The last rows of tensors of more than 2^32 bytes (and 2^31 elements) equal those of small ones."""
    require_gpu()
    log("block past 2^32 bytes")
    M, C = 40000, 65536                                             # 2.6e9 elements
    x = torch.empty(M, C, dtype=BF, device="cuda").fill_(0.5)
    part = torch.randn(6, C, device="cuda").to(BF)
    x[:3], x[-3:] = part[:3], part[3:]
    log("quantize")
    q, qs = nv.MXFP8Rows.empty(M, C), nv.MXFP8Rows.empty(6, C)
    nv.moe_mxfp8_quantize(x, q.codes, q.scales)
    nv.moe_mxfp8_quantize(part, qs.codes, qs.scales)
    ends = lambda t: torch.cat([t[:3], t[-3:]])  # noqa: E731
    assert torch.equal(ends(q.codes), qs.codes) and torch.equal(ends(q.scales), qs.scales)
    log("dequantize")
    y, ys = torch.empty_like(x), torch.empty_like(part)
    nv.moe_mxfp8_dequantize(q.codes, q.scales, y)
    nv.moe_mxfp8_dequantize(qs.codes, qs.scales, ys)
    assert torch.equal(ends(y), ys)
    log("swiglu and its gradient from kept rows")
    F = C // 2
    da, das = torch.empty(M, F, dtype=BF, device="cuda").fill_(0.25), torch.randn(6, F, device="cuda").to(BF)
    da[:3], da[-3:] = das[:3], das[3:]
    p, ps = nv.make_swiglu_problem(M, F), nv.make_swiglu_problem(6, F)
    a, as_ = torch.empty_like(da), torch.empty_like(das)
    nv.moe_swiglu(p, x, None, a, None, q)
    nv.moe_swiglu(ps, part, None, as_, None, qs)
    assert torch.equal(ends(a), as_) and torch.equal(ends(q.codes), qs.codes)
    nv.moe_swiglu_backward(p, q, None, da, y)
    nv.moe_swiglu_backward(ps, qs, None, das, ys)
    assert torch.equal(ends(y), ys)
    log("norm")
    w, rstd, rs = torch.randn(C, device="cuda").to(BF), torch.empty(M, device="cuda"), torch.empty(6, device="cuda")
    nv.moe_norm(nv.make_norm_problem(M, C), x, None, w, None, y, q, rstd)
    nv.moe_norm(nv.make_norm_problem(6, C), part, None, w, None, ys, qs, rs)
    assert torch.equal(ends(y), ys) and torch.equal(ends(q.codes), qs.codes) and torch.equal(ends(rstd), rs)
    del a, da
    log("norm gradient")
    nv.moe_norm_backward(nv.make_norm_problem(M, C), x, w, rstd, y, None, x.new_empty(M, C), None)
    dx, dxs = torch.empty_like(x), torch.empty_like(part)
    nv.moe_norm_backward(nv.make_norm_problem(M, C), x, w, rstd, y, None, dx, None)
    nv.moe_norm_backward(nv.make_norm_problem(6, C), part, w, rs, ys, None, dxs, None)
    assert torch.equal(ends(dx), dxs)


def test_route_of_many_tokens_past_four_gigabytes():
    require_gpu()
    log("route past 2^32 bytes")
    T, E, k = 4_300_000, 512, 4                                     # 2.2e9 logits, 8.8e9 bytes
    l = torch.zeros(T, E, device="cuda")
    part = torch.randn(6, E, device="cuda")
    l[:3], l[-3:] = part[:3], part[3:]
    b = torch.randn(E, device="cuda") * 0.01
    ends = lambda t: torch.cat([t[:3], t[-3:]])  # noqa: E731
    p, ps = (nv.make_route_problem(n, E, k, nv.ROUTE_SIGMOID) for n in (T, 6))
    ids, w = torch.empty(T, k, dtype=torch.int32, device="cuda"), torch.empty(T, k, device="cuda")
    i6, w6 = torch.empty(6, k, dtype=torch.int32, device="cuda"), torch.empty(6, k, device="cuda")
    nv.moe_route(p, l, b, ids, w)
    nv.moe_route(ps, part, b, i6, w6)
    assert torch.equal(ends(ids), i6) and torch.equal(ends(w), w6)
    # zeros everywhere else: the bias decides, the weights are equal
    want = b.sort(descending=True, stable=True).indices[:k].int()
    assert torch.equal(ids[3:-3], want.expand(T - 6, k)) and (w[3:-3] == 0.25).all()
    d, d6 = torch.empty_like(l), torch.empty_like(part)
    nv.moe_route_backward(p, l, ids, w, d)
    nv.moe_route_backward(ps, part, i6, w6, d6)
    assert torch.equal(ends(d), d6)


def test_product_past_four_gigabytes():
    """Rows, weights and outputs whose offsets pass 32 bits."""
    require_gpu()
    log("product8 past 2^32 bytes")
    M, K = 70000, 65536                                             # 4.6e9 codes
    q = nv.MXFP8Rows(torch.zeros(M, K, dtype=torch.uint8, device="cuda"), torch.full((M, K // 32), 127, dtype=torch.uint8,
                                                                                    device="cuda"))
    part = nv.MXFP8Rows.empty(200, K)
    nv.moe_mxfp8_quantize(torch.randn(200, K, device="cuda"), part.codes, part.scales)
    q.codes[-200:], q.scales[-200:] = part.codes, part.scales
    w = nv.quantize_mxfp4_weights(torch.randn(2, 24, K, device="cuda"))
    off = torch.tensor([0, M - 150, M], dtype=torch.int32, device="cuda")
    out = torch.empty(M, 24, dtype=torch.float32, device="cuda")
    nv.moe_mxfp8_product(nv.make_product_problem(M, 24, K, 2), q, w, off, out)
    small = torch.empty(200, 24, dtype=torch.float32, device="cuda")
    po = torch.tensor([0, 50, 200], dtype=torch.int32, device="cuda")
    nv.moe_mxfp8_product(nv.make_product_problem(200, 24, K, 2), part, w, po, small)
    # (tiles and streaming add in other orders: both are within the bound of exact sums)
    mag = torch.empty_like(small)
    pos = nv.MXFP8Rows(part.codes & 0x7F, part.scales)
    wp = nv.MXFP4Weights(w.codes & 0x77, w.scales)
    nv.moe_mxfp8_product(nv.make_product_problem(200, 24, K, 2), pos, wp, po, mag)
    assert ((out[-200:] - small).abs() <= (2.0 ** -9 + K * 2.0 ** -23) * mag).all()
    assert (out[:-200] == 0).all()
    del q
    # weights of 5.4e9 codes' bytes: the last group's reach past 2^32
    G, N, K = 1024, 2560, 4096
    w = nv.MXFP4Weights(torch.zeros(G, N, K // 2, dtype=torch.uint8, device="cuda"),
                        torch.full((G, N, K // 32), 127, dtype=torch.uint8, device="cuda"))
    last = nv.quantize_mxfp4_weights(torch.randn(1, N, K, device="cuda"))
    w.codes[-1], w.scales[-1] = last.codes[0], last.scales[0]
    for rows in (20, 500):
        x = nv.MXFP8Rows.empty(rows, K)
        nv.moe_mxfp8_quantize(torch.randn(rows, K, device="cuda"), x.codes, x.scales)
        off = torch.zeros(G + 1, dtype=torch.int32, device="cuda")
        off[-1] = rows
        a, b = torch.empty(rows, N, device="cuda"), torch.empty(rows, N, device="cuda")
        nv.moe_mxfp8_product(nv.make_product_problem(rows, N, K, G), x, w, off, a)
        nv.moe_mxfp8_product(nv.make_product_problem(rows, N, K, 1), x, last, None, b)
        mag = torch.empty_like(a)
        nv.moe_mxfp8_product(nv.make_product_problem(rows, N, K, 1), nv.MXFP8Rows(x.codes & 0x7F, x.scales),
                             nv.MXFP4Weights(last.codes & 0x77, last.scales), None, mag)
        assert ((a - b).abs() <= (2.0 ** -9 + K * 2.0 ** -23) * mag).all()


def test_columns_of_one_buffer():
    """Inputs and outputs in different columns of one buffer, against buffers of their own."""
    require_gpu()
    log("block columns")
    T, d, E = 37, 96, 40
    x, r, w = (torch.randn(*s, device="cuda").to(BF) for s in ((T, d), (T, d), (d,)))
    h, y = torch.empty_like(x), torch.empty_like(x)
    p = nv.make_norm_problem(T, d)
    nv.moe_norm(p, x, r, w, h, y, None, None)
    buf = torch.full((T, 4 * d + 4), 7.0, dtype=BF, device="cuda")
    v = [buf[:, i * (d + 1):i * (d + 1) + d] for i in range(4)]
    v[0].copy_(x)
    v[1].copy_(r)
    nv.moe_norm(p, v[0], v[1], w, v[2], v[3], None, None)
    assert torch.equal(v[2], h) and torch.equal(v[3], y) and (buf[:, d::d + 1] == 7).all()
    l = torch.randn(T, 2 * E, device="cuda")
    rp = nv.make_route_problem(T, E, 4, renormalize=False)
    ids, rw = torch.empty(T, 4, dtype=torch.int32, device="cuda"), torch.empty(T, 4, device="cuda")
    nv.moe_route(rp, l[:, :E], None, ids, rw)
    want = torch.empty(T, E, device="cuda")
    nv.moe_route_backward(rp, l[:, :E], ids, rw, want)
    nv.moe_route_backward(rp, l[:, :E], ids, rw, l[:, E:])
    assert torch.equal(l[:, E:], want)
    with pytest.raises(RuntimeError, match="overlaps"):
        nv.moe_route_backward(rp, l[:, :E], ids, rw, l[:, E - 1:2 * E - 1])
    with pytest.raises(RuntimeError, match="overlaps"):
        nv.moe_norm(p, x, r, w, r, y, None, None)


def test_long_axes():
    """One row of the widest kind through each operator; many rows of the narrowest."""
    require_gpu()
    log("block long axes")
    x = torch.randn(1, 65536, device="cuda")
    w, rstd = torch.ones(65536, device="cuda"), torch.empty(1, device="cuda")
    y = torch.empty_like(x)
    nv.moe_norm(nv.make_norm_problem(1, 65536, 0.0, torch.float32), x, None, w, None, y, None, rstd)
    assert abs(float(y.double().square().mean()) - 1) <= 1e-5
    T = 1 << 21
    x = torch.randn(T, 1, device="cuda")
    y, dw = torch.empty_like(x), torch.empty(1, device="cuda")
    p = nv.make_norm_problem(T, 1, 0.0, torch.float32)
    rstd = torch.empty(T, device="cuda")
    nv.moe_norm(p, x, None, torch.ones(1, device="cuda"), None, y, None, rstd)
    zero = x == 0                                                   # with eps = 0: 0 / 0
    assert ((y.abs() - 1).abs() <= 1e-6)[~zero].all() and torch.isnan(y[zero]).all()
    rstd = (x[:, 0].square() + 1e-6).rsqrt()
    nv.moe_norm_backward(p, x, torch.ones(1, device="cuda"), rstd, torch.ones_like(x), None, y, dw, nv.alloc_norm_workspace(p))
    n = x.double() * rstd.double().unsqueeze(1)
    # a column's sum: up to T / 512 rows in a row, then trees
    assert abs(float(dw) - float(n.sum())) <= (T / 512 + 60) * 2.0 ** -24 * float(n.abs().sum())

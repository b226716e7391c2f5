"""The operators together, as a layer uses them: a residual's addition and the norm, the
router's choice, dispatch of 8-bit rows, W4A8 products with a SwiGLU that keeps its input in
8 bits, combine; and the way back to the residual stream, the norm's weight and the router's
logits.  Each step against its formula in fp64 on the tensors that the chain itself holds."""
import numpy as np
import pytest
import torch

import nvfp4_expert_layer_amd as nv
from oracle import block, mxfp4
from tests.gpu_helpers import log, require_gpu

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
U = 2.0 ** -24


def near(got, ref, slack, what):
    """One bf16 rounding and what the sums before it may lose."""
    err = (got.double() - ref).abs()
    lim = slack + 2.0 ** -8 * 1.01 * ref.abs() + 1e-30
    assert (err <= lim).all(), (what, float((err / lim).max()))


def values8(q):
    return torch.from_numpy(block.mxfp8_dequantize(q.codes.cpu().numpy(), q.scales.cpu().numpy())).cuda()


class Layer:
    """One shard of a layer and its buffers."""

    def __init__(self, T, E, k, offset, L, d=256, F=128, seed=0):
        self.T, self.E, self.k, self.L, self.d, self.F = T, E, k, L, d, F
        g = torch.Generator(device="cuda").manual_seed(seed + T)
        randn = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
        self.x, self.res, self.nw = randn(T, d).to(BF), randn(T, d).to(BF), (1 + 0.1 * randn(d)).to(BF)
        self.gate, self.bias = (randn(E, d) * 0.1).to(BF), randn(E) * 0.05
        self.w13 = nv.quantize_mxfp4_weights(randn(L, 2 * F, d) / 16)
        self.w2 = nv.quantize_mxfp4_weights(randn(L, d, F) / 11)
        self.dout, self.dres = (randn(T, d) * 0.1).to(BF), (randn(T, d) * 0.1).to(BF)
        M, i32 = T * k, dict(dtype=torch.int32, device="cuda")
        rows = lambda n, m=M: torch.zeros(m, n, dtype=BF, device="cuda")  # noqa: E731
        self.h, self.y, self.rstd, self.yq = rows(d, T), rows(d, T), torch.empty(T, device="cuda"), nv.MXFP8Rows.empty(T, d)
        self.ids, self.w = torch.empty(T, k, **i32), torch.empty(T, k, device="cuda")
        self.offsets, self.inv = torch.empty(L + 1, **i32), torch.empty(T, k, **i32)
        q = lambda n: nv.MXFP8Rows(torch.zeros(M, n, dtype=torch.uint8, device="cuda"),  # noqa: E731
                                   torch.full((M, n // 32), 127, dtype=torch.uint8, device="cuda"))
        self.xs, self.aq, self.kept = q(d), q(F), q(2 * F)
        self.u, self.z, self.out = rows(2 * F), rows(d), rows(d, T)
        self.dz, self.dw, self.da, self.du, self.dxs = rows(d), torch.empty(T, k, device="cuda"), rows(F), rows(2 * F), rows(d)
        self.dy, self.dx, self.dnw = rows(d, T), rows(d, T), torch.empty(d, device="cuda")
        self.logits, self.dlogits = torch.empty(T, E, device="cuda"), torch.empty(T, E, device="cuda")
        self.pn, self.pr = nv.make_norm_problem(T, d), nv.make_route_problem(T, E, k, nv.ROUTE_SIGMOID, 2, 1, scale=2.5)
        u8 = torch.uint8
        self.pc, self.ps = nv.make_dispatch_problem(T, d, E, k, offset, L, u8), nv.make_dispatch_problem(T, d // 32, E, k, offset, L, u8)
        self.pd = nv.make_dispatch_problem(T, d, E, k, offset, L)
        self.p13, self.p2 = nv.make_product_problem(M, 2 * F, d, L), nv.make_product_problem(M, d, F, L)
        self.pa = nv.make_swiglu_problem(M, F, L)
        self.ws, self.wn = nv.alloc_dispatch_workspace(self.pc), nv.alloc_norm_workspace(self.pn)

    def forward(self):
        nv.moe_norm(self.pn, self.x, self.res, self.nw, self.h, self.y, self.yq, self.rstd)
        torch.matmul(self.y.float(), self.gate.float().t(), out=self.logits)
        nv.moe_route(self.pr, self.logits, self.bias, self.ids, self.w)
        nv.moe_dispatch(self.pc, self.ids, self.yq.codes, None, self.offsets, None, self.inv, self.xs.codes, self.ws)
        nv.moe_dispatch(self.ps, self.ids, self.yq.scales, None, None, None, None, self.xs.scales, self.ws)
        nv.moe_mxfp8_product(self.p13, self.xs, self.w13, self.offsets, self.u)
        nv.moe_swiglu(self.pa, self.u, self.offsets, None, self.aq, self.kept)
        nv.moe_mxfp8_product(self.p2, self.aq, self.w2, self.offsets, self.z)
        return nv.moe_combine(self.pd, self.inv, self.w, self.z, self.out)

    def backward(self):
        nv.moe_combine_backward(self.pd, self.inv, self.w, self.z, self.dout, self.dz, self.dw)
        nv.moe_mxfp4_product_backward(self.p2, self.dz, self.w2, self.offsets, self.da)
        nv.moe_swiglu_backward(self.pa, self.kept, self.offsets, self.da, self.du)
        nv.moe_mxfp4_product_backward(self.p13, self.du, self.w13, self.offsets, self.dxs)
        nv.moe_dispatch_backward(self.pd, self.inv, self.dxs, self.dy)
        nv.moe_route_backward(self.pr, self.logits, self.ids, self.dw, self.dlogits)
        self.dy += torch.matmul(self.dlogits, self.gate.float()).to(BF)
        nv.moe_norm_backward(self.pn, self.h, self.nw, self.rstd, self.dy, self.dres, self.dx, self.dnw, self.wn)
        return self.dx, self.dnw, self.dlogits

    def results(self):
        return [t.clone() for t in (self.out, self.w, self.ids, self.dx, self.dnw, self.dlogits)]


def products(a, v, offsets, transposed):
    """a[r] times its group's weight values, and the same of the magnitudes."""
    out = torch.zeros(a.shape[0], v.shape[1 if transposed else 2], dtype=torch.float64, device="cuda")
    mag, o = out.clone(), offsets.tolist()
    for g in range(v.shape[0]):
        m = v[g].t().contiguous() if transposed else v[g]
        out[o[g]:o[g + 1]] = a[o[g]:o[g + 1]].double() @ m
        mag[o[g]:o[g + 1]] = a[o[g]:o[g + 1]].double().abs() @ m.abs()
    return out, mag


def aligned_loss(a, v, offsets):
    """Up to 2^-13 of the largest product of a block for each of its 32."""
    top = lambda t: t.abs().unflatten(-1, (-1, 32)).amax(-1)  # noqa: E731
    return 32 * 2.0 ** -13 * products(top(a), top(v), offsets, True)[0]


@pytest.mark.parametrize("T,E,k,offset,L", [(1, 16, 2, 0, 16), (50, 24, 4, 6, 12), (1500, 8, 3, 0, 8)])
def test_layer_and_its_gradients(T, E, k, offset, L):
    require_gpu()
    log(f"block chain T={T} E={E} k={k} shard [{offset}, {offset + L})")
    s = Layer(T, E, k, offset, L)
    s.forward()
    s.backward()
    torch.cuda.synchronize()
    val = lambda w: torch.from_numpy(mxfp4.dequantize(w.codes.cpu().numpy(), w.scales.cpu().numpy())).cuda()  # noqa: E731
    v13, v2, n = val(s.w13), val(s.w2), int(s.offsets[-1])
    num = lambda t: t.double().cpu().numpy()  # noqa: E731
    dev = lambda a: torch.from_numpy(a).cuda()  # noqa: E731

    # norm, choice
    assert torch.equal(s.h, (s.x.float() + s.res.float()).to(BF))
    wy, wr = block.norm(num(s.h), num(s.nw), 1e-6)
    near(s.y, dev(wy), 100 * U * dev(np.abs(wy)), "norm")
    assert (np.abs(num(s.rstd) - wr) <= 60 * U * wr).all()
    l = num(s.logits)
    for t in range(0, T, 7):
        ids, w, _ = block.route_token(l[t], k, "sigmoid", num(s.bias), 2, 1, scale=2.5)
        assert np.array_equal(ids, s.ids[t].cpu().numpy()) and (np.abs(num(s.w[t]) - w) <= U * 1.001 * w).all()
    # 8-bit rows reach their places with their scales
    kept = s.inv >= 0
    token = torch.arange(T, device="cuda").unsqueeze(1).expand(T, k)[kept]
    assert torch.equal(s.xs.codes[s.inv[kept].long()], s.yq.codes[token])
    assert torch.equal(s.xs.scales[s.inv[kept].long()], s.yq.scales[token])
    # products and SwiGLU
    a = values8(s.xs)
    ref, mag = products(a, v13, s.offsets, True)
    near(s.u, ref, aligned_loss(a, v13, s.offsets) + s.d * 2.0 ** -23 * mag, "gate/up")
    codes, scales = block.mxfp8_quantize(num(s.u))
    assert np.array_equal(s.kept.codes[:n].cpu().numpy(), codes[:n]) and np.array_equal(s.kept.scales[:n].cpu().numpy(), scales[:n])
    act, got = block.swiglu(num(s.u[:n])), num(values8(s.aq)[:n])
    step = np.repeat(np.ldexp(1.0, s.aq.scales[:n].cpu().numpy().astype(int) - 127), 32, axis=1)
    over = np.maximum(np.abs(act) - 448 * step, 0)
    assert (np.abs(got - act) <= 1.001 * np.maximum(2.0 ** -4 * np.abs(act), 2.0 ** -10 * step) + over + 40 * U * np.abs(act)).all()
    a = values8(s.aq)
    ref, mag = products(a, v2, s.offsets, True)
    near(s.z, ref, aligned_loss(a, v2, s.offsets) + s.F * 2.0 ** -23 * mag, "down")
    at, live = s.inv.clamp(min=0).long(), kept.double().unsqueeze(2)
    terms = s.w.double().unsqueeze(2) * s.z.double()[at] * live
    near(s.out, terms.sum(1), (k + 1) * 2 * U * terms.abs().sum(1), "combine")

    # back: the rows
    ref, mag = products(s.dz, v2, s.offsets, False)
    near(s.da, ref, s.d * 2 * U * mag, "down gradient")
    u8 = num(values8(s.kept)[:n])
    da = num(s.da[:n])
    want = block.swiglu_gradient(u8, da)
    g, up = u8[:, :s.F], u8[:, s.F:]
    bound = np.concatenate([np.abs(da * up) * (1 + np.abs(g)), np.abs(da * g)], 1) * block.sigmoid(np.concatenate([g, g], 1))
    near(s.du[:n], dev(want), (14 + 2 * float(np.abs(g).max(initial=0))) * U * dev(bound), "SwiGLU gradient")
    ref, mag = products(s.du, v13, s.offsets, False)
    near(s.dxs, ref, 2 * s.F * 2 * U * mag, "gate/up gradient")
    # the router and the norm
    for t in range(0, T, 7):
        i, dw = s.ids[t].cpu().numpy(), num(s.dw[t])
        want = block.route_gradient(l[t], i, dw, "sigmoid", True, 2.5)
        sc = block.sigmoid(l[t][i])
        p = sc / sc.sum()
        lim = np.zeros(E)
        np.add.at(lim, i, 2.5 * p * (np.abs(dw) + (p * np.abs(dw)).sum()))
        assert (np.abs(num(s.dlogits[t]) - want) <= (k + 24) * U * lim + 1e-38).all()
    wx, ww = block.norm_gradient(num(s.h), num(s.nw), num(s.rstd), num(s.dy), num(s.dres))
    nn, gg = np.abs(num(s.h)) * num(s.rstd)[:, None], np.abs(num(s.dy) * num(s.nw))
    near(s.dx, dev(wx), dev(U * (num(s.rstd)[:, None] * (5 * gg + nn * (gg * nn).mean(1)[:, None] * 100) + 2 * np.abs(num(s.dres)))),
         "norm gradient")
    assert (np.abs(num(s.dnw) - ww) <= 100 * U * (np.abs(num(s.dy)) * nn).sum(0) + 1e-38).all()


def test_captured_and_replayed():
    """The whole step as one graph, replayed on new inputs in the same buffers with eager work between,
    and two graphs of two layers in turn: equal bits."""
    require_gpu()
    log("block chain graphs")
    layers = [Layer(70, 24, 4, 6, 12, seed=1), Layer(900, 16, 3, 0, 16, seed=2)]
    graphs = []
    for s in layers:
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            s.forward()
            s.backward()
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            s.forward()
            s.backward()
        graphs.append(g)
    for turn in range(4):
        for s in layers:
            s.x.copy_(torch.randn_like(s.x, dtype=torch.float32))
            s.dout.copy_(torch.randn_like(s.dout, dtype=torch.float32) * 0.1)
        replayed = []
        for s, g in zip(layers, graphs):
            g.replay()
        torch.cuda.synchronize()
        replayed = [s.results() for s in layers]
        for s, r in zip(layers, replayed):
            s.forward()
            s.backward()
            torch.cuda.synchronize()
            for a, b in zip(s.results(), r):
                assert torch.equal(a, b), turn


def test_two_streams_at_once():
    require_gpu()
    log("block chain streams")
    a, b = Layer(300, 24, 4, 0, 24, seed=3), Layer(310, 24, 4, 0, 24, seed=4)
    alone = []
    for s in (a, b):
        s.forward()
        s.backward()
        torch.cuda.synchronize()
        alone.append(s.results())
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(5):
        for s, st in zip((a, b), streams):
            with torch.cuda.stream(st):
                s.forward()
                s.backward()
    torch.cuda.synchronize()
    for s, r in zip((a, b), alone):
        assert all(torch.equal(x, y) for x, y in zip(s.results(), r))


def test_given_stream_and_wrong_device():
    """A stream handed over; its tensors stay the current device's."""
    require_gpu()
    log("block stream argument")
    x = torch.randn(64, 128, device="cuda").to(BF)
    q, r = nv.MXFP8Rows.empty(64, 128), nv.MXFP8Rows.empty(64, 128)
    nv.moe_mxfp8_quantize(x, q.codes, q.scales)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    nv.moe_mxfp8_quantize(x, r.codes, r.scales, stream=st)
    st.synchronize()
    assert torch.equal(q.codes, r.codes) and torch.equal(q.scales, r.scales)
    with pytest.raises(ValueError, match="must be on the GPU"):
        nv.moe_mxfp8_quantize(x, q.codes.cpu(), q.scales)
    with pytest.raises(ValueError, match="must be on the GPU"):
        nv.moe_norm(nv.make_norm_problem(64, 128), x, None, torch.ones(128, dtype=BF), None, x.clone(), None, None)

"""Calls of the operators that the other tests do not make: buffers past 2^32 bytes,
many count blocks, sliced weights and rows, long reductions with few rows, two streams
at once, an explicit stream, one workspace under two graphs."""
import numpy as np
import pytest
import torch

import nvfp4_expert_layer_amd as nv
from oracle import dispatch, mxfp4
from tests.gpu_helpers import log, require_gpu

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
I32 = dict(dtype=torch.int32, device="cuda")


def plan_buffers(p, d, dtype=BF):
    T, k, L = p.num_tokens, p.top_k, p.num_local_experts
    return dict(counts=torch.empty(L, **I32), offsets=torch.empty(L + 1, **I32), perm=torch.full((T * k,), -7, **I32),
                inv=torch.empty(T, k, **I32), rows=torch.zeros(T * k, d, dtype=dtype, device="cuda"))


@pytest.mark.parametrize("T,k,E,L", [(70000, 8, 40, 30), (300000, 1, 1024, 1024)])
def test_dispatch_with_many_count_blocks(T, k, E, L):
    require_gpu()
    log(f"dispatch T={T} k={k} L={L}")
    ids = torch.randint(0, E, (T, k), generator=torch.Generator().manual_seed(1), dtype=torch.int32)
    p = nv.make_dispatch_problem(T, 4, E, k, E - L, L)
    b = plan_buffers(p, 4)
    x = torch.arange(T, device="cuda").view(T, 1).remainder(251).expand(T, 4).to(BF).contiguous()
    nv.moe_dispatch(p, ids.cuda(), x, workspace=nv.alloc_dispatch_workspace(p), **b)
    local = ids.reshape(-1).numpy().astype(np.int64) - (E - L)
    kept = local >= 0
    order = np.argsort(np.where(kept, local, L), kind="stable")[:kept.sum()]
    P = len(order)
    assert np.array_equal(b["perm"].cpu().numpy()[:P], order) and (b["perm"][P:] == -7).all()
    assert np.array_equal(b["counts"].cpu().numpy(), np.bincount(local[kept], minlength=L))
    inv = np.full(T * k, -1)
    inv[order] = np.arange(P)
    assert np.array_equal(b["inv"].cpu().numpy().reshape(-1), inv)
    assert torch.equal(b["rows"][:P], x[torch.from_numpy(order // k).cuda()]) and not b["rows"][P:].any()


def test_rows_past_2_to_the_32_bytes():
    """41000 x 8 rows of 8192 bf16: 5.4 GB; row numbers and byte offsets past 2^32."""
    require_gpu()
    log("dispatch / combine rows past 2^32 bytes")
    T, k, E, d = 41000, 8, 16, 8192
    gen = torch.Generator(device="cuda").manual_seed(3)
    ids = torch.rand(T, E, generator=gen, device="cuda").topk(k, 1).indices.int()
    x = torch.randint(-64, 65, (T, d), generator=gen, device="cuda", dtype=torch.int8).to(BF)
    p = nv.make_dispatch_problem(T, d, E, k, 0, E)
    b = plan_buffers(p, d)
    nv.moe_dispatch(p, ids, x, workspace=nv.alloc_dispatch_workspace(p), **b)
    perm = b["perm"].long()
    assert torch.equal(perm.sort().values, torch.arange(T * k, device="cuda"))
    for r0 in range(0, T * k, 41000):
        assert torch.equal(b["rows"][r0:r0 + 41000], x[perm[r0:r0 + 41000] // k])
    out = torch.empty_like(x)
    nv.moe_dispatch_backward(p, b["inv"], b["rows"], out)
    assert torch.equal(out, x * 8)                                 # eight copies of integers up to 64: exact
    w = torch.full((T, k), 0.125, device="cuda")
    nv.moe_combine(p, b["inv"], w, b["rows"], out)
    assert torch.equal(out, x)
    dw = torch.empty(T, k, device="cuda")
    ones = torch.ones_like(x)
    nv.moe_combine_backward(p, b["inv"], w, b["rows"], ones, None, dw)
    assert torch.equal(dw, x.float().sum(1, keepdim=True).expand(T, k))          # integers below 2^24: exact
    nv.moe_combine_backward(p, b["inv"], w, None, ones, b["rows"], None)
    assert (b["rows"] == 0.125).all()


def test_quantize_past_2_to_the_32_elements():
    require_gpu()
    log("quantize past 2^32 elements")
    R, C = 131072 + 3, 32768
    x = torch.zeros(R, C, dtype=BF, device="cuda")
    x[-1] = torch.arange(C, device="cuda").remainder(13).to(BF)
    x[R // 2, :64] = -3.0
    q = nv.MXFP4Rows.empty(R, C)
    nv.moe_mxfp4_quantize(x, q.codes, q.scales)
    for r in (0, R // 2, R - 1):
        c, s = mxfp4.quantize(x[r:r + 1].double().cpu().numpy())
        assert np.array_equal(q.codes[r].cpu().numpy(), c[0]) and np.array_equal(q.scales[r].cpu().numpy(), s[0])
    nv.moe_mxfp4_dequantize(q.codes, q.scales, x)
    assert torch.equal(x[-1].cpu().double(), torch.from_numpy(mxfp4.dequantize(c, s)[0]))
    assert (x[R // 2, :64] == -3).all() and x[1:R // 2].count_nonzero() == 0


@pytest.mark.parametrize("M", [3000, 300000])
def test_product_weights_and_outputs_past_2_to_the_32_bytes(M):
    """1024 experts of 2112 x 4096 (4.4 GB of codes): the last experts' weights; 300000 rows of 8192
    fp32 (9.8 GB) through one small weight."""
    require_gpu()
    log(f"product past 2^32 bytes M={M}")
    gen = torch.Generator(device="cuda").manual_seed(M)
    G, N, K = (1024, 2112, 4096) if M == 3000 else (2, 8192, 64)
    w = nv.MXFP4Weights.empty(G, N, K)
    w.codes.fill_(0x22)                                            # ones
    w.scales.fill_(127)
    last = torch.randint(0, 256, (2, N, K // 2), generator=gen, dtype=torch.uint8, device="cuda")
    w.codes[-2:] = last
    off = torch.full((G + 1,), M, **I32)
    off[:G - 2] = 0
    off[G - 2], off[G - 1] = 5, M // 2
    if G == 2:
        off[0] = 0
    a = torch.randint(-4, 5, (M, K), generator=gen, device="cuda").to(BF)
    out = torch.zeros(M, N, device="cuda")
    p = nv.make_product_problem(M, N, K, G)
    nv.moe_mxfp4_product(p, a, w, off, out)
    v = torch.from_numpy(mxfp4.dequantize(w.codes[-2:].cpu().numpy(), w.scales[-2:].cpu().numpy())).float().cuda()
    o = off.tolist()
    for g in (0, 1):                                               # exact: integers and halves
        b, e = o[G - 2 + g], o[G - 1 + g]
        for s in {b, (b + e) // 2, e - 300}:
            assert torch.equal(out[s:s + 300], a[s:s + 300].float() @ v[g].t().contiguous())
    del out
    da = torch.zeros(M, K, device="cuda")
    dout = torch.randint(-4, 5, (M, N), generator=gen, device="cuda").to(BF)
    nv.moe_mxfp4_product_backward(p, dout, w, off, da)
    for g in (0, 1):
        e = o[G - 1 + g]
        assert torch.equal(da[e - 300:e], dout[e - 300:e].float() @ v[g])


@pytest.mark.parametrize("mode", ["w4a16", "w4a4"])
@pytest.mark.parametrize("counts,N,K", [([3, 0, 18], 40, 4128), ([2], 33, 8192), ([17, 40], 20, 8224),
                                        ([1], 16, 65536), ([90], 16, 16384)], ids=str)
def test_long_reductions_with_few_rows(mode, counts, N, K):
    """Unit scales: products are multiples of 1/4 up to 36 (rows up to 8: 48), sums below 2^22 / 4: exact."""
    require_gpu()
    log(f"long product {mode} counts={counts} N={N} K={K}")
    gen = torch.Generator().manual_seed(K)
    off = np.concatenate([[0], np.cumsum(counts)])
    M, G = int(off[-1]), len(counts)
    wc = torch.randint(0, 256, (G, N, K // 2), generator=gen, dtype=torch.uint8)
    ws = torch.full((G, N, K // 32), 127, dtype=torch.uint8)
    w64 = mxfp4.dequantize(wc.numpy(), ws.numpy())
    w = nv.MXFP4Weights(wc.cuda(), ws.cuda())
    ac = torch.randint(0, 256, (M, K // 2), generator=gen, dtype=torch.uint8)
    as_ = torch.full((M, K // 32), 127, dtype=torch.uint8)
    a64 = mxfp4.dequantize(ac.numpy(), as_.numpy())
    a = nv.MXFP4Rows(ac.cuda(), as_.cuda()) if mode == "w4a4" else torch.from_numpy(a64).to(BF).cuda()
    out = torch.empty(M, N, device="cuda")
    p = nv.make_product_problem(M, N, K, G)
    o = torch.from_numpy(off).int().cuda()
    nv.moe_mxfp4_product(p, a, w, o, out)
    assert np.array_equal(out.double().cpu().numpy(), dispatch.product(a64, w64, off)[0])
    # the same weights as a backward of K columns
    dout = torch.randint(-8, 9, (M, N), generator=gen).to(BF)
    da = torch.empty(M, K, device="cuda")
    nv.moe_mxfp4_product_backward(p, dout.cuda(), w, o, da)
    assert np.array_equal(da.double().cpu().numpy(), dispatch.product(dout.double().numpy(), w64, off, True)[0])


@pytest.mark.parametrize("M", [5, 700])
@pytest.mark.parametrize("K", [96, 256])
def test_slices_of_weights_and_rows(M, K):
    """Experts [1, 3) of four and rows from the second on: scales at any byte."""
    require_gpu()
    log(f"sliced product M={M} K={K}")
    gen = torch.Generator().manual_seed(M + K)
    N = 51
    wc = torch.randint(0, 256, (4, N, K // 2), generator=gen, dtype=torch.uint8)
    ws = torch.randint(126, 129, (4, N, K // 32), generator=gen, dtype=torch.uint8)
    ac = torch.randint(0, 256, (M + 1, K // 2), generator=gen, dtype=torch.uint8)
    as_ = torch.randint(126, 129, (M + 1, K // 32), generator=gen, dtype=torch.uint8)
    w = nv.MXFP4Weights(wc.cuda(), ws.cuda()).slice(1, 2)
    a = nv.MXFP4Rows(ac.cuda()[1:], as_.cuda()[1:])
    off = torch.tensor([0, M // 3, M], **I32)
    out = torch.empty(M, N, device="cuda")
    nv.moe_mxfp4_product(nv.make_product_problem(M, N, K, 2), a, w, off, out)
    ref = dispatch.product(mxfp4.dequantize(ac.numpy(), as_.numpy())[1:],
                           mxfp4.dequantize(wc.numpy(), ws.numpy())[1:3], off.cpu().numpy())[0]
    assert np.array_equal(out.double().cpu().numpy(), ref)


def test_two_streams_at_once_and_an_explicit_stream():
    """Independent chains on two streams, each with its own buffers and workspace."""
    require_gpu()
    log("two streams")
    T, k, E, d = 3000, 6, 20, 512
    gen = torch.Generator(device="cuda").manual_seed(9)
    p = nv.make_dispatch_problem(T, d, E, k, 0, E)
    w = nv.quantize_mxfp4_weights(torch.randn(E, 384, d, generator=gen, device="cuda").to(BF))
    jobs = []
    for _ in range(2):
        ids = torch.rand(T, E, generator=gen, device="cuda").topk(k, 1).indices.int()
        jobs.append((ids, torch.randn(T, d, generator=gen, device="cuda").to(BF), plan_buffers(p, d),
                     torch.zeros(T * k, 384, dtype=BF, device="cuda"), nv.MXFP4Rows.empty(T * k, d),
                     nv.alloc_dispatch_workspace(p)))
    pp = nv.make_product_problem(T * k, 384, d, E)

    def chain(ids, x, b, out, q, ws, stream=None):
        nv.moe_dispatch(p, ids, x, workspace=ws, stream=stream, **b)
        nv.moe_mxfp4_quantize(b["rows"], q.codes, q.scales, stream=stream)
        nv.moe_mxfp4_product(pp, q, w, b["offsets"], out, stream=stream)

    refs = []
    for j in jobs:
        chain(*j)
        torch.cuda.synchronize()
        refs.append([t.clone() for t in (*j[2].values(), j[3])])
    streams = [torch.cuda.Stream() for _ in range(2)]
    for r in range(3):
        for j in jobs:
            for t in (*j[2].values(), j[3]):
                t.zero_()
        torch.cuda.synchronize()
        for s, j in zip(streams, jobs):
            chain(*j, stream=s)
        torch.cuda.synchronize()
        for j, ref in zip(jobs, refs):
            for i, (t, want) in enumerate(zip((*j[2].values(), j[3]), ref)):
                assert torch.equal(t, want), (r, i)


def test_one_workspace_under_two_graphs():
    require_gpu()
    log("two graphs, one workspace")
    T, k, E = 4000, 8, 32
    ps = [nv.make_dispatch_problem(T, 64, E, k, 0, E), nv.make_dispatch_problem(T - 500, 64, E, k, 8, 16)]
    ws = torch.empty(max(nv.moe_dispatch_workspace_size(p) for p in ps), dtype=torch.uint8, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(2)
    graphs = []
    for p in ps:
        ids = torch.zeros(p.num_tokens, k, **I32)
        x = torch.randn(p.num_tokens, 64, generator=gen, device="cuda").to(BF)
        b = plan_buffers(p, 64)
        nv.moe_dispatch(p, ids, x, workspace=ws, **b)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            nv.moe_dispatch(p, ids, x, workspace=ws, **b)
        graphs.append((p, ids, b, g))
    for r in range(3):
        for p, ids, b, g in graphs:
            ids.copy_(torch.rand(p.num_tokens, E, generator=gen, device="cuda").topk(k, 1).indices)
        for _, _, _, g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for p, ids, b, g in graphs:
            c, o, pm, iv = dispatch.plan(ids.cpu().numpy(), p.local_expert_offset, p.num_local_experts)
            assert np.array_equal(b["inv"].cpu().numpy(), iv) and np.array_equal(b["offsets"].cpu().numpy(), o), r


def _ragged(G, seed):
    """Rows of G groups: empty ones, a few rows, tile edges and beyond; their offsets."""
    gen = torch.Generator().manual_seed(seed)
    pick = torch.tensor([0, 1, 31, 33, 128, 129, 255, 256, 257, 400, 512, 700])
    counts = pick[torch.randint(0, len(pick), (G,), generator=gen)]
    return torch.cat([torch.zeros(1, dtype=torch.int64), counts.cumsum(0)])


def _mx_values(codes, scales):
    out = torch.empty(codes.shape[0], codes.shape[1] * 2, device="cuda")
    return nv.moe_mxfp4_dequantize(codes, scales, out)


@pytest.mark.parametrize("mode", ["w4a16", "w4a4"])
@pytest.mark.parametrize("K", [32, 96, 128, 256, 288, 384, 512, 640])
def test_tiles_one_after_another_of_few_stages(mode, K):
    """About 1000 tiles, several a workgroup, of one to a few stages each.  Exact: with |a| <= 12,
    |w| <= 12 products are multiples of 1/16 and sums of 640 below 2^17, so fp32 holds them."""
    require_gpu()
    log(f"{mode} many tiles K={K}")
    gen = torch.Generator(device="cuda").manual_seed(K)
    G, N = 90, 1100
    off = _ragged(G, K)
    M = int(off[-1])
    u8 = dict(dtype=torch.uint8, device="cuda", generator=gen)
    w = nv.MXFP4Weights(torch.randint(0, 256, (G, N, K // 2), **u8), torch.randint(126, 129, (G, N, K // 32), **u8))
    if mode == "w4a4":
        a = nv.MXFP4Rows(torch.randint(0, 256, (M, K // 2), **u8), torch.randint(126, 129, (M, K // 32), **u8))
        av = _mx_values(a.codes, a.scales)
    else:
        av = torch.randint(-8, 9, (M, K), generator=gen, device="cuda").float()
        a = av.to(BF)
    out = torch.full((M, N), 55.0, device="cuda")
    nv.moe_mxfp4_product(nv.make_product_problem(M, N, K, G), a, w, off.int().cuda(), out)
    for g in range(G):
        b, e = int(off[g]), int(off[g + 1])
        if e > b:
            want = av[b:e] @ _mx_values(w.codes[g], w.scales[g]).t().contiguous()
            assert torch.equal(out[b:e], want), (g, b, e)


@pytest.mark.parametrize("N", [8, 13, 64, 72, 136, 200, 264])
def test_gradient_tiles_one_after_another_of_few_stages(N):
    """The same for the gradient (|dout| <= 8, |w| <= 12)."""
    require_gpu()
    log(f"gradient many tiles N={N}")
    gen = torch.Generator(device="cuda").manual_seed(N)
    G, K = 90, 1120
    off = _ragged(G, N)
    M = int(off[-1])
    u8 = dict(dtype=torch.uint8, device="cuda", generator=gen)
    w = nv.MXFP4Weights(torch.randint(0, 256, (G, N, K // 2), **u8), torch.randint(126, 129, (G, N, K // 32), **u8))
    dv = torch.randint(-8, 9, (M, N), generator=gen, device="cuda").float()
    out = torch.full((M, K), 55.0, device="cuda")
    nv.moe_mxfp4_product_backward(nv.make_product_problem(M, N, K, G), dv.to(BF), w, off.int().cuda(), out)
    for g in range(G):
        b, e = int(off[g]), int(off[g + 1])
        if e > b:
            assert torch.equal(out[b:e], dv[b:e] @ _mx_values(w.codes[g], w.scales[g])), (g, b, e)

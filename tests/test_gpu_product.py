"""GPU parity of the grouped MXFP4 products with the fp64 oracle.

Exact cases: scales 2^-1 .. 2^1 and small integer rows (or MXFP4 rows of such
scales) make every product a multiple of 1/16 and every partial sum less than 2^20,
so fp32 holds all of them and the fp32 outputs must equal the oracle's, whatever
the order.  Real-valued cases: n products summed in fp32 are off by at most n u'
sum |a w|, u' = 2^-23 (an adder may truncate), and the result is rounded once."""
import numpy as np
import pytest
import torch

import nvfp4_expert_layer_amd as nv
from oracle import dispatch, mxfp4
from tests.gpu_helpers import log, require_gpu

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
REAL = dict(lo=110, hi=130)


def f64(t):
    return t.double().cpu().numpy()


def mx_random(gen, *shape, lo=126, hi=128):
    codes = torch.randint(0, 256, (*shape[:-1], shape[-1] // 2), generator=gen, dtype=torch.uint8)
    scales = torch.randint(lo, hi + 1, (*shape[:-1], shape[-1] // 32), generator=gen, dtype=torch.uint8)
    return codes, scales


def bounds(counts, lead=0):
    return np.concatenate([[lead], lead + np.cumsum(counts)]).astype(np.int64)


def forward(mode, counts, N, K, out_dtype=torch.float32, lead=0, tail=0, seed=0, real=False, a_pad=0, out_pad=0,
            unaligned_scales=False):
    """Runs one product; returns (out, reference, sum of magnitudes, first and last row)."""
    gen = torch.Generator().manual_seed(seed)
    off = bounds(counts, lead)
    M, G = int(off[-1]) + tail, len(counts)
    wc, ws = mx_random(gen, G, N, K, **REAL if real else {})
    w64 = mxfp4.dequantize(wc.numpy(), ws.numpy())
    ws_g = ws.cuda()
    if unaligned_scales:
        buf = torch.empty(ws.numel() + 1, dtype=torch.uint8, device="cuda")
        ws_g = buf[1:].view(ws.shape)
        ws_g.copy_(ws)
    w = nv.MXFP4Weights(wc.cuda(), ws_g)
    if mode == "w4a4":
        ac, as_ = mx_random(gen, M, K, **REAL if real else {})
        a64 = mxfp4.dequantize(ac.numpy(), as_.numpy())
        as_g = as_.cuda()
        if lead or tail:                                         # rows of no group: NaN scales
            as_g[:lead] = 255
            as_g[M - tail:] = 255
        a = nv.MXFP4Rows(ac.cuda(), as_g)
    else:
        av = torch.randn(M, K, generator=gen) if real else torch.randint(-8, 9, (M, K), generator=gen).float()
        av = av.to(BF)
        a64 = f64(av)
        a = torch.full((M, K + a_pad), float("nan"), dtype=BF, device="cuda")[:, :K]
        a.copy_(av)
        a[:lead] = float("nan")
        a[M - tail:] = float("nan")
    out = torch.full((M, N + out_pad), 55.0, dtype=out_dtype, device="cuda")[:, :N]
    p = nv.make_product_problem(M, N, K, G)
    nv.moe_mxfp4_product(p, a, w, torch.from_numpy(off).int().cuda(), out)
    torch.cuda.synchronize()
    ref, mag = dispatch.product(a64, w64, off)
    assert (out[:lead] == 55).all() and (out[M - tail:] == 55).all() if lead or tail else True
    if out_pad:
        assert (out._base[:, N:] == 55).all()
    return out, ref, mag, int(off[0]), int(off[-1])


# rows per group: none, one, tile edges, many (both kernels' ranges)
COUNTS = [[1], [0, 1, 0], [16, 17, 0, 33], [64, 65, 3], [0, 0, 128, 0], [300, 0, 70, 257], [1000], [255, 256, 513]]


@pytest.mark.parametrize("mode", ["w4a16", "w4a4"])
@pytest.mark.parametrize("counts", COUNTS, ids=str)
@pytest.mark.parametrize("N,K", [(1, 32), (16, 256), (100, 96), (257, 288), (512, 1056), (40, 2080), (256, 512)])
def test_exact_sums(mode, counts, N, K):
    require_gpu()
    log(f"product {mode} counts={counts} N={N} K={K}")
    out, ref, _, b, e = forward(mode, counts, N, K, seed=N + K)
    assert np.array_equal(f64(out)[b:e], ref[b:e])


@pytest.mark.parametrize("mode", ["w4a16", "w4a4"])
@pytest.mark.parametrize("dtype", [BF, torch.float16, torch.float32])
@pytest.mark.parametrize("counts", [[5, 0, 20], [200, 130, 0, 300]], ids=str)
def test_types_strides_and_rows_of_no_group(mode, dtype, counts):
    require_gpu()
    log(f"product {mode} {dtype} counts={counts}")
    for N, K, a_pad, out_pad, un in ((96, 160, 8, 0, False), (128, 512, 64, 8, False), (100, 128, 0, 3, True),
                                     (33, 1024, 0, 1, True)):
        out, ref, _, b, e = forward(mode, counts, N, K, dtype, lead=7, tail=9, seed=K, a_pad=a_pad, out_pad=out_pad,
                                    unaligned_scales=un)
        # the fp32 sum is exact: one rounding, the same as torch's
        want = torch.from_numpy(ref[b:e]).float().to(dtype)
        assert torch.equal(out[b:e].cpu(), want)


@pytest.mark.parametrize("mode", ["w4a16", "w4a4"])
@pytest.mark.parametrize("counts,N,K", [([1], 300, 4096), ([3, 0, 40], 64, 4096), ([500, 90], 200, 4128)], ids=str)
def test_real_values(mode, counts, N, K):
    require_gpu()
    log(f"product real {mode} counts={counts} N={N} K={K}")
    out, ref, mag, b, e = forward(mode, counts, N, K, seed=1, real=True)
    err = np.abs(f64(out)[b:e] - ref[b:e])
    assert (err <= K * 2.0 ** -23 * mag[b:e]).all()


@pytest.mark.parametrize("mode", ["w4a16", "w4a4"])
@pytest.mark.parametrize("M", [3, 300])
def test_nan_blocks_reach_their_outputs_alone(mode, M):
    require_gpu()
    log(f"product NaN {mode} M={M}")
    gen = torch.Generator().manual_seed(M)
    N, K = 70, 96
    wc, ws = mx_random(gen, 1, N, K)
    ws[0, 17, 1] = 255
    ac, as_ = mx_random(gen, M, K)
    a = nv.MXFP4Rows(ac.cuda(), as_.cuda())
    if mode == "w4a16":
        a = torch.from_numpy(mxfp4.dequantize(ac.numpy(), as_.numpy())).to(BF).cuda()
        a[2, 5] = float("nan")
    else:
        a.scales[2, 0] = 255
    out = torch.empty(M, N, device="cuda")
    nv.moe_mxfp4_product(nv.make_product_problem(M, N, K), a, nv.MXFP4Weights(wc.cuda(), ws.cuda()), None, out)
    nan = torch.isnan(out).cpu()
    want = torch.zeros(M, N, dtype=torch.bool)
    want[2], want[:, 17] = True, True
    assert torch.equal(nan, want)


def backward(counts, N, K, out_dtype=torch.float32, lead=0, tail=0, seed=0, pad=0, out_pad=0, real=False):
    gen = torch.Generator().manual_seed(seed)
    off = bounds(counts, lead)
    M, G = int(off[-1]) + tail, len(counts)
    wc, ws = mx_random(gen, G, N, K, **REAL if real else {})
    dv = (torch.randn(M, N, generator=gen) if real else torch.randint(-8, 9, (M, N), generator=gen).float()).to(BF)
    dout = torch.full((M, N + pad), float("nan"), dtype=BF, device="cuda")[:, :N]
    dout.copy_(dv)
    dout[:lead] = float("nan")
    dout[M - tail:] = float("nan")
    out = torch.full((M, K + out_pad), 55.0, dtype=out_dtype, device="cuda")[:, :K]
    nv.moe_mxfp4_product_backward(nv.make_product_problem(M, N, K, G), dout, nv.MXFP4Weights(wc.cuda(), ws.cuda()),
                                  torch.from_numpy(off).int().cuda(), out)
    torch.cuda.synchronize()
    ref, mag = dispatch.product(f64(dv), mxfp4.dequantize(wc.numpy(), ws.numpy()), off, backward=True)
    assert (out[:lead] == 55).all() and (out[M - tail:] == 55).all() if lead or tail else True
    if out_pad:
        assert (out._base[:, K:] == 55).all()
    return out, ref, mag, int(off[0]), int(off[-1])


@pytest.mark.parametrize("counts", COUNTS, ids=str)
@pytest.mark.parametrize("N,K", [(1, 32), (8, 256), (100, 96), (257, 288), (512, 1056), (264, 128), (1000, 160)])
def test_backward_exact_sums(counts, N, K):
    require_gpu()
    log(f"product backward counts={counts} N={N} K={K}")
    out, ref, _, b, e = backward(counts, N, K, seed=N + K)
    assert np.array_equal(f64(out)[b:e], ref[b:e])


@pytest.mark.parametrize("dtype", [BF, torch.float16, torch.float32])
@pytest.mark.parametrize("counts", [[5, 0, 20], [200, 130, 0, 300]], ids=str)
def test_backward_types_strides_and_rows_of_no_group(dtype, counts):
    require_gpu()
    log(f"product backward {dtype} counts={counts}")
    for N, K, pad, out_pad in ((96, 160, 8, 0), (128, 512, 3, 8), (101, 128, 0, 3), (40, 1056, 1, 1)):
        out, ref, _, b, e = backward(counts, N, K, dtype, lead=7, tail=9, seed=K, pad=pad, out_pad=out_pad)
        assert torch.equal(out[b:e].cpu(), torch.from_numpy(ref[b:e]).float().to(dtype))


@pytest.mark.parametrize("counts,N,K", [([1], 2048, 300 // 32 * 32), ([3, 0, 40], 2048, 64), ([500, 90], 1001, 224)],
                         ids=str)
def test_backward_real_values(counts, N, K):
    require_gpu()
    log(f"product backward real counts={counts} N={N} K={K}")
    out, ref, mag, b, e = backward(counts, N, K, seed=1, real=True)
    assert (np.abs(f64(out)[b:e] - ref[b:e]) <= N * 2.0 ** -23 * mag[b:e]).all()


def test_backward_is_the_forward_s_gradient_by_differences():
    """The forward is linear in its rows: out(a + h) - out(a) along one element equals that row of the
    weight, and its sum against dout the element's gradient (exact sums: integers)."""
    require_gpu()
    log("product gradient by differences")
    gen = torch.Generator().manual_seed(5)
    M, N, K = 40, 24, 64
    wc, ws = mx_random(gen, 2, N, K)
    w = nv.MXFP4Weights(wc.cuda(), ws.cuda())
    off = torch.tensor([0, 19, 40], dtype=torch.int32, device="cuda")
    p = nv.make_product_problem(M, N, K, 2)
    a = torch.randint(-8, 9, (M, K), generator=gen).to(BF).cuda()
    dout = torch.randint(-8, 9, (M, N), generator=gen).to(BF).cuda()
    da, base, moved = torch.empty(M, K, device="cuda"), torch.empty(M, N, device="cuda"), torch.empty(M, N, device="cuda")
    nv.moe_mxfp4_product_backward(p, dout, w, off, da)
    nv.moe_mxfp4_product(p, a, w, off, base)
    for k in range(0, K, 7):
        b = a.clone()
        b[:, k] += 2
        nv.moe_mxfp4_product(p, b, w, off, moved)
        diff = ((moved - base) * dout.float()).sum(1) / 2
        assert torch.equal(diff, da[:, k])


@pytest.mark.parametrize("M", [4, 600])
def test_offsets_beyond_the_rows_are_clamped(M):
    require_gpu()
    log(f"product clamped offsets M={M}")
    gen = torch.Generator().manual_seed(M)
    wc, ws = mx_random(gen, 3, 32, 64)
    w64 = mxfp4.dequantize(wc.numpy(), ws.numpy())
    w = nv.MXFP4Weights(wc.cuda(), ws.cuda())
    a = torch.randint(-8, 9, (M, 64), generator=gen).to(BF)
    off = torch.tensor([-9, 2, M + 100, M + 2 ** 20], dtype=torch.int32)
    p = nv.make_product_problem(M, 32, 64, 3)
    out, da = torch.empty(M, 32, device="cuda"), torch.empty(M, 64, device="cuda")
    nv.moe_mxfp4_product(p, a.cuda(), w, off.cuda(), out)
    nv.moe_mxfp4_product_backward(p, a[:, :32].contiguous().cuda(), w, off.cuda(), da)
    b = np.clip(off.numpy(), 0, M)
    assert np.array_equal(f64(out), dispatch.product(f64(a), w64, b)[0])
    assert np.array_equal(f64(da), dispatch.product(f64(a[:, :32]), w64, b, backward=True)[0])


@pytest.mark.parametrize("M,G", [(3, 200), (50, 64), (2000, 6)])
def test_few_rows_many_groups_repeats_and_graph_replays(M, G):
    require_gpu()
    log(f"product graph M={M} G={G}")
    gen = torch.Generator().manual_seed(M)
    N, K = 144, 256
    wc, ws = mx_random(gen, G, N, K, lo=100, hi=140)
    w = nv.MXFP4Weights(wc.cuda(), ws.cuda())
    p = nv.make_product_problem(M, N, K, G)

    def new():
        cuts = torch.randint(0, M + 1, (G - 1,), generator=gen).sort().values
        return torch.cat([torch.tensor([0]), cuts, torch.tensor([M])]).int().cuda(), \
            torch.randn(M, K, generator=gen).to(BF).cuda()

    off, a = new()
    q = nv.MXFP4Rows.empty(M, K)
    outs = [torch.empty(M, N, dtype=BF, device="cuda") for _ in range(2)] + [torch.empty(M, K, dtype=BF, device="cuda")]

    def step(q, o):
        nv.moe_mxfp4_product(p, a, w, off, o[0])
        nv.moe_mxfp4_quantize(a, q.codes, q.scales)
        nv.moe_mxfp4_product(p, q, w, off, o[1])
        nv.moe_mxfp4_product_backward(p, o[0], w, off, o[2])

    step(q, outs)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(q, outs)
    for r in range(3):
        o2, a2 = new()
        off.copy_(o2)
        a.copy_(a2)
        for o in outs:
            o.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        eager = [torch.empty_like(o) for o in outs]
        step(nv.MXFP4Rows.empty(M, K), eager)
        torch.cuda.synchronize()
        for o, e in zip(outs, eager):
            assert torch.equal(o, e) and torch.isfinite(o).all(), r

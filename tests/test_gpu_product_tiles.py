"""The products' tile kernels against the fp64 oracle; every shape is held against the library's
own rule first, so that none of these can move to the streaming kernels unnoticed.

Exact cases, as in test_gpu_product: integer rows up to 8 (or MXFP4 rows up to 12) times weights
up to 12 are multiples of 1/16, and the K of these cases keep every partial sum below 2^20, so
that fp32 holds all of them: 144 * 7168 = 1032192 < 2^20 = 1048576."""
import numpy as np
import pytest
import torch

import nvfp4_expert_layer_amd as nv
from oracle import dispatch, mxfp4
from tests.gpu_helpers import log, require_gpu
from tests.product_choice import streams
from tests.test_gpu_product import BF, backward, f64, forward, mx_random

pytestmark = pytest.mark.gpu

# empty groups, one row, tile edges, more than two tiles
RAGGED = [300, 0, 257, 256, 255, 700, 1, 513]


def on_tiles(*shape, **kw):
    assert not streams(*shape, **kw), shape


@pytest.mark.parametrize("mode", ["w4a16", "w4a4"])
@pytest.mark.parametrize("dtype", [BF, torch.float16, torch.float32])
@pytest.mark.parametrize("N,K,a_pad,out_pad,unaligned", [
    (96, 160, 8, 0, False), (128, 512, 64, 8, False), (100, 128, 0, 3, True), (33, 1024, 0, 1, True),
    (250, 288, 8, 5, True), (257, 96, 0, 0, False), (1, 32, 16, 2, False), (510, 256, 0, 1, False),
    (24, 7168, 0, 0, False)])
def test_types_strides_and_rows_of_no_group(mode, dtype, N, K, a_pad, out_pad, unaligned):
    require_gpu()
    log(f"tiles {mode} {dtype} N={N} K={K}")
    on_tiles(mode, sum(RAGGED) + 16, N, K, len(RAGGED), stride=K + a_pad if mode == "w4a16" else K)
    out, ref, _, b, e = forward(mode, RAGGED, N, K, dtype, lead=7, tail=9, seed=K, a_pad=a_pad, out_pad=out_pad,
                                unaligned_scales=unaligned)
    # the fp32 sum is exact: one rounding, the same as torch's
    assert torch.equal(out[b:e].cpu(), torch.from_numpy(ref[b:e]).float().to(dtype))


@pytest.mark.parametrize("mode", ["w4a16", "w4a4"])
@pytest.mark.parametrize("N,K", [(200, 4128), (64, 2048)])
def test_real_values(mode, N, K):
    require_gpu()
    log(f"tiles real {mode} N={N} K={K}")
    on_tiles(mode, sum(RAGGED), N, K, len(RAGGED))
    out, ref, mag, b, e = forward(mode, RAGGED, N, K, seed=1, real=True)
    assert (np.abs(f64(out)[b:e] - ref[b:e]) <= K * 2.0 ** -23 * mag[b:e]).all()


@pytest.mark.parametrize("dtype", [BF, torch.float16, torch.float32])
@pytest.mark.parametrize("N,K,pad,out_pad", [(96, 160, 8, 0), (128, 512, 3, 8), (101, 128, 0, 3), (40, 1056, 1, 1),
                                             (264, 224, 0, 2), (1, 32, 0, 0)])
def test_backward_types_strides_and_rows_of_no_group(dtype, N, K, pad, out_pad):
    require_gpu()
    log(f"gradient tiles {dtype} N={N} K={K}")
    on_tiles("backward", sum(RAGGED) + 16, N, K, len(RAGGED), stride=N + pad)
    out, ref, _, b, e = backward(RAGGED, N, K, dtype, lead=7, tail=9, seed=K, pad=pad, out_pad=out_pad)
    assert torch.equal(out[b:e].cpu(), torch.from_numpy(ref[b:e]).float().to(dtype))


@pytest.mark.parametrize("N,K", [(1001, 224), (2048, 64)])
def test_backward_real_values(N, K):
    require_gpu()
    log(f"gradient tiles real N={N} K={K}")
    on_tiles("backward", sum(RAGGED), N, K, len(RAGGED))
    out, ref, mag, b, e = backward(RAGGED, N, K, seed=1, real=True)
    assert (np.abs(f64(out)[b:e] - ref[b:e]) <= N * 2.0 ** -23 * mag[b:e]).all()


@pytest.mark.parametrize("mode", ["w4a16", "w4a4", "backward"])
@pytest.mark.parametrize("K", [96, 256])
def test_nan_reaches_its_outputs_alone(mode, K):
    """One weight block and one row element (block) of two groups are NaN."""
    require_gpu()
    log(f"tiles NaN {mode} K={K}")
    gen = torch.Generator().manual_seed(K)
    N, G, rows = 70, 8, 290
    M = G * rows
    on_tiles(mode, M, N, K, G)
    off = torch.arange(0, M + 1, rows, dtype=torch.int32).cuda()
    wc, ws = mx_random(gen, G, N, K)
    ws[5, 17, 1] = 255
    w, p = nv.MXFP4Weights(wc.cuda(), ws.cuda()), nv.make_product_problem(M, N, K, G)
    width = N if mode != "backward" else K
    out, want = torch.empty(M, width, device="cuda"), torch.zeros(M, width, dtype=torch.bool)
    row = 3 * rows + 261                                          # the second tile of its group
    want[row] = True
    if mode == "backward":
        d = torch.randint(-8, 9, (M, N), generator=gen).to(BF)
        d[row, 5] = float("nan")
        want[5 * rows:6 * rows, 32:64] = True
        nv.moe_mxfp4_product_backward(p, d.cuda(), w, off, out)
    else:
        want[5 * rows:6 * rows, 17] = True
        ac, as_ = mx_random(gen, M, K)
        if mode == "w4a4":
            as_[row, 2] = 255
            a = nv.MXFP4Rows(ac.cuda(), as_.cuda())
        else:
            a = torch.from_numpy(mxfp4.dequantize(ac.numpy(), as_.numpy())).to(BF)
            a[row, 5] = float("nan")
            a = a.cuda()
        nv.moe_mxfp4_product(p, a, w, off, out)
    assert torch.equal(torch.isnan(out).cpu(), want)


def test_offsets_beyond_the_rows_are_clamped():
    require_gpu()
    log("tiles clamped offsets")
    gen = torch.Generator().manual_seed(8)
    M, N, K, G = 2300, 32, 64, 8
    for mode in ("w4a16", "w4a4", "backward"):
        on_tiles(mode, M, N, K, G)
    wc, ws = mx_random(gen, G, N, K)
    w64, w = mxfp4.dequantize(wc.numpy(), ws.numpy()), nv.MXFP4Weights(wc.cuda(), ws.cuda())
    off = torch.tensor([-9, 300, 600, 600, 1200, 1500, 1800, M + 100, M + 2 ** 20], dtype=torch.int32)
    b, p = np.clip(off.numpy(), 0, M), nv.make_product_problem(M, N, K, G)
    a = torch.randint(-8, 9, (M, K), generator=gen).to(BF)
    ac, as_ = mx_random(gen, M, K)
    out, da = torch.empty(M, N, device="cuda"), torch.empty(M, K, device="cuda")
    nv.moe_mxfp4_product(p, a.cuda(), w, off.cuda(), out)
    assert np.array_equal(f64(out), dispatch.product(f64(a), w64, b)[0])
    q = nv.MXFP4Rows(ac.cuda(), as_.cuda())
    nv.moe_mxfp4_product(p, q, w, off.cuda(), out)
    assert np.array_equal(f64(out), dispatch.product(mxfp4.dequantize(ac.numpy(), as_.numpy()), w64, b)[0])
    d = a[:, :N].contiguous()
    nv.moe_mxfp4_product_backward(p, d.cuda(), w, off.cuda(), da)
    assert np.array_equal(f64(da), dispatch.product(f64(d), w64, b, backward=True)[0])


@pytest.mark.parametrize("K,shift", [(96, 0), (160, 0), (128, 1), (128, 3), (384, 2), (512, 4)])
@pytest.mark.parametrize("dtype", [BF, torch.float32])
def test_scales_of_both_operands_at_any_byte(K, shift, dtype):
    """W4A4 over experts [1, 9) of nine and rows from the second on, both scale tensors `shift`
    bytes past an aligned address."""
    require_gpu()
    log(f"tiles scales at any byte K={K} shift={shift} {dtype}")
    gen = torch.Generator().manual_seed(K + shift)
    N, G = 51, 8
    off = np.concatenate([[0], np.cumsum(RAGGED)])
    M = int(off[-1])

    def shifted(s):
        buf = torch.empty(s.numel() + shift, dtype=torch.uint8, device="cuda")
        view = buf[shift:].view(s.shape)
        return view.copy_(s)

    wc, ws = mx_random(gen, G + 1, N, K)
    ac, as_ = mx_random(gen, M + 1, K)
    w = nv.MXFP4Weights(wc.cuda(), shifted(ws)).slice(1, G)
    a = nv.MXFP4Rows(ac.cuda()[1:], shifted(as_)[1:])
    out = torch.empty(M, N, dtype=dtype, device="cuda")
    on_tiles("w4a4", M, N, K, G)
    nv.moe_mxfp4_product(nv.make_product_problem(M, N, K, G), a, w, torch.from_numpy(off).int().cuda(), out)
    ref = dispatch.product(mxfp4.dequantize(ac.numpy(), as_.numpy())[1:],
                           mxfp4.dequantize(wc.numpy(), ws.numpy())[1:], off)[0]
    assert torch.equal(out.cpu(), torch.from_numpy(ref).float().to(dtype))


@pytest.mark.parametrize("stride,tiles", [(2 ** 22, True), (2 ** 22 + 8, False)])
def test_rows_as_far_apart_as_the_tiles_reach(stride, tiles):
    """300 rows at the largest stride that the tiles' 32-bit lane offsets take, and past it (2.5 GB a
    tensor); outputs at the same stride."""
    require_gpu()
    log(f"rows {stride} elements apart")
    gen = torch.Generator().manual_seed(stride % 97)
    M, N, K = 300, 40, 256
    wc, ws = mx_random(gen, 1, N, K)
    w64, w = mxfp4.dequantize(wc.numpy(), ws.numpy()), nv.MXFP4Weights(wc.cuda(), ws.cuda())
    wide = [torch.full((M * stride,), 3.0, dtype=BF, device="cuda").view(M, stride) for _ in range(2)]
    av = torch.randint(-8, 9, (M, K), generator=gen).to(BF)
    a, out = wide[0][:, :K], wide[1][:, 64:64 + N]
    a.copy_(av)
    p = nv.make_product_problem(M, N, K)
    off = np.array([0, M])
    for mode in ("w4a16", "backward"):
        assert streams(mode, M, N, K, 1, stride=stride) != tiles
    nv.moe_mxfp4_product(p, a, w, None, out)
    want = torch.from_numpy(dispatch.product(f64(av), w64, off)[0]).float().to(BF)
    assert torch.equal(out.cpu(), want)
    assert (wide[1][:, :64] == 3).all() and (wide[1][:, 64 + N:64 + N + 256] == 3).all()
    dv = torch.randint(-8, 9, (M, N), generator=gen).to(BF)
    d, da = wide[0][:, 8:8 + N], wide[1][:, 1000:1000 + K]
    d.copy_(dv)
    nv.moe_mxfp4_product_backward(p, d, w, None, da)
    want = torch.from_numpy(dispatch.product(f64(dv), w64, off, backward=True)[0]).float().to(BF)
    assert torch.equal(da.cpu(), want)
    if tiles:                                                      # an odd stride: element by element
        odd = wide[0].view(-1)[:M * (stride - 1)].view(M, stride - 1)[:, 5:5 + N]
        odd.copy_(dv)
        nv.moe_mxfp4_product_backward(p, odd, w, None, da.zero_())
        assert torch.equal(da.cpu(), want)


def tile_count(off, width):
    c = off[1:] - off[:-1]
    return int(((c + 255) // 256).sum()) * ((width + 255) // 256)


def many_tiles(seed):
    """Offsets of 180 groups: empty ones, a few rows, tile edges and beyond."""
    gen = torch.Generator().manual_seed(seed)
    pick = torch.tensor([0, 1, 31, 33, 128, 129, 255, 256, 257, 400, 512, 700])
    counts = pick[torch.randint(0, len(pick), (180,), generator=gen)]
    return torch.cat([torch.zeros(1, dtype=torch.int64), counts.cumsum(0)])


def values(codes, scales):
    return nv.moe_mxfp4_dequantize(codes, scales, torch.empty(codes.shape[0], codes.shape[1] * 2, device="cuda"))


@pytest.mark.parametrize("K", [32, 128, 256, 288, 384, 640, 768])
def test_a_workgroup_takes_five_tiles_or_more(K):
    """W4A4: at least 5 tiles for each of the CUs (the rings and scale pairs turn over many tiles).
    |a|, |w| <= 12: sums of 768 products are below 2^17 and multiples of 1/16, exact in fp32."""
    require_gpu()
    log(f"w4a4 five tiles a workgroup K={K}")
    gen = torch.Generator(device="cuda").manual_seed(K)
    off, N, G = many_tiles(K), 2200, 180
    M = int(off[-1])
    assert tile_count(off, N) >= 5 * torch.cuda.get_device_properties(0).multi_processor_count
    u8 = dict(dtype=torch.uint8, device="cuda", generator=gen)
    w = nv.MXFP4Weights(torch.randint(0, 256, (G, N, K // 2), **u8), torch.randint(126, 129, (G, N, K // 32), **u8))
    a = nv.MXFP4Rows(torch.randint(0, 256, (M, K // 2), **u8), torch.randint(126, 129, (M, K // 32), **u8))
    av, out = values(a.codes, a.scales), torch.full((M, N), 55.0, device="cuda")
    on_tiles("w4a4", M, N, K, G)
    nv.moe_mxfp4_product(nv.make_product_problem(M, N, K, G), a, w, off.int().cuda(), out)
    for g in range(G):
        b, e = int(off[g]), int(off[g + 1])
        if e > b:
            assert torch.equal(out[b:e], av[b:e] @ values(w.codes[g], w.scales[g]).t().contiguous()), (g, b, e)


@pytest.mark.parametrize("N", [8, 13, 64, 136, 200, 264])
def test_a_workgroup_takes_five_gradient_tiles_or_more(N):
    """The same for the gradient (|dout| <= 8, |w| <= 12)."""
    require_gpu()
    log(f"gradient five tiles a workgroup N={N}")
    gen = torch.Generator(device="cuda").manual_seed(N)
    off, K, G = many_tiles(N), 2208, 180
    M = int(off[-1])
    assert tile_count(off, K) >= 5 * torch.cuda.get_device_properties(0).multi_processor_count
    u8 = dict(dtype=torch.uint8, device="cuda", generator=gen)
    w = nv.MXFP4Weights(torch.randint(0, 256, (G, N, K // 2), **u8), torch.randint(126, 129, (G, N, K // 32), **u8))
    dv = torch.randint(-8, 9, (M, N), generator=gen, device="cuda").float()
    d, out = dv.to(BF), torch.full((M, K), 55.0, device="cuda")
    on_tiles("backward", M, N, K, G)
    nv.moe_mxfp4_product_backward(nv.make_product_problem(M, N, K, G), d, w, off.int().cuda(), out)
    for g in range(G):
        b, e = int(off[g]), int(off[g + 1])
        if e > b:
            assert torch.equal(out[b:e], dv[b:e] @ values(w.codes[g], w.scales[g])), (g, b, e)


@pytest.mark.parametrize("mode", ["w4a16", "w4a4", "backward"])
@pytest.mark.parametrize("G", [513, 1023, 1024])
def test_as_many_groups_as_there_can_be(mode, G):
    """Exact sums, every group."""
    require_gpu()
    log(f"tiles {mode} G={G}")
    gen = torch.Generator(device="cuda").manual_seed(G)
    N, K = (40, 128) if mode != "backward" else (24, 96)
    counts = torch.randint(0, 120, (G,), generator=gen, device="cuda")
    counts[G // 2], counts[G - 1] = 600, 300
    off = torch.cat([torch.zeros(1, dtype=torch.int64, device="cuda"), counts.cumsum(0)])
    M = int(off[-1])
    on_tiles(mode, M, N, K, G)
    u8 = dict(dtype=torch.uint8, device="cuda", generator=gen)
    w = nv.MXFP4Weights(torch.randint(0, 256, (G, N, K // 2), **u8), torch.randint(126, 129, (G, N, K // 32), **u8))
    v = values(w.codes.view(G * N, K // 2), w.scales.view(G * N, K // 32)).view(G, N, K)
    p, width = nv.make_product_problem(M, N, K, G), N if mode == "backward" else K
    a = av = torch.randint(-8, 9, (M, width), generator=gen, device="cuda").to(BF)
    if mode == "w4a4":
        a = nv.MXFP4Rows(torch.randint(0, 256, (M, K // 2), **u8), torch.randint(126, 129, (M, K // 32), **u8))
        av = values(a.codes, a.scales)
    out = torch.full((M, K if mode == "backward" else N), 55.0, device="cuda")
    if mode == "backward":
        nv.moe_mxfp4_product_backward(p, a, w, off.int(), out)
    else:
        nv.moe_mxfp4_product(p, a, w, off.int(), out)
    bounds = off.tolist()
    for g in range(G):
        b, e = bounds[g], bounds[g + 1]
        if e > b:
            want = av[b:e].float() @ (v[g] if mode == "backward" else v[g].t().contiguous())
            assert torch.equal(out[b:e], want), (g, b, e)

"""GPU parity of the W4A8 product with fp64 products of the values that the codes stand for."""
import numpy as np
import pytest
import torch

import nvfp4_expert_layer_amd as nv
from oracle import block, mxfp4
from tests.gpu_helpers import log, require_gpu

pytestmark = pytest.mark.gpu


def weights(G, N, K, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return nv.quantize_mxfp4_weights(torch.randn(G, N, K, generator=g, device="cuda") * K ** -0.5)


def rows(M, K, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(M, K, generator=g, device="cuda")
    x[:, ::64] *= 8
    q = nv.MXFP8Rows.empty(M, K)
    nv.moe_mxfp8_quantize(x, q.codes, q.scales)
    return q


def values(q, w):
    f = lambda t: torch.from_numpy(t).cuda()  # noqa: E731
    return (f(block.mxfp8_dequantize(q.codes.cpu().numpy(), q.scales.cpu().numpy())),
            f(mxfp4.dequantize(w.codes.cpu().numpy(), w.scales.cpu().numpy())))


def bound(a, w):
    """What the matrix cores may lose on a [m, K] . w [n, K]^T: each product up to 2^-13 of the largest of
    its eight (of its block, at most), and fp32 sums of K / 8 terms."""
    top = lambda v: v.abs().unflatten(-1, (-1, 32)).amax(-1)  # noqa: E731
    aligned = 32 * 2.0 ** -13 * (top(a) @ top(w).t().contiguous())
    return aligned + (a.shape[1] / 8 + 16) * 2.0 ** -23 * (a.abs() @ w.abs().t().contiguous())


def check(M, N, K, offsets, dtype=torch.bfloat16, seed=1, pad=0, q=None, w=None):
    G = 1 if offsets is None else len(offsets) - 1
    q, w = q or rows(M, K, seed), w or weights(G, N, K, seed + 1)
    buf = torch.full((M, N + pad), 7.0, dtype=dtype, device="cuda")
    out = buf[:, 1:1 + N] if pad else buf
    off = None if offsets is None else torch.tensor(offsets, dtype=torch.int32, device="cuda")
    nv.moe_mxfp8_product(nv.make_product_problem(M, N, K, G), q, w, off, out)
    torch.cuda.synchronize()
    a, v = values(q, w)
    half = torch.finfo(dtype).eps / 2
    keep = torch.ones(M, dtype=torch.bool, device="cuda")
    num = den = 0.0
    for g in range(G):
        b, e = (0, M) if offsets is None else (max(0, offsets[g]), min(M, offsets[g + 1]))
        if e <= b:
            continue
        keep[b:e] = False
        want = a[b:e] @ v[g].t().contiguous()
        err = (out[b:e].double() - want).abs()
        lim = bound(a[b:e], v[g]) + half * 1.01 * want.abs() + 1e-30
        assert (err <= lim).all(), (g, float((err / lim).max()))
        num += float(err.square().sum())
        den += float(want.square().sum())
    # over many results the losses are far below a rounding to bf16
    assert num <= (half + 2e-4) ** 2 * den
    assert (out[keep] == 7).all()
    if pad:
        assert (buf[:, 0] == 7).all() and (buf[:, 1 + N:] == 7).all()
    return q, w, out


def spread(M, G, seed, live=None):
    rng = np.random.default_rng(seed)
    return [0] + sorted(rng.integers(0, (M if live is None else live) + 1, G - 1).tolist()) + [M if live is None else live]


@pytest.mark.parametrize("K", [32, 64, 96, 128, 160, 256, 1024, 1056, 2048, 2080, 4096, 4128, 8192, 8224])
@pytest.mark.parametrize("M,N", [(1, 16), (5, 100), (17, 33), (40, 64)])
def test_few_rows(M, N, K):
    require_gpu()
    log(f"product8 M={M} N={N} K={K}")
    check(M, N, K, None)
    check(M, N, K, spread(M, 4, K), pad=3)


@pytest.mark.parametrize("K", [32, 96, 128, 160, 256, 384, 512, 640, 1056, 2048])
@pytest.mark.parametrize("M,N,G", [(300, 256, 1), (700, 300, 1), (2000, 1000, 3), (3000, 129, 5), (513, 15, 1)])
def test_many_rows(M, N, G, K):
    require_gpu()
    log(f"product8 M={M} N={N} K={K} G={G}")
    check(M, N, K, spread(M, G, K, M - 7))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("M,N,K,G", [(3, 70, 256, 2), (90, 1000, 512, 4), (1500, 515, 384, 2), (2600, 260, 288, 2)])
def test_output_types_and_strides(dtype, M, N, K, G):
    require_gpu()
    log(f"product8 {dtype} M={M} N={N} K={K}")
    check(M, N, K, spread(M, G, 3), dtype, pad=5)
    check(M, N, K, spread(M, G, 3), dtype)


def test_many_groups():
    """More groups than rows, empty groups, offsets that pass the buffer."""
    require_gpu()
    log("product8 groups")
    check(20, 64, 256, spread(20, 160, 1))
    check(1024, 48, 128, spread(1024, 1024, 2))
    check(3000, 64, 128, spread(3000, 700, 3))
    check(6, 32, 64, [-4, 2, 2, 9])
    check(2000, 256, 256, [0, 0, 1, 1999, 1999, 2000])
    check(4, 16, 32, [0, 0, 0])


def test_scales_of_unaligned_weights():
    """A shard's scales may start at any byte of a wider tensor."""
    require_gpu()
    log("product8 unaligned scales")
    for M in (20, 900):
        for K in (96, 256):
            w = weights(3, 40, K, 5)
            buf = torch.zeros(w.scales.numel() + 1, dtype=torch.uint8, device="cuda")
            buf[1:] = w.scales.flatten()
            check(M, 40, K, spread(M, 3, 2), w=nv.MXFP4Weights(w.codes, buf[1:].view_as(w.scales)))
            q = rows(M, K, 6)
            buf = torch.zeros(q.scales.numel() + 1, dtype=torch.uint8, device="cuda")
            buf[1:] = q.scales.flatten()
            check(M, 40, K, spread(M, 3, 2), w=w, q=nv.MXFP8Rows(q.codes, buf[1:].view_as(q.scales)))


@pytest.mark.parametrize("M", [3, 40, 700])
@pytest.mark.parametrize("K", [96, 256])
def test_every_scale_byte_and_nan(M, K):
    """A NaN block reaches its row or column alone; scale bytes over the whole range of fp32 results."""
    require_gpu()
    log(f"product8 scales M={M} K={K}")
    q, w = rows(M, K, 1), weights(1, 70, K, 2)
    q.scales[1, 1] = 255
    w.scales[0, 5, 0] = 255
    out = torch.zeros(M, 70, dtype=torch.float32, device="cuda")
    nv.moe_mxfp8_product(nv.make_product_problem(M, 70, K), q, w, None, out)
    bad = torch.isnan(out)
    want = torch.zeros_like(bad)
    want[1], want[:, 5] = True, True
    assert torch.equal(bad, want)
    # block powers from 2^-127 to 2^120 against their inverses: every product near 1
    q, w = rows(M, K, 3), weights(1, 70, K, 4)
    e = torch.randint(0, 241, (1, K // 32), generator=torch.Generator().manual_seed(1)).int().cuda()
    e[0, 0], e[0, -1] = 0, 240
    q.scales.copy_(e.expand(M, -1).to(torch.uint8))
    w.scales.copy_((245 - e).expand(70, -1).to(torch.uint8).unsqueeze(0))
    check(M, 70, K, None, torch.float32, q=q, w=w)


def test_equal_inputs_give_equal_bits():
    require_gpu()
    log("product8 repeat")
    for M, G in ((64, 8), (2500, 3)):
        off = spread(M, G, 1)
        q, w, out = check(M, 200, 1056, off)
        again = torch.zeros_like(out)
        nv.moe_mxfp8_product(nv.make_product_problem(M, 200, 1056, G), q, w,
                             torch.tensor(off, dtype=torch.int32, device="cuda"), again)
        n = off[-1]
        assert torch.equal(out[:n], again[:n])


def test_no_rows():
    require_gpu()
    w = weights(2, 16, 64, 1)
    q = nv.MXFP8Rows.empty(0, 64)
    nv.moe_mxfp8_product(nv.make_product_problem(0, 16, 64, 2), q, w, torch.zeros(3, dtype=torch.int32, device="cuda"),
                         torch.empty(0, 16, device="cuda"))


@pytest.mark.parametrize("K", [32, 64, 96, 128, 160, 192, 224, 256, 288, 384, 480, 512, 544, 640, 800, 1280])
@pytest.mark.parametrize("M,N,G", [(3026, 841, 66), (4100, 515, 100), (1200, 4099, 20), (90000, 257, 3), (6000, 1500, 31),
                                   (9000, 1100, 40)])
def test_workgroups_of_several_tiles(M, N, G, K):
    """More tiles than compute units: scale rows that lie differently to dwords in a workgroup's tiles, of one
    chunk of K and more."""
    require_gpu()
    log(f"product8 several tiles M={M} N={N} G={G} K={K}")
    assert not nv.lib().moe_internal_product_streams(M, N, K, G, K, 2, 0, 256)
    check(M, N, K, spread(M, G, K, M - 5))


@pytest.mark.parametrize("M,N,K,G", [(3000, 700, 640, 50), (1000, 2048, 1024, 3), (60000, 520, 384, 2)])
def test_captured_with_other_offsets(M, N, K, G):
    """One graph of short (or tall) tiles, replayed with other offsets and rows, beside work on another stream."""
    require_gpu()
    log(f"product8 captured M={M} N={N} K={K} G={G}")
    q, w = rows(M, K, 1), weights(G, N, K, 2)
    p = nv.make_product_problem(M, N, K, G)
    off = torch.tensor(spread(M, G, 1), dtype=torch.int32, device="cuda")
    out, want = (torch.zeros(M, N, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    nv.moe_mxfp8_product(p, q, w, off, out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        nv.moe_mxfp8_product(p, q, w, off, out)
    side = torch.cuda.Stream()
    for i in range(5):
        off.copy_(torch.tensor(spread(M, G, 10 + i, [M, 0, 1, M - 9, M][i]), dtype=torch.int32))
        q.codes.copy_(rows(M, K, 20 + i).codes)
        out.fill_(3.0)
        want.fill_(3.0)
        side.wait_stream(torch.cuda.current_stream())
        graph.replay()
        nv.moe_mxfp8_product(p, q, w, off, want, stream=side)
        torch.cuda.synchronize()
        assert torch.equal(out, want), i
        check(M, N, K, off.tolist(), q=nv.MXFP8Rows(q.codes, q.scales), w=w)

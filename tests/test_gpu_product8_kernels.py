"""GPU parity of each kernel of the W4A8 product with fp64, every case on the kernel that it names: output
types, strides, scales, groups, repeated calls."""
import numpy as np
import pytest
import torch

import nvfp4_expert_layer_amd as nv
from tests.gpu_helpers import log, require_gpu
from tests.product8_kernel import NORMWISE, bound, kernel, row_values, weight_values

pytestmark = pytest.mark.gpu

BF, F16, F32 = torch.bfloat16, torch.float16, torch.float32


def rows(M, K, seed):
    x = torch.randn(M, K, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda")
    x[:, ::64] *= 8
    q = nv.MXFP8Rows.empty(M, K)
    nv.moe_mxfp8_quantize(x, q.codes, q.scales)
    return q


def weights(G, N, K, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return nv.quantize_mxfp4_weights(torch.randn(G, N, K, generator=g, device="cuda") * K ** -0.5)


def spread(M, G, seed):
    return [0] + sorted(np.random.default_rng(seed).integers(0, M + 1, G - 1).tolist()) + [M]


def check(which, M, N, K, offsets, dtype=BF, pad=0, q=None, w=None, normwise=True):
    """Two calls against fp64, on the kernel `which`; rows of no group and the columns beside stay."""
    G = 1 if offsets is None else len(offsets) - 1
    assert kernel(M, N, K, G) == which
    q, w = q or rows(M, K, M + N), w or weights(G, N, K, K + N)
    off = None if offsets is None else torch.tensor(offsets, dtype=torch.int32, device="cuda")
    bufs = [torch.full((M, N + pad), 7.0, dtype=dtype, device="cuda") for _ in range(2)]
    for buf in bufs:
        out = buf[:, 1:1 + N] if pad else buf
        nv.moe_mxfp8_product(nv.make_product_problem(M, N, K, G), q, w, off, out)
    torch.cuda.synchronize()
    assert torch.equal(bufs[0].view(torch.uint8), bufs[1].view(torch.uint8))
    half, tiny = torch.finfo(dtype).eps / 2, float(torch.finfo(dtype).smallest_normal) * torch.finfo(dtype).eps
    keep = torch.ones(M, dtype=torch.bool, device="cuda")
    num = den = 0.0
    for g in range(G):
        b, e = (0, M) if offsets is None else (max(0, offsets[g]), min(M, offsets[g + 1]))
        if e <= b:
            continue
        keep[b:e] = False
        a = row_values(nv.MXFP8Rows(q.codes[b:e], q.scales[b:e]))
        v = weight_values(w.codes[g], w.scales[g])
        want = a @ v.t().contiguous()
        got = out[b:e].double()
        bad = torch.isnan(want)
        assert torch.equal(torch.isnan(got), bad)
        err = torch.where(bad, 0.0, (got - want).abs())
        want = torch.where(bad, 0.0, want)
        # (a NaN block's own bounds are not looked at)
        lim = torch.where(bad, 1.0, bound(a, v)) + half * 1.01 * want.abs() + tiny
        assert (err <= lim).all(), (g, float((err / lim).max()))
        num += float(err.square().sum())
        den += float(want.square().sum())
    if normwise:
        assert num <= (half + NORMWISE) ** 2 * den, (num / den) ** 0.5
    assert (out[keep] == 7).all()
    if pad:
        assert (buf[:, 0] == 7).all() and (buf[:, 1 + N:] == 7).all()


# one and several chunks of 256 k, an odd number of half chunks; one tile a workgroup and several
TALL = [(20000, 300, 128, 2), (70000, 300, 384, 3), (18000, 520, 640, 2), (40000, 257, 768, 5), (2300, 4100, 2048, 3),
        (2300, 4100, 4096, 1)]


@pytest.mark.parametrize("dtype,pad", [(BF, 0), (BF, 5), (F16, 0), (F16, 7), (F32, 0), (F32, 3)])
@pytest.mark.parametrize("M,N,K,G", TALL)
def test_tall_tiles(M, N, K, G, dtype, pad):
    require_gpu()
    log(f"product8 tall {dtype} M={M} N={N} K={K} G={G} pad={pad}")
    check("tall", M, N, K, spread(M, G, K) if G > 1 else None, dtype, pad)


@pytest.mark.parametrize("which,M,N,K,G", [("stream", 40, 70, 4096, 4), ("stream", 33, 100, 8320, 3),
                                           ("short", 900, 300, 128, 2), ("short", 700, 515, 384, 3),
                                           ("short", 400, 257, 4096, 2), ("short", 9000, 300, 640, 200),
                                           ("tall bytes", 900, 515, 96, 2), ("tall bytes", 3000, 300, 2080, 5),
                                           ("tall bytes", 20000, 1000, 288, 40)])
@pytest.mark.parametrize("dtype,pad", [(BF, 5), (F16, 0), (F32, 3)])
def test_other_kernels(which, M, N, K, G, dtype, pad):
    require_gpu()
    log(f"product8 {which} {dtype} M={M} N={N} K={K} G={G} pad={pad}")
    check(which, M, N, K, spread(M, G, K), dtype, pad)


@pytest.mark.parametrize("which,M,N,K", [("tall", 20000, 300, 1024), ("tall", 20000, 300, 896), ("tall", 20000, 300, 128),
                                         ("short", 900, 300, 1024), ("short", 900, 300, 896),
                                         ("tall bytes", 900, 300, 928), ("stream", 20, 300, 1024)])
def test_nan_and_every_power(which, M, N, K):
    """NaN blocks at every place of two chunks' scales reach their rows and columns alone; block powers from
    2^-127 to 2^120 against their inverses, every product near 1."""
    require_gpu()
    log(f"product8 {which} NaN M={M} N={N} K={K}")
    q, w = rows(M, K, 1), weights(1, N, K, 2)
    for b in range(K // 32):
        q.scales[(b * 13 + 1) % M, b] = 255
        w.scales[0, (b * 7 + 3) % N, b] = 255
    check(which, M, N, K, None, F32, q=q, w=w)
    log("powers")
    q, w = rows(M, K, 3), weights(1, N, K, 4)
    e = torch.randint(0, 241, (1, K // 32), generator=torch.Generator().manual_seed(K)).int().cuda()
    e[0, 0], e[0, -1] = 0, 240
    q.scales.copy_(e.expand(M, -1).to(torch.uint8))
    w.scales.copy_((245 - e).expand(N, -1).to(torch.uint8).unsqueeze(0))
    check(which, M, N, K, None, F32, q=q, w=w)


@pytest.mark.parametrize("which,M,N,K", [("tall", 20000, 300, 384), ("tall", 20000, 300, 2048), ("short", 1500, 300, 384),
                                         ("tall bytes", 1500, 300, 416), ("stream", 30, 300, 384)])
def test_empty_groups_and_far_offsets(which, M, N, K):
    """Groups without rows, offsets before and past the buffer, rows behind the last group."""
    require_gpu()
    log(f"product8 {which} groups M={M} N={N} K={K}")
    half = M // 2
    check(which, M, N, K, [0, 0, 1, 1, half, half, M - 3], pad=3)
    check(which, M, N, K, [-4, 2, 2, half, M + 900, 1 << 30])
    check(which, M, N, K, [-9, -5, 0, 0, M])
    check(which, M, N, K, [0, 0, 0, 0], normwise=False)
    check(which, M, N, K, [M, M + 5, M + 5], normwise=False)

"""Few rows over many groups against the fp64 oracle, every group: workgroups find their group by
rank when there are fewer rows than groups, and the gradient's workgroups are handed out around the
XCDs (eight groups and more; fewer groups with a multiple of eight column blocks; neither).  Exact
sums, as in test_gpu_product."""
import numpy as np
import pytest
import torch

import nvfp4_expert_layer_amd as nv
from oracle import dispatch, mxfp4
from tests.gpu_helpers import log, require_gpu
from tests.product_choice import streams
from tests.test_gpu_product import BF, f64, mx_random

pytestmark = pytest.mark.gpu


def counts_of(kind, M, G, gen):
    """Rows of each group: spread by chance, all in one group, or one row in every other group."""
    if kind == "one":
        c = torch.zeros(G, dtype=torch.int64)
        c[G - 1 - G // 3] = M
    elif kind == "alternate":
        c = torch.zeros(G, dtype=torch.int64)
        c[1::2][:M] = 1
    else:
        c = torch.bincount(torch.randint(0, G, (M,), generator=gen), minlength=G)
    return torch.cat([torch.zeros(1, dtype=torch.int64), c.cumsum(0)])


SHAPES = [(3, 200, "chance"), (20, 24, "chance"), (7, 8, "one"), (50, 64, "chance"), (100, 200, "alternate"),
          (9, 1024, "chance"), (300, 64, "chance"), (130, 16, "chance"), (60, 8, "one"), (40, 5, "chance"), (5, 7, "chance")]


@pytest.mark.parametrize("M,G,kind", SHAPES)
@pytest.mark.parametrize("N,K", [(40, 1024), (72, 384), (33, 128), (17, 2048)])
def test_gradient_of_every_group(M, G, kind, N, K):
    require_gpu()
    log(f"gradient groups M={M} G={G} {kind} N={N} K={K}")
    assert streams("backward", M, N, K, G)
    gen = torch.Generator().manual_seed(M * G + K)
    off = counts_of(kind, M, G, gen)
    wc, ws = mx_random(gen, G, N, K)
    d = torch.randint(-8, 9, (M, N), generator=gen).to(BF)
    out = torch.full((M, K), 55.0, device="cuda")
    nv.moe_mxfp4_product_backward(nv.make_product_problem(M, N, K, G), d.cuda(), nv.MXFP4Weights(wc.cuda(), ws.cuda()),
                                  off.int().cuda(), out)
    e = int(off[-1])
    ref = dispatch.product(f64(d), mxfp4.dequantize(wc.numpy(), ws.numpy()), off.numpy(), backward=True)[0]
    assert np.array_equal(f64(out)[:e], ref[:e]) and (out[e:] == 55).all()


@pytest.mark.parametrize("mode", ["w4a16", "w4a4"])
@pytest.mark.parametrize("M,G,kind", SHAPES)
@pytest.mark.parametrize("N,K", [(40, 1024), (300, 96), (24, 4128)])
def test_product_of_every_group(mode, M, G, kind, N, K):
    require_gpu()
    log(f"product groups {mode} M={M} G={G} {kind} N={N} K={K}")
    if G * N * K > 1 << 26:
        N = 8
    assert streams(mode, M, N, K, G)
    gen = torch.Generator().manual_seed(M * G + K)
    off = counts_of(kind, M, G, gen)
    wc, ws = mx_random(gen, G, N, K)
    ac, as_ = mx_random(gen, M, K)
    a64 = mxfp4.dequantize(ac.numpy(), as_.numpy())
    a = nv.MXFP4Rows(ac.cuda(), as_.cuda()) if mode == "w4a4" else torch.from_numpy(a64).to(BF).cuda()
    out = torch.full((M, N), 55.0, device="cuda")
    nv.moe_mxfp4_product(nv.make_product_problem(M, N, K, G), a, nv.MXFP4Weights(wc.cuda(), ws.cuda()),
                         off.int().cuda(), out)
    e = int(off[-1])
    ref = dispatch.product(a64, mxfp4.dequantize(wc.numpy(), ws.numpy()), off.numpy())[0]
    assert np.array_equal(f64(out)[:e], ref[:e]) and (out[e:] == 55).all()

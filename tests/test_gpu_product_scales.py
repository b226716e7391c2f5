"""Every scale byte through every product kernel.

One output has one weight scale s (and, W4A4, its row one scale), so that an output is an integer
below 2^24 times a power of two 2^q; it is exact in fp32 where q >= -149 (subnormal outputs too) and
the sum of magnitudes stays below 2^128, and is compared there bit for bit.  W4A16 and the gradient
hold weights in bf16: code * 2^(s - 127) from 2^128 on (s 253 and 254) is Inf there."""
import numpy as np
import pytest
import torch

import nvfp4_expert_layer_amd as nv
from oracle import mxfp4
from tests.gpu_helpers import log, require_gpu
from tests.product_choice import streams
from tests.test_gpu_product import BF, f64, mx_random

pytestmark = pytest.mark.gpu

S = np.arange(256)
GROUPS = 2


def offsets(M):
    return np.linspace(0, M, GROUPS + 1).astype(np.int64)


def by_group(rows, w, off, backward):
    """In fp64: the product with Inf and NaN where the terms give them, the sum of magnitudes, the
    same of the finite terms alone."""
    with np.errstate(all="ignore"):
        p = [(rows[off[g]:off[g + 1]], w[g] if backward else w[g].T) for g in range(GROUPS)]
        fin = lambda x: np.where(np.isfinite(x), np.abs(x), 0.0)                                 # noqa: E731
        return (np.concatenate([a @ m for a, m in p]), np.concatenate([np.abs(a) @ np.abs(m) for a, m in p]),
                np.concatenate([fin(a) @ fin(m) for a, m in p]))


def check(out, ref, mag, finite, unit):
    """unit [columns]: log2 of what every term of a column is a multiple of."""
    got = f64(out)
    exact = np.isfinite(mag) & (mag < 2.0 ** 128) & (unit >= -149)
    assert np.array_equal(got[exact], ref[exact])
    # a term that is Inf or NaN: never a finite sum; and where no finite term can overflow beside it
    # (fp32 would make that one Inf of its own sign), the sum's own value, whatever the order
    special = ~np.isfinite(mag)
    assert not np.isfinite(got[special]).any()
    alone = special & (finite < 2.0 ** 128)
    assert np.array_equal(got[alone], ref[alone], equal_nan=True)
    return exact


@pytest.mark.parametrize("M,K,tiled", [(5, 64, False), (40, 512, False), (20, 4128, False), (1100, 128, True),
                                       (1100, 160, True)])
@pytest.mark.parametrize("e", [-130, -100, 0, 100])
def test_w4a16(M, K, tiled, e):
    require_gpu()
    log(f"scale bytes w4a16 M={M} K={K} e={e}")
    N = 256
    assert streams("w4a16", M, N, K, GROUPS) != tiled
    gen = torch.Generator().manual_seed(K)
    wc, _ = mx_random(gen, GROUPS, N, K)
    ws = torch.arange(N, dtype=torch.uint8).view(1, N, 1).expand(GROUPS, N, K // 32).contiguous()
    a = torch.ldexp(torch.randint(-8, 9, (M, K), generator=gen).float(), torch.tensor(e)).to(BF)
    off, out = offsets(M), torch.empty(M, N, device="cuda")
    nv.moe_mxfp4_product(nv.make_product_problem(M, N, K, GROUPS), a.cuda(), nv.MXFP4Weights(wc.cuda(), ws.cuda()),
                         torch.from_numpy(off).int().cuda(), out)
    w = mxfp4.dequantize(wc.numpy(), ws.numpy())
    w = np.where(np.abs(w) >= 2.0 ** 128, np.copysign(np.inf, w), w)
    exact = check(out, *by_group(f64(a), w, off, False), S - 128 + e)
    assert exact[:, 60:253].any(0).sum() > 40 and (e > -100 or exact[:, 79 if e == -100 else 109:253].all())


@pytest.mark.parametrize("M,N,tiled", [(5, 40, False), (40, 72, False), (700, 64, True), (700, 43, True)])
@pytest.mark.parametrize("e", [-130, -100, 0, 100])
def test_gradient(M, N, tiled, e):
    """The columns' blocks hold the scale bytes."""
    require_gpu()
    log(f"scale bytes gradient M={M} N={N} e={e}")
    K = 8192
    assert streams("backward", M, N, K, GROUPS) != tiled
    gen = torch.Generator().manual_seed(N)
    wc, _ = mx_random(gen, GROUPS, N, K)
    ws = torch.arange(256, dtype=torch.uint8).view(1, 1, 256).expand(GROUPS, N, 256).contiguous()
    d = torch.ldexp(torch.randint(-8, 9, (M, N), generator=gen).float(), torch.tensor(e)).to(BF)
    off, out = offsets(M), torch.empty(M, K, device="cuda")
    nv.moe_mxfp4_product_backward(nv.make_product_problem(M, N, K, GROUPS), d.cuda(),
                                  nv.MXFP4Weights(wc.cuda(), ws.cuda()), torch.from_numpy(off).int().cuda(), out)
    w = mxfp4.dequantize(wc.numpy(), ws.numpy())
    w = np.where(np.abs(w) >= 2.0 ** 128, np.copysign(np.inf, w), w)
    check(out, *by_group(f64(d), w, off, True), np.repeat(S - 128 + e, 32))


@pytest.mark.parametrize("M,K,tiled", [(256, 64, False), (300, 512, False), (256, 8224, False), (1024, 128, True),
                                       (1024, 160, True), (1024, 384, True)])
def test_w4a4(M, K, tiled):
    """Rows and weight rows run through all bytes: every pair of two scales."""
    require_gpu()
    log(f"scale bytes w4a4 M={M} K={K}")
    N = 256
    assert streams("w4a4", M, N, K, GROUPS) != tiled
    gen = torch.Generator().manual_seed(K)
    wc, _ = mx_random(gen, GROUPS, N, K)
    ws = torch.arange(N, dtype=torch.uint8).view(1, N, 1).expand(GROUPS, N, K // 32).contiguous()
    ac, _ = mx_random(gen, M, K)
    sa = torch.arange(M).remainder(256).to(torch.uint8)
    as_ = sa.view(M, 1).expand(M, K // 32).contiguous()
    off, out = offsets(M), torch.empty(M, N, device="cuda")
    nv.moe_mxfp4_product(nv.make_product_problem(M, N, K, GROUPS), nv.MXFP4Rows(ac.cuda(), as_.cuda()),
                         nv.MXFP4Weights(wc.cuda(), ws.cuda()), torch.from_numpy(off).int().cuda(), out)
    terms = by_group(mxfp4.dequantize(ac.numpy(), as_.numpy()), mxfp4.dequantize(wc.numpy(), ws.numpy()), off, False)
    exact = check(out, *terms, sa.numpy().astype(int)[:, None] + S[None, :] - 256)
    assert exact.sum() > exact.size // 3 and np.isnan(f64(out)[sa.numpy() == 255]).all()

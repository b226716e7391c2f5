"""The tile kernels of the W4A8 product over rows, weights and outputs whose offsets pass 32 bits, against fp64."""
import pytest
import torch

import nvfp4_expert_layer_amd as nv
from tests.gpu_helpers import log, require_gpu
from tests.product8_kernel import NORMWISE, bound, kernel, row_values, weight_values

pytestmark = pytest.mark.gpu


def compare(out, a, v):
    """fp32 outputs of rows a with weights v."""
    want = a @ v.t().contiguous()
    err = (out.double() - want).abs()
    assert (err <= bound(a, v) + 2.0 ** -24 * 1.01 * want.abs()).all()
    assert float(err.norm()) <= (NORMWISE + 2.0 ** -24) * float(want.norm())


@pytest.mark.parametrize("which,M", [("stream", 600), ("short", 9000), ("tall", 66000)])
def test_weights(which, M):
    """5.4e9 bytes of codes; the first, a middle and the last group hold rows, whose weights lie before, on and
    past 2^32 bytes."""
    require_gpu()
    log(f"product8 far weights {which} M={M}")
    G, N, K = 1024, 2560, 4096
    assert kernel(M, N, K, G) == which
    w = nv.MXFP4Weights(torch.zeros(G, N, K // 2, dtype=torch.uint8, device="cuda"),
                        torch.full((G, N, K // 32), 127, dtype=torch.uint8, device="cuda"))
    mid = 2 ** 32 // (N * K // 2)                                   # its codes hold byte 2^32
    gen = torch.Generator(device="cuda").manual_seed(M)
    own = nv.quantize_mxfp4_weights(torch.randn(3, N, K, generator=gen, device="cuda") * K ** -0.5)
    for i, g in enumerate((0, mid, G - 1)):
        w.codes[g], w.scales[g] = own.codes[i], own.scales[i]
    x = nv.MXFP8Rows.empty(M, K)
    nv.moe_mxfp8_quantize(torch.randn(M, K, generator=gen, device="cuda"), x.codes, x.scales)
    ends = torch.zeros(G + 1, dtype=torch.int32)
    ends[1:] = 70                                                   # group 0: 70 rows
    ends[mid + 1:] = M // 2                                         # the middle one the next
    ends[-1] = M
    out = torch.empty(M, N, device="cuda")
    nv.moe_mxfp8_product(nv.make_product_problem(M, N, K, G), x, w, ends.cuda(), out)
    part = lambda b, e: nv.MXFP8Rows(x.codes[b:e], x.scales[b:e])  # noqa: E731
    for i, (b, e) in enumerate(((0, 70), (70, M // 2), (M // 2, M))):
        v = weight_values(own.codes[i], own.scales[i])
        for lo, hi in ((b, min(e, b + 200)), (max(b, e - 200), e)):
            compare(out[lo:hi], row_values(part(lo, hi)), v)


@pytest.mark.parametrize("which,M,G", [("short", 65500, 1024), ("tall", 70000, 2)])
def test_rows_and_outputs(which, M, G):
    """Rows of 4.3e9 (short tiles take no more) and 4.6e9 bytes, outputs over 1e10 bytes (2.6e9 elements) and more."""
    require_gpu()
    log(f"product8 far rows {which}")
    N, K, stride = 24, 65536, 40000
    assert kernel(M, N, K, G) == which and M * K > 2 ** 31 and M * stride * 4 > 2 ** 32
    q = nv.MXFP8Rows(torch.zeros(M, K, dtype=torch.uint8, device="cuda"),
                     torch.full((M, K // 32), 127, dtype=torch.uint8, device="cuda"))
    gen = torch.Generator(device="cuda").manual_seed(M)
    part = nv.MXFP8Rows.empty(300, K)
    nv.moe_mxfp8_quantize(torch.randn(300, K, generator=gen, device="cuda"), part.codes, part.scales)
    q.codes[:100], q.scales[:100] = part.codes[:100], part.scales[:100]
    q.codes[-200:], q.scales[-200:] = part.codes[100:], part.scales[100:]
    own = nv.quantize_mxfp4_weights(torch.randn(2, N, K, generator=gen, device="cuda") * K ** -0.5)
    w = nv.MXFP4Weights(torch.zeros(G, N, K // 2, dtype=torch.uint8, device="cuda"),
                        torch.full((G, N, K // 32), 127, dtype=torch.uint8, device="cuda"))
    w.codes[0], w.scales[0], w.codes[-1], w.scales[-1] = own.codes[0], own.scales[0], own.codes[1], own.scales[1]
    ends = torch.full((G + 1,), M - 150, dtype=torch.int32)
    ends[0], ends[-1] = 0, M
    out = torch.full((M, stride), 7.0, device="cuda")
    nv.moe_mxfp8_product(nv.make_product_problem(M, N, K, G), q, w, ends.cuda(), out[:, 3:3 + N])
    a = row_values(part)
    first, last = (weight_values(own.codes[i], own.scales[i]) for i in (0, 1))
    compare(out[:100, 3:3 + N], a[:100], first)
    compare(out[-200:-150, 3:3 + N], a[100:150], first)
    compare(out[-150:, 3:3 + N], a[150:], last)
    assert (out[100:-200, 3:3 + N] == 0).all()
    for b in range(0, M, 10000):
        assert (out[b:b + 10000, :3] == 7).all() and (out[b:b + 10000, 3 + N:] == 7).all()

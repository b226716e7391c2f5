"""GPU parity of the MXFP4 quantizer and dequantizer: codes, scales and values must
equal the fp64 oracle's (every decision is exact in fp32)."""
import numpy as np
import pytest
import torch

import nvfp4_expert_layer_amd as nv
from oracle import mxfp4
from tests.gpu_helpers import log, require_gpu

pytestmark = pytest.mark.gpu

FLOATS = [torch.bfloat16, torch.float16, torch.float32]


def run(x):
    R, C = x.shape
    codes = torch.full((R, C // 2), 0xA5, dtype=torch.uint8, device="cuda")
    scales = torch.full((R, C // 32), 0xA5, dtype=torch.uint8, device="cuda")
    nv.moe_mxfp4_quantize(x, codes, scales)
    torch.cuda.synchronize()
    return codes, scales


def draw(R, C, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(R, C, generator=g) * torch.exp2(torch.randint(-12, 10, (R, C // 32), generator=g).float()
                                                    ).repeat_interleave(32, 1)
    x[0, :32] = 0.0
    x[R // 2, -32:] = 0.0
    x[R // 2, -1] = -1e-7                                        # a block of one tiny element
    return x.to(dtype)


def check(x, codes, scales):
    qc, qs = mxfp4.quantize(x.double().cpu().numpy())
    assert np.array_equal(scales.cpu().numpy(), qs)
    assert np.array_equal(codes.cpu().numpy(), qc)


@pytest.mark.parametrize("dtype", FLOATS)
@pytest.mark.parametrize("R,C", [(1, 32), (3, 64), (64, 4096), (257, 1056), (1, 65536), (1000, 96)])
def test_quantizer_bit_exact(dtype, R, C):
    require_gpu()
    log(f"mxfp4 quantize {dtype} {R}x{C}")
    x = draw(R, C, dtype, R + C)
    check(x, *run(x.cuda()))


@pytest.mark.parametrize("dtype", FLOATS)
@pytest.mark.parametrize("start,width", [(0, 128), (16, 192), (3, 101)])
def test_quantizer_strided_rows(dtype, start, width):
    require_gpu()
    log(f"mxfp4 quantize strided {dtype} start={start} width={width}")
    wide = draw(50, 96, dtype, 7)
    x = torch.zeros(50, width, dtype=dtype, device="cuda")[:, start:start + 96]
    x.copy_(wide)
    check(wide, *run(x))


@pytest.mark.parametrize("dtype", FLOATS)
def test_ties_saturation_and_every_binade(dtype):
    """In every scale the type reaches: all code values, all midpoints, their neighbours, 6 to 8."""
    require_gpu()
    log(f"mxfp4 quantize ties {dtype}")
    grid = torch.tensor([0, .25, .5, .75, 1, 1.25, 1.5, 1.75, 2, 2.5, 3, 3.5, 4, 5, 6, 7.5])
    lo, hi = (-14, 13) if dtype == torch.float16 else (-126, 125)
    rows = []
    for e in range(lo, hi + 1):
        v = torch.ldexp(grid.double(), torch.tensor(e)).to(dtype)
        up = torch.nextafter(v.float(), torch.full((16,), float("inf"))).to(dtype) if dtype == torch.float32 else \
            (v.view(torch.int16) + 1).view(dtype)
        rows += [torch.cat([v, -up]), torch.cat([-v, up])]
        up = up.clone()
        up[-1] = v[-1]
    x = torch.stack(rows)
    x = torch.cat([x, x], dim=1)
    check(x, *run(x.cuda()))


@pytest.mark.parametrize("dtype", FLOATS)
def test_subnormals_inf_nan(dtype):
    require_gpu()
    log(f"mxfp4 quantize extremes {dtype}")
    fi = torch.finfo(dtype)
    x = torch.zeros(8, 64, dtype=dtype)
    x[0, :8] = fi.tiny * torch.tensor([1, .5, .25, -.125, 2, 3, -4, 1.5]).to(dtype)
    x[1, 3] = fi.max
    x[1, 40] = -fi.max
    x[2, 0], x[2, 33] = float("inf"), 1.0
    x[3, 31], x[3, 32] = float("nan"), -2.0
    x[4, 63] = float("-inf")
    x[5, 0] = fi.tiny * fi.eps                                   # the smallest subnormal
    x[6] = -0.0
    codes, scales = run(x.cuda())
    check(x, codes, scales)
    assert scales[2].tolist()[0] == 255 and scales[3].tolist()[0] == 255 and scales[4].tolist()[1] == 255


@pytest.mark.parametrize("dtype", FLOATS)
def test_dequantizer_every_scale_and_code(dtype):
    """All 256 scales x 16 codes; f16 rounds to nearest even and overflows to Inf as numpy does."""
    require_gpu()
    log(f"mxfp4 dequantize {dtype}")
    scales = torch.arange(256, dtype=torch.uint8).reshape(256, 1)
    codes = torch.arange(16, dtype=torch.uint8).repeat(256, 1)
    codes = codes | ((15 - codes) << 4)
    for start, width in ((0, 32), (8, 64), (1, 41)):
        out = torch.zeros(256, width, dtype=dtype, device="cuda")[:, start:start + 32]
        nv.moe_mxfp4_dequantize(codes.cuda(), scales.cuda(), out)
        with np.errstate(over="ignore"):
            ref = torch.from_numpy(mxfp4.dequantize(codes.numpy(), scales.numpy()).astype(np.float32)).to(dtype)
        got = out.cpu()
        assert torch.equal(torch.isnan(got), torch.isnan(ref)) and torch.isnan(got[255]).all()
        assert torch.equal(got[:255], ref[:255])
        assert torch.equal(torch.signbit(got[:255]), torch.signbit(ref[:255]))


def test_weights_helper_and_round_trip():
    require_gpu()
    log("mxfp4 weights")
    w = torch.randn(3, 50, 96, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    q = nv.quantize_mxfp4_weights(w)
    one = nv.MXFP4Weights.empty(4, 50, 96)
    nv.quantize_mxfp4_weights(w[1:2], one, 2)
    assert torch.equal(one.codes[2], q.codes[1]) and torch.equal(one.slice(2, 1).scales[0], q.scales[1])
    v = torch.empty(150, 96, device="cuda")
    nv.moe_mxfp4_dequantize(q.codes.view(150, 48), q.scales.view(150, 3), v)
    c2, s2 = run(v)
    v2 = torch.empty_like(v)
    nv.moe_mxfp4_dequantize(c2, s2, v2)
    assert torch.equal(v, v2)                                    # its own values stay

"""GPU parity of the MXFP8 quantizer and dequantizer: codes, scales and values must equal the
fp64 oracle's (every decision is exact)."""
import numpy as np
import pytest
import torch

import nvfp4_expert_layer_amd as nv
from oracle import block
from tests.gpu_helpers import log, require_gpu

pytestmark = pytest.mark.gpu

FLOATS = [torch.bfloat16, torch.float16, torch.float32]


def run(x):
    q = nv.MXFP8Rows.empty(*x.shape)
    q.codes.fill_(0xA5)
    q.scales.fill_(0xA5)
    nv.moe_mxfp8_quantize(x, q.codes, q.scales)
    torch.cuda.synchronize()
    return q


def draw(R, C, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(R, C, generator=g) * torch.exp2(torch.randint(-12, 10, (R, C // 32), generator=g).float()
                                                    ).repeat_interleave(32, 1)
    x[0, :32] = 0.0
    x[R // 2, -32:] = 0.0
    x[R // 2, -1] = -1e-7                                        # a block of one tiny element
    return x.to(dtype)


def check(x, q):
    codes, scales = block.mxfp8_quantize(x.double().cpu().numpy())
    assert np.array_equal(q.scales.cpu().numpy(), scales)
    assert np.array_equal(q.codes.cpu().numpy(), codes)


@pytest.mark.parametrize("dtype", FLOATS)
@pytest.mark.parametrize("R,C", [(1, 32), (3, 64), (64, 4096), (257, 1056), (1, 65536), (1000, 96)])
def test_quantizer_bit_exact(dtype, R, C):
    require_gpu()
    log(f"mxfp8 quantize {dtype} {R}x{C}")
    x = draw(R, C, dtype, R + C)
    check(x, run(x.cuda()))


@pytest.mark.parametrize("dtype", FLOATS)
@pytest.mark.parametrize("start,width", [(0, 128), (16, 192), (3, 101)])
def test_strided_rows(dtype, start, width):
    require_gpu()
    log(f"mxfp8 strided {dtype} start={start} width={width}")
    wide = draw(50, 96, dtype, 7)
    buf = torch.full((50, width), 3.0, dtype=dtype, device="cuda")
    x = buf[:, start:start + 96]
    x.copy_(wide)
    q = run(x)
    check(wide, q)
    nv.moe_mxfp8_dequantize(q.codes, q.scales, x)
    want = torch.from_numpy(block.mxfp8_dequantize(q.codes.cpu().numpy(), q.scales.cpu().numpy())).to(dtype)
    assert torch.equal(x.cpu(), want)
    buf[:, start:start + 96] = 3.0
    assert (buf == 3.0).all()


def test_every_midpoint_and_its_neighbours():
    """Values next to every border between two codes, under scales over fp32's whole range."""
    require_gpu()
    log("mxfp8 midpoints")
    mid = (block.E4M3[1:] + block.E4M3[:-1]) / 2
    around = np.concatenate([mid.astype(np.float32), np.nextafter(mid.astype(np.float32), np.float32(0)),
                             np.nextafter(mid.astype(np.float32), np.float32(1e9)), block.E4M3.astype(np.float32),
                             np.linspace(448, 511.9, 63, dtype=np.float32)])
    around = np.concatenate([around, -around])
    around = np.resize(around, (len(around) + 30) // 31 * 31).reshape(-1, 31)
    x = np.concatenate([np.full((len(around), 1), 256.0, np.float32), around], axis=1)   # the block's scale is 2^0
    rows = np.concatenate([np.ldexp(x.astype(np.float64), e).astype(np.float32) for e in (0, -20, 100, 118, -117, -127, 7)])
    assert np.isfinite(rows).all()
    t = torch.from_numpy(rows)
    check(t, run(t.cuda()))


@pytest.mark.parametrize("dtype", FLOATS)
def test_specials(dtype):
    """Inf and NaN spoil their own block alone; signed zeros, subnormals and the largest values."""
    require_gpu()
    log(f"mxfp8 specials {dtype}")
    top = torch.finfo(dtype).max
    x = torch.randn(8, 96, generator=torch.Generator().manual_seed(1)).to(dtype)
    x[0, 40], x[1, 0], x[2, 95], x[3, 64:] = float("inf"), float("nan"), float("-inf"), -0.0
    x[4, :32], x[5, 7] = top, -top
    x[6, :32] = torch.tensor(torch.finfo(dtype).tiny, dtype=dtype) / 4
    x[6, 32:64] = torch.finfo(dtype).tiny
    q = run(x.cuda())
    check(x, q)
    for out in FLOATS:
        v = torch.empty(8, 96, dtype=out, device="cuda")
        nv.moe_mxfp8_dequantize(q.codes, q.scales, v)
        want = torch.from_numpy(block.mxfp8_dequantize(q.codes.cpu().numpy(), q.scales.cpu().numpy())).to(out)
        assert torch.equal(torch.isnan(v).cpu(), torch.isnan(want))
        assert torch.equal(v.cpu().nan_to_num(7.0), want.nan_to_num(7.0))


@pytest.mark.parametrize("dtype", FLOATS)
def test_dequantizer_every_code_and_scale(dtype):
    require_gpu()
    log(f"mxfp8 dequantize {dtype}")
    codes = torch.arange(256, dtype=torch.uint8).repeat(256, 1)
    scales = torch.arange(256, dtype=torch.uint8).unsqueeze(1).repeat(1, 8)
    out = torch.empty(256, 256, dtype=dtype, device="cuda")
    nv.moe_mxfp8_dequantize(codes.cuda(), scales.cuda(), out)
    want = torch.from_numpy(block.mxfp8_dequantize(codes.numpy(), scales.numpy())).to(dtype)
    assert torch.equal(torch.isnan(out).cpu(), torch.isnan(want))
    assert torch.equal(out.cpu().nan_to_num(7.0), want.nan_to_num(7.0))


def test_no_rows():
    require_gpu()
    q = run(torch.empty(0, 64, dtype=torch.bfloat16, device="cuda"))
    nv.moe_mxfp8_dequantize(q.codes, q.scales, torch.empty(0, 64, device="cuda"))

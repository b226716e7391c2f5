"""Which kernel a W4A8 product takes, and its fp64 result (test infrastructure): the rule that the library's
launches use; values by table on the GPU, the tables from the oracle."""
import ctypes

import numpy as np
import torch

import nvfp4_expert_layer_amd as nv
from oracle import block, mxfp4


def kernel(M, N, K, G, cus=None):
    """"stream", "short" (tiles of 64 rows), "tall" (of 256) or "tall bytes" (scale rows that are no whole
    dwords), for 4-byte aligned scales; cus: by default the device's."""
    if cus is None:
        cus = torch.cuda.get_device_properties(torch.cuda.current_device()).multi_processor_count
    streams, short = nv.lib().moe_internal_product_streams, nv.lib().moe_internal_product8_short
    streams.argtypes = [ctypes.c_int] * 4 + [ctypes.c_int64] + [ctypes.c_int] * 3
    short.argtypes = [ctypes.c_int] * 5
    streams.restype = short.restype = ctypes.c_int
    if streams(M, N, K, G, K, 2, 0, cus):
        return "stream"
    return "tall bytes" if K % 128 else ("short" if short(M, N, K, G, cus) else "tall")


def _scale_table():
    return torch.from_numpy(np.where(np.arange(256) == 255, np.nan, np.ldexp(1.0, np.arange(256) - 127))).cuda()


def row_values(q):
    """fp64 values of MXFP8Rows [M, K]."""
    table = torch.from_numpy(block.mxfp8_dequantize(np.arange(256, dtype=np.uint8), np.full(8, 127, np.uint8))).cuda()
    return table[q.codes.int()] * _scale_table()[q.scales.int()].repeat_interleave(32, -1)


def weight_values(codes, scales):
    """fp64 values of MXFP4 codes [..., K/2] and scales [..., K/32]."""
    pairs = np.arange(256, dtype=np.uint8)
    table = torch.from_numpy(mxfp4.dequantize(pairs.reshape(16, 16), np.full((16, 1), 127, np.uint8)).reshape(256, 2)).cuda()
    # (a gather of pairs at once has given zeros here beyond 2^26 of them)
    both = torch.stack([table[:, i].contiguous()[codes.int()] for i in (0, 1)], -1).flatten(-2)
    return both * _scale_table()[scales.int()].repeat_interleave(32, -1)


def bound(a, w):
    """What the matrix cores may lose on a [m, K] . w [n, K]^T: each product up to 2^-13 of the largest of its
    eight (of its block, at most), and fp32 sums of K / 8 terms."""
    top = lambda v: v.abs().unflatten(-1, (-1, 32)).amax(-1)  # noqa: E731
    aligned = 32 * 2.0 ** -13 * (top(a) @ top(w).t().contiguous())
    return aligned + (a.shape[1] / 8 + 16) * 2.0 ** -23 * (a.abs() @ w.abs().t().contiguous())


# Over many results, relative to their norm: a product loses up to 2^-13 of the largest m of its eight, in the
# mean square 2^-26 m^2 / 3, and m^2 is at most the eight's sum of squares: 2^-13 sqrt(8 / 3) = 2.0e-4, where the
# losses' signs are by chance.
NORMWISE = 2.0e-4

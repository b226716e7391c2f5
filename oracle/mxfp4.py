"""MXFP4 in plain numpy fp64 (test infrastructure; shares nothing with the GPU path).

From the Open Compute Project's microscaling format: a block is 32 elements, its
scale 2^(floor(log2 amax) - 2) held as a power-of-two byte (E8M0, bias 127, 255 =
NaN), its elements E2M1, each the nearest of the sixteen values (ties to the even
code, beyond 6 saturating).  Codes are found by searching the value set.
"""
import numpy as np

BLOCK = 32
MAGNITUDES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def quantize(x):
    """x [R, C] -> codes uint8 [R, C/2] (even element in the low nibble), scales uint8 [R, C/32]."""
    x = np.asarray(x, dtype=np.float64)
    R, C = x.shape
    b = x.reshape(R, C // BLOCK, BLOCK)
    bad = ~np.isfinite(b).all(axis=2)
    b = np.where(bad[:, :, None], 0.0, b)
    amax = np.abs(b).max(axis=2)
    e = np.full(amax.shape, -127)
    nz = amax > 0
    e[nz] = np.clip(np.floor(np.log2(amax[nz])).astype(int) - 2, -127, 127)
    # log2 of a value just below a power of two may round up to it
    e = np.where(nz & (amax < np.ldexp(1.0, e + 2)) & (e > -127), e - 1, e)
    q = np.ldexp(b, -e[:, :, None])
    dist = np.abs(np.abs(q)[..., None] - MAGNITUDES)
    # nearest magnitude; of two equally near ones the even code
    near = dist <= dist.min(axis=-1, keepdims=True)
    rank = near * np.where(np.arange(8) % 2 == 0, 2, 1)
    code = rank.argmax(axis=-1) | (np.signbit(q) * 8)
    code = np.where(bad[:, :, None], 0, code).astype(np.uint8).reshape(R, C)
    scales = np.where(bad, 255, e + 127).astype(np.uint8)
    return code[:, 0::2] | (code[:, 1::2] << 4), scales


def dequantize(codes, scales):
    """fp64 values of codes [..., C/2] and scales [..., C/32] (NaN where a scale is 255)."""
    codes, scales = np.asarray(codes), np.asarray(scales)
    c = np.stack([codes & 15, codes >> 4], axis=-1).reshape(*codes.shape[:-1], -1)
    v = np.where(c & 8, -1.0, 1.0) * MAGNITUDES[c & 7]
    s = np.where(scales == 255, np.nan, np.ldexp(1.0, scales.astype(int) - 127))
    return v * np.repeat(s, BLOCK, axis=-1)

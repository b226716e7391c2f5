"""Rows that take different columns of one buffer are not an overlap (CPU: the pointers are
never followed); rows that share a byte still are."""
import ctypes
import random

import pytest

import nvfp4_expert_layer_amd as nv
from tests.test_abi_ops import G, INV, at, combine_backward, dequantize, dispatch, dp, product, product_backward
from tests.test_abi_ops import combine, well_formed


def test_neighbouring_columns_of_one_buffer():
    """T=64, k=8, d=4096 bf16 unless said: byte offsets of two for an element."""
    # gathered rows in the right half of a buffer, combined ones' gradient in its left half
    assert well_formed(combine_backward(rows=at(2, 8192), rs=8192, drows=at(2), drs=8192))
    assert well_formed(combine_backward(rows=at(2), rs=8192, drows=at(2, 8192), drs=8192))
    # every k-th row of the same buffer: strides that divide each other
    assert well_formed(combine(rows=at(2, 8192), rs=8192, out=at(2), os_=8 * 8192))
    assert well_formed(dispatch(x=at(1), xs=8 * 8192, rows=at(1, 8192), rs=8192))
    assert well_formed(product(N=32, K=96, a=at(0), as_=128, out=at(0, 192), os_=128))
    assert well_formed(product_backward(N=96, K=32, a=at(0), as_=128, out=at(0, 192), os_=128))
    # one dense piece in a gap between rows
    assert well_formed(dequantize(R=8, C=64, xs=128, x=at(0), scales=at(0, 128 + 8)))
    # fp32 outputs beside bf16 rows: equal strides in bytes
    assert well_formed(product(N=32, K=96, a=at(0), as_=160, out=at(0, 192), od=2, os_=80))


def test_rows_that_share_a_byte():
    assert combine_backward(rows=at(2, 8190), rs=8192, drows=at(2), drs=8192) == INV
    assert combine_backward(rows=at(2), rs=8191, drows=at(2, 8192), drs=8191) == INV
    assert combine(rows=at(2, 8192), rs=8192, out=at(2, 2), os_=8 * 8192) == INV
    assert dispatch(x=at(1), xs=8 * 8192, rows=at(1, 8190), rs=8192) == INV
    assert product(N=32, K=96, a=at(0), as_=128, out=at(0, 190), os_=128) == INV
    assert product(N=33, K=96, a=at(0), as_=128, out=at(0, 192), os_=128) == INV
    assert product_backward(N=96, K=33 + 31, a=at(0), as_=128, out=at(0, 192), os_=128) == INV
    assert dequantize(R=8, C=64, xs=128, x=at(0), scales=at(0, 128 + 120)) == INV
    # strides without a common step: their ends decide
    assert combine(rows=at(2), rs=4096, out=at(2, 512 * 8192 - 2), os_=4099) == INV
    assert well_formed(combine(rows=at(2), rs=4096, out=at(2, 512 * 8192), os_=4099))


def test_refusals_are_those_of_a_byte_count():
    """Random small byte rows: refused exactly when a byte is shared, for equal strides and single
    rows; never accepted when one is, whatever the strides."""
    rng = random.Random(4)
    seen = [0, 0]
    for i in range(4000):
        T, k, d = rng.choice([1, 2, 5]), rng.choice([1, 2, 3]), rng.randint(1, 12)
        xs, rs = d + rng.randint(0, 14), d + rng.randint(0, 14)
        if i % 2:
            rs = xs
        off = rng.randint(-60, 60)
        x = {G + off + t * xs + c for t in range(T) for c in range(d)}
        rows = {G + r * rs + c for r in range(T * k) for c in range(d)}
        p = dp(T=T, k=k, d=d, E=4, L=4, dtype=3)
        refused = dispatch(p, x=G + off, xs=xs, rows=G, rs=rs, ids=at(3), counts=None, offsets=None, perm=None,
                           inv=None) == INV
        shared = bool(x & rows)
        seen[shared] += 1
        assert refused or not shared, (T, k, d, xs, rs, off)
        if xs == rs or T == 1:
            assert refused == shared, (T, k, d, xs, rs, off)
    assert min(seen) > 500

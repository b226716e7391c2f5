"""CPU pins of the operators' fp64 oracle: MXFP4 against the format's definition,
the plan and the gradients against brute force and differences."""
import numpy as np
import pytest

from oracle import dispatch, mxfp4


def test_mxfp4_value_set_and_nibble_order():
    codes = np.array([[i | (((i + 1) & 15) << 4) for i in range(16)]], dtype=np.uint8)
    v = mxfp4.dequantize(codes, np.array([[127]], dtype=np.uint8))[0]
    table = [0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6]
    assert v[0::2].tolist() == table
    assert v[1::2].tolist() == table[1:] + table[:1]


def test_mxfp4_scale_of_the_largest_element():
    for top, byte in ((1.0, 125), (4.0, 127), (7.99, 127), (8.0, 128), (6.0, 127), (3.9999, 126),
                      (2.0 ** -126, 0), (2.0 ** -149, 0), (2.0 ** -124, 1), (float(np.finfo(np.float32).max), 252)):
        x = np.zeros((1, 32))
        x[0, 5] = -top
        assert mxfp4.quantize(x)[1][0, 0] == byte, top
    assert mxfp4.quantize(np.zeros((1, 32)))[1][0, 0] == 0
    for v in (np.inf, -np.inf, np.nan):
        x = np.ones((1, 64))
        x[0, 40] = v
        codes, scales = mxfp4.quantize(x)
        assert scales.tolist() == [[125, 255]] and not codes[0, 16:].any()
        assert np.isnan(mxfp4.dequantize(codes, scales)[0, 32:]).all()


def test_mxfp4_rounds_to_nearest_ties_to_even_and_saturates():
    x = np.zeros((1, 32))
    x[0, :12] = [7.5, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -5.0001, 0.2501, -0.25, 6.9]
    codes, scales = mxfp4.quantize(x)
    assert scales[0, 0] == 127
    assert mxfp4.dequantize(codes, scales)[0, :12].tolist() == [6, 0, 1, 1, 2, 2, 4, 4, -6, .5, -0., 6]


def test_mxfp4_round_trip_of_its_own_values():
    rng = np.random.default_rng(3)
    x = rng.standard_normal((40, 96)) * np.exp2(rng.integers(-30, 30, (40, 1)))
    codes, scales = mxfp4.quantize(x)
    v = mxfp4.dequantize(codes, scales)
    c2, s2 = mxfp4.quantize(v)
    assert np.array_equal(mxfp4.dequantize(c2, s2), v)
    # half a grid step at most (1/2 below 2, 1 below 4, 2 above), 6 ends the range (amax < 8)
    s = np.repeat(np.exp2(scales.astype(float) - 127), 32, axis=1)
    q = np.abs(x) / s
    step = np.where(q < 2, .5, np.where(q < 4, 1, 2))
    assert (np.abs(v - x) <= np.where(q > 6, 2.0, step / 2) * s).all()


@pytest.mark.parametrize("T,k,E,offset,L", [(1, 1, 1, 0, 1), (7, 3, 5, 1, 3), (40, 4, 9, 0, 9)])
def test_plan_is_a_stable_sort(T, k, E, offset, L):
    ids = np.random.default_rng(T).integers(-1, E + 1, (T, k))        # repeated and foreign ids among them
    counts, offsets, perm, inv = dispatch.plan(ids, offset, L)
    flat = ids.reshape(-1) - offset
    assert np.array_equal(perm, [p for e in range(L) for p in range(T * k) if flat[p] == e])
    assert np.array_equal(counts, [(flat == e).sum() for e in range(L)])
    assert offsets[0] == 0 and np.array_equal(np.diff(offsets), counts)
    for p in range(T * k):
        r = inv.reshape(-1)[p]
        assert (perm[r] == p) if 0 <= flat[p] < L else r == -1


def test_combine_backward_against_differences():
    rng = np.random.default_rng(1)
    ids = rng.integers(0, 4, (5, 3))
    _, _, perm, inv = dispatch.plan(ids, 1, 2)
    w, rows, dout = rng.standard_normal((5, 3)), rng.standard_normal((15, 6)), rng.standard_normal((5, 6))
    drows, dw, _ = dispatch.combine_backward(inv, w, rows, dout)
    f = lambda w_, r_: (dispatch.combine(inv, w_, r_)[0] * dout).sum()      # noqa: E731
    h = 1e-6
    for t in range(5):
        for j in range(3):
            d = np.zeros_like(w)
            d[t, j] = h
            assert abs((f(w + d, rows) - f(w - d, rows)) / (2 * h) - dw[t, j]) < 1e-7
    for r in range(len(perm)):
        d = np.zeros_like(rows)
        d[r, 2] = h
        assert abs((f(w, rows + d) - f(w, rows - d)) / (2 * h) - drows[r, 2]) < 1e-7
    assert np.isnan(drows[len(perm):]).all()


def test_product_backward_against_differences():
    rng = np.random.default_rng(2)
    a, w = rng.standard_normal((6, 8)), rng.standard_normal((3, 5, 8))
    off, dout = np.array([1, 3, 3, 5]), rng.standard_normal((6, 5))
    da = dispatch.product(dout, w, off, backward=True)[0]
    f = lambda x: np.nansum(dispatch.product(x, w, off)[0] * dout)          # noqa: E731
    for r in range(1, 5):
        for k in range(8):
            d = np.zeros_like(a)
            d[r, k] = 1e-6
            assert abs((f(a + d) - f(a - d)) / 2e-6 - da[r, k]) < 1e-7
    assert np.isnan(da[[0, 5]]).all()

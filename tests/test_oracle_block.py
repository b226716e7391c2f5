"""Pins of oracle/block.py: formats against torch's own conversion and the format's fields,
the choice against hand-made cases, gradients against central differences."""
import numpy as np
import pytest
import torch

from oracle import block


def test_e4m3_values_and_codes():
    codes = np.arange(256, dtype=np.uint8)
    want = torch.from_numpy(codes).view(torch.float8_e4m3fn).double().numpy()
    fine = (codes & 127) != 127
    got = block.mxfp8_dequantize(np.repeat(codes[:, None], 32, 1), np.full((256, 1), 127, np.uint8))[:, 0]
    assert np.array_equal(got[fine], want[fine]) and np.isnan(got[~fine]).all()
    assert np.array_equal(block.e4m3_codes(want[fine]), codes[fine])
    # every midpoint goes to the even code, its neighbours to their sides
    mid = (block.E4M3[1:] + block.E4M3[:-1]) / 2
    even = np.arange(126) + (np.arange(126) % 2)
    assert np.array_equal(block.e4m3_codes(mid), even)
    assert np.array_equal(block.e4m3_codes(np.nextafter(mid, 0)), np.arange(126))
    assert np.array_equal(block.e4m3_codes(np.nextafter(mid, 1e9)), np.arange(1, 127))
    assert np.array_equal(block.e4m3_codes(np.array([448.0, 463.9, 464.0, 511.0, -1e9])), [126, 126, 126, 126, 254])


def test_mxfp8_scales():
    x = np.zeros((6, 32))
    x[1, 3], x[2, 0], x[3, 31], x[4, 7], x[5, 5] = 256.0, -511.9, 2.0 ** -140, np.inf, 1.9
    codes, scales = block.mxfp8_quantize(x)
    assert scales[:, 0].tolist() == [0, 127, 127, 0, 255, 119]
    assert codes[1, 3] == 0x78 and codes[2, 0] == 0xFE and (codes[4] == 0).all()
    v = block.mxfp8_dequantize(codes, scales)
    assert v[1, 3] == 256 and v[2, 0] == -448 and np.isnan(v[4]).all()
    assert v[5, 5] == 1.75                               # 1.9 * 2^8 = 486.4 lies beyond 448: saturated


def test_route_by_hand():
    r = block.route_token
    ids, w, _ = r([0.0, 2.0, 1.0, 2.0], 2)
    assert ids.tolist() == [1, 3] and np.allclose(w, 0.5)                     # equal logits: the lower id first
    ids, w, _ = r([0.0, 2.0, 1.0, 2.0], 2, renormalize=False, scale=3.0)
    assert np.allclose(w, 3 * np.exp(2) / (1 + np.e + 2 * np.exp(2)))
    ids, w, _ = r([0.0, 2.0, 1.0, 2.0], 2, "sigmoid", bias=[1.0, 0, 0, 0])
    assert ids.tolist() == [0, 1]
    assert np.allclose(w, np.array([0.5, block.sigmoid(2)]) / (0.5 + block.sigmoid(2)))   # no bias in the weights
    # groups {0, 1}, {2, 3}: 2.0 + 1.9 beats 3.0 + 0
    ids, _, _ = r([3.0, -9.0, 2.0, 1.9], 2, "sigmoid", groups=2, top_groups=1)
    assert ids.tolist() == [2, 3]
    ids, _, _ = r([3.0, -9.0, 2.0, 1.9], 2, "sigmoid", groups=2, top_groups=1, group_keys=1)
    assert ids.tolist() == [0, 1]
    ids, w, _ = r([-np.inf, np.nan, -np.inf, 5.0], 2)
    assert ids.tolist() == [3, -1] and w.tolist() == [1.0, 0.0]
    ids, w, _ = r([-np.inf] * 4, 2, "sigmoid")
    assert ids.tolist() == [-1, -1] and w.tolist() == [0.0, 0.0]
    ids, w, _ = r([np.inf, 1.0, np.inf], 2)
    assert ids.tolist() == [0, 2] and w.tolist() == [0.5, 0.5]


def differences(f, x, h=1e-6):
    out = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        a, b = x.copy(), x.copy()
        a[i] += h
        b[i] -= h
        out[i] = (f(a) - f(b)) / (2 * h)
    return out


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [True, False])
def test_route_gradient_against_differences(kind, renormalize):
    rng = np.random.default_rng(1)
    l, dw = rng.normal(size=9), rng.normal(size=3)
    ids = np.array([4, 0, 7])

    def loss(x):
        s = block.scores(x, kind)[ids]
        return 2.5 * ((s / s.sum() if renormalize else s) * dw).sum()

    got = block.route_gradient(l, ids, dw, kind, renormalize, 2.5)
    assert np.abs(got - differences(loss, l)).max() < 1e-8
    assert np.array_equal(block.route_gradient(l, np.array([-1, 9, -1]), dw, kind, renormalize), np.zeros(9))


def test_norm_and_swiglu_gradients_against_differences():
    rng = np.random.default_rng(2)
    h, w, dy, dh = rng.normal(size=(3, 7)), rng.normal(size=7), rng.normal(size=(3, 7)), rng.normal(size=(3, 7))
    r = block.norm(h, w, 1e-5)[1]
    dx, dw = block.norm_gradient(h, w, r, dy, dh)
    assert np.abs(dx - dh - differences(lambda x: (block.norm(x, w, 1e-5)[0] * dy).sum(), h)).max() < 1e-8
    assert np.abs(dw - differences(lambda x: (block.norm(h, x, 1e-5)[0] * dy).sum(), w)).max() < 1e-8
    u, da = rng.normal(size=(2, 10)) * 3, rng.normal(size=(2, 5))
    assert np.abs(block.swiglu_gradient(u, da) - differences(lambda x: (block.swiglu(x) * da).sum(), u)).max() < 1e-8

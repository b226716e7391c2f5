"""GPU parity of moe_norm and its gradients with the fp64 oracle."""
import numpy as np
import pytest
import torch

import nvfp4_expert_layer_amd as nv
from oracle import block
from tests.gpu_helpers import log, require_gpu

pytestmark = pytest.mark.gpu

FLOATS = [torch.bfloat16, torch.float16, torch.float32]
U = 2.0 ** -24                                                   # half a step of fp32, relative
EPS = 1e-6


def draw(T, d, dtype, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(T, d, generator=g) * scale).to(dtype)


def view(t, pad):
    """t on the GPU, its rows `pad` elements apart and one element off (pad 0: dense)."""
    if not pad:
        return t.cuda()
    buf = torch.full((t.shape[0], t.shape[1] + pad), 3.0, dtype=t.dtype, device="cuda")
    buf[:, 1:1 + t.shape[1]] = t.cuda()
    return buf[:, 1:1 + t.shape[1]]


def forward(x, res, w, mx, eps=EPS, pad=0):
    T, d = x.shape
    p = nv.make_norm_problem(T, d, eps, x.dtype, w.dtype)
    h, y = view(torch.full_like(x, 7.0), pad), view(torch.full_like(x, 7.0), pad)
    q = nv.MXFP8Rows.empty(T, d) if mx else None
    rstd = torch.full((T,), 7.0, device="cuda")
    nv.moe_norm(p, view(x, pad), None if res is None else view(res, pad), w.cuda(), h, y, q, rstd)
    torch.cuda.synchronize()
    return h, y, q, rstd


def rstd_bound(d):
    """Relative: the mean's sum (at most 64 elements a thread, then trees and 16 waves in a row) and three
    more operations, halved by the root; the root and the division."""
    return ((min(d, 64) + 6 + 16 + 3) / 2 + 2) * U


def check_forward(x, res, w, mx, eps=EPS, pad=0):
    h, y, q, rstd = forward(x, res, w, mx, eps, pad)
    want_h = x if res is None else (x.float() + res.float()).to(x.dtype)
    assert torch.equal(h.cpu(), want_h)
    wy, wr = block.norm(want_h.double().numpy(), w.double().numpy(), eps)
    d = x.shape[1]
    assert (np.abs(rstd.double().cpu().numpy() - wr) <= rstd_bound(d) * wr).all()
    err = np.abs(y.double().cpu().numpy() - wy)
    half = torch.finfo(x.dtype).eps / 2
    tiny = float(torch.finfo(x.dtype).tiny) * half * 2           # half a step of the subnormals
    assert (err <= ((rstd_bound(d) + 2 * U) * 1.01 + half) * np.abs(wy) + tiny).all(), float((err / np.abs(wy)).max())
    if mx:
        # codes and scales of some fp32 y within the bound: a step is decided either way only at its border
        v = block.mxfp8_dequantize(q.codes.cpu().numpy(), q.scales.cpu().numpy())
        step = np.repeat(np.ldexp(1.0, q.scales.cpu().numpy().astype(int) - 127), 32, axis=1)
        near = (rstd_bound(d) + 2 * U) * 1.01 * np.abs(wy)
        over = np.maximum(np.abs(wy) - 448 * step, 0.0)          # saturated
        assert (np.abs(v - wy) <= np.maximum(2.0 ** -4 * np.abs(wy), 2.0 ** -10 * step) + near + over).all()
        _, scales = block.mxfp8_quantize(wy)
        off = scales != q.scales.cpu().numpy()
        top = np.abs(wy).reshape(len(wy), -1, 32).max(2)
        m = np.frexp(top)[0]
        assert not off.any() or (np.minimum(np.abs(m[off] - 0.5), 1 - m[off]) <= 2 * rstd_bound(d)).all()
        if x.dtype == torch.float32:                             # y holds the very values that were quantized
            q2 = nv.MXFP8Rows.empty(*x.shape)
            nv.moe_mxfp8_quantize(y, q2.codes, q2.scales)
            assert torch.equal(q.codes, q2.codes) and torch.equal(q.scales, q2.scales)
    return h, y, q, rstd


@pytest.mark.parametrize("dtype", FLOATS)
@pytest.mark.parametrize("T,d", [(1, 1), (3, 7), (2, 8), (5, 9), (1, 4096), (300, 100), (64, 513), (2100, 1000), (3, 8200),
                                 (2, 65535), (9, 2055)])
def test_norm(dtype, T, d):
    require_gpu()
    log(f"norm {dtype} {T}x{d}")
    x, r = draw(T, d, dtype, d), draw(T, d, dtype, d + 1)
    w = draw(1, d, torch.float32, 3)[0]
    check_forward(x, r, w.to(dtype), False)
    check_forward(x, None, w, False, pad=3)


@pytest.mark.parametrize("dtype", FLOATS)
@pytest.mark.parametrize("T,d", [(1, 32), (7, 64), (1, 4096), (50, 1056), (3000, 256), (2, 65536), (33, 4096), (5000, 4096)])
def test_norm_to_mxfp8(dtype, T, d):
    require_gpu()
    log(f"norm mxfp8 {dtype} {T}x{d}")
    x, r = draw(T, d, dtype, d), draw(T, d, dtype, d + 1)
    check_forward(x, r if d % 64 else None, (1 + 0.1 * draw(1, d, torch.float32, 3)[0]).to(torch.bfloat16), True, pad=5 * (T % 2))


def test_outputs_may_be_left_out():
    require_gpu()
    log("norm outputs")
    x, r, w = draw(40, 96, torch.bfloat16, 1), draw(40, 96, torch.bfloat16, 2), draw(1, 96, torch.bfloat16, 3)[0]
    h, y, q, rstd = check_forward(x, r, w, True)
    p = nv.make_norm_problem(40, 96, EPS)
    for skip in range(16):
        o = [torch.full_like(h, 9.0), torch.full_like(y, 9.0), nv.MXFP8Rows.empty(40, 96), torch.full_like(rstd, 9.0)]
        kept = [None if skip >> i & 1 else v for i, v in enumerate(o)]
        nv.moe_norm(p, x.cuda(), r.cuda(), w.cuda(), *kept)
        for i, (got, want) in enumerate(zip(kept, (h, y, q, rstd))):
            if got is None:
                assert i == 2 or (o[i] == 9).all()
            elif i == 2:
                assert torch.equal(got.codes, want.codes) and torch.equal(got.scales, want.scales)
            else:
                assert torch.equal(got, want)


@pytest.mark.parametrize("dtype", FLOATS)
def test_special_rows(dtype):
    """A row of zeros is scaled by 1 / sqrt(eps); Inf and NaN stay in their row."""
    require_gpu()
    log(f"norm specials {dtype}")
    x = draw(6, 64, dtype, 1)
    x[0] = 0
    x[2, 5], x[3, 9] = float("inf"), float("nan")
    x[4] = torch.finfo(dtype).tiny
    w = draw(1, 64, dtype, 2)[0]
    h, y, q, rstd = forward(x, None, w, True)
    assert torch.equal(h.cpu().nan_to_num(5.0), x.nan_to_num(5.0))
    assert abs(float(rstd[0]) - EPS ** -0.5) <= 3 * U * EPS ** -0.5 and (y[0] == 0).all() and (q.codes[0] & 127 == 0).all()
    assert rstd[2] == 0 and torch.isnan(rstd[3])
    assert torch.isnan(y[2, 5]) and (y[2].cpu()[torch.arange(64) != 5] == 0).all() and torch.isnan(y[3]).all()
    assert q.scales[2, 0] == 255 and q.scales[2, 1] != 255 and (q.scales[3] == 255).all()
    fine = [1, 4, 5]
    wy, _ = block.norm(x[fine].double().numpy(), w.double().numpy(), EPS)
    half = torch.finfo(dtype).eps / 2
    assert (np.abs(y[fine].double().cpu().numpy() - wy) <= (half + 60 * U) * np.abs(wy) + float(torch.finfo(dtype).tiny) * half * 2).all()


# --------------------------------------------------------------------- gradients
def backward(x, w, rstd, dy, dh, pad=0, want=(True, True)):
    T, d = x.shape
    p = nv.make_norm_problem(T, d, EPS, x.dtype, w.dtype)
    dx = view(torch.full_like(x, 7.0), pad) if want[0] else None
    dw = torch.full((d,), 7.0, device="cuda") if want[1] else None
    ws = nv.alloc_norm_workspace(p) if want[1] else None
    if ws is not None:
        ws.fill_(0xFF)                                           # NaN, were it read before it is written
    nv.moe_norm_backward(p, view(x, pad), w.cuda(), rstd, view(dy, pad), None if dh is None else view(dh, pad), dx, dw, ws)
    torch.cuda.synchronize()
    return dx, dw


def check_backward(x, w, dy, dh, pad=0):
    T, d = x.shape
    h = x.double().numpy()
    rstd = torch.from_numpy(block.norm(h, w.double().numpy(), EPS)[1]).float()
    r64, g64, w64 = rstd.double().numpy(), dy.double().numpy(), w.double().numpy()
    d64 = None if dh is None else dh.double().numpy()
    wx, ww = block.norm_gradient(h, w64, r64, g64, d64)
    dx, dw = backward(x, w, rstd.cuda(), dy, dh, pad)
    n = np.abs(h * r64[:, None])
    g = np.abs(g64 * w64)
    terms = min(d, 64) + 6 + 16 + 4                              # the mean: a thread's elements, trees, waves, products
    mag = r64[:, None] * (5 * g + n * (g * n).mean(1)[:, None] * (terms + 5)) + (0 if dh is None else 2 * np.abs(d64))
    half = torch.finfo(x.dtype).eps / 2
    err = np.abs(dx.double().cpu().numpy() - wx)
    assert (err <= U * 1.01 * mag + half * np.abs(wx) * 1.01 + float(torch.finfo(x.dtype).tiny) * half * 2).all()
    # a column's sum: a block's rows one after another, the blocks in 32 chains and a chain of 32
    blocks = max(1, nv.moe_norm_workspace_size(nv.make_norm_problem(T, d)) // (4 * d))
    chain = -(-T // blocks) + -(-blocks // 32) + 32 + 2
    lim = chain * U * 1.01 * (np.abs(g64) * n).sum(0) + 1e-38
    assert (np.abs(dw.double().cpu().numpy() - ww) <= lim).all()
    return rstd, dx, dw


@pytest.mark.parametrize("dtype", FLOATS)
@pytest.mark.parametrize("T,d", [(1, 1), (3, 7), (2, 8), (5, 9), (1, 4096), (300, 100), (64, 513), (2100, 1000), (3, 8200),
                                 (2, 65535), (9, 2055), (9000, 33), (600, 4096)])
def test_gradients(dtype, T, d):
    require_gpu()
    log(f"norm gradient {dtype} {T}x{d}")
    x, dy, dh = draw(T, d, dtype, d), draw(T, d, dtype, d + 1), draw(T, d, dtype, d + 2, 0.1)
    w = draw(1, d, torch.float32, 3)[0]
    check_backward(x, w.to(dtype), dy, dh)
    rstd, dx, dw = check_backward(x, w, dy, None, pad=3)
    # each output alone is the same
    x_only, _ = backward(x, w, rstd.cuda(), dy, None, want=(True, False))
    _, w_only = backward(x, w, rstd.cuda(), dy, None, want=(False, True))
    assert torch.equal(x_only, dx) and torch.equal(w_only, dw)


def test_gradient_against_differences():
    """The library's own y in fp32, moved by hand."""
    require_gpu()
    log("norm gradient differences")
    x, w, dy = draw(3, 40, torch.float32, 1), draw(1, 40, torch.float32, 2)[0], draw(3, 40, torch.float32, 3)
    rstd, dx, dw = check_backward(x, w, dy, None)
    step = 2.0 ** -7

    def loss(x, w):
        return float((forward(x, None, w, False)[1].double().cpu() * dy.double()).sum())

    for t, c in ((0, 0), (1, 17), (2, 39)):
        vals = []
        for sign in (1, -1):
            m = x.clone()
            m[t, c] += sign * step
            vals.append(loss(m, w))
        # y rounds by about 30 U of its size; the third derivative of a row's loss is below 40 |dy| |w| here
        mag = float((dy[t].abs() * w.abs()).sum())
        assert abs((vals[0] - vals[1]) / (2 * step) - float(dx[t, c])) <= 30 * U * 4 * mag / step + 40 * step ** 2 / 6 * mag
    for c in (0, 25):
        vals = []
        for sign in (1, -1):
            m = w.clone()
            m[c] += sign * step
            vals.append(loss(x, m))
        mag = float((dy.abs() * w.abs()).sum())
        assert abs((vals[0] - vals[1]) / (2 * step) - float(dw[c])) <= 30 * U * 4 * mag / step


def test_no_rows():
    """The weight's gradient of no rows is 0."""
    require_gpu()
    log("norm no rows")
    e = torch.empty(0, 64, dtype=torch.bfloat16)
    w = torch.ones(64, dtype=torch.bfloat16)
    forward(e, None, w, True)
    _, dw = backward(e, w, torch.empty(0, device="cuda"), e, None)
    assert (dw == 0).all()

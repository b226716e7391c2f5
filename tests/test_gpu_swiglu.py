"""GPU parity of moe_swiglu and its gradient with the fp64 oracle."""
import numpy as np
import pytest
import torch

import nvfp4_expert_layer_amd as nv
from oracle import block
from tests.gpu_helpers import log, require_gpu

pytestmark = pytest.mark.gpu

FLOATS = [torch.bfloat16, torch.float16, torch.float32]
U = 2.0 ** -24                                                   # half a step of fp32, relative


def draw(M, C, dtype, seed, scale=3.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(M, C, generator=g) * scale).to(dtype)


def view(t, pad):
    """t on the GPU, its rows `pad` elements apart and one element off (pad 0: dense)."""
    if not pad:
        return t.cuda()
    buf = torch.full((t.shape[0], t.shape[1] + pad), 3.0, dtype=t.dtype, device="cuda")
    buf[:, 1:1 + t.shape[1]] = t.cuda()
    return buf[:, 1:1 + t.shape[1]]


def offsets_of(M, live, groups):
    """Device offsets of `groups` groups that end at `live`."""
    cut = np.sort(np.random.default_rng(M + live).integers(0, live + 1, groups - 1))
    return torch.from_numpy(np.concatenate([[0], cut, [live]]).astype(np.int32)).cuda()


def filled(M, C):
    q = nv.MXFP8Rows.empty(M, C)
    q.codes.fill_(0x55)
    q.scales.fill_(0x66)
    return q


def untouched(q, live):
    return bool((q.codes[live:] == 0x55).all() and (q.scales[live:] == 0x66).all())


def forward(u, live=None, mx=True, pad=0, groups=3):
    M, F = u.shape[0], u.shape[1] // 2
    p = nv.make_swiglu_problem(M, F, groups, u.dtype)
    off = None if live is None else offsets_of(M, live, groups)
    a = view(torch.full((M, F), 7.0, dtype=u.dtype), pad)
    q, kept = (filled(M, F), filled(M, 2 * F)) if mx else (None, None)
    nv.moe_swiglu(p, view(u, pad), off, a, q, kept)
    torch.cuda.synchronize()
    n = M if live is None else live
    assert (a[n:] == 7).all()
    if mx:
        assert untouched(q, n) and untouched(kept, n)
    return a, q, kept


def bound(u):
    """Relative error of silu(gate): an exponential whose argument rounds, a sum, a division, a product."""
    return (8 + 2 * np.abs(np.minimum(u[:, :u.shape[1] // 2], 0))) * U


def check_forward(u, live=None, mx=True, pad=0):
    a, q, kept = forward(u, live, mx, pad)
    n = len(u) if live is None else live
    u64 = u[:n].double().numpy()
    want = block.swiglu(u64)
    half = torch.finfo(u.dtype).eps / 2
    tiny = float(torch.finfo(u.dtype).tiny) * half * 2
    err = np.abs(a[:n].double().cpu().numpy() - want)
    # (fp32 overflows in exp(-gate) beyond 88: the result is 0 there)
    lim = (bound(u64) + half) * np.abs(want) + tiny + np.where(u64[:, :u.shape[1] // 2] < -87, np.abs(want), 0)
    assert (err <= lim).all(), float((err / lim).max())
    if mx:
        codes, scales = block.mxfp8_quantize(u64)
        assert np.array_equal(kept.codes[:n].cpu().numpy(), codes) and np.array_equal(kept.scales[:n].cpu().numpy(), scales)
        v = block.mxfp8_dequantize(q.codes[:n].cpu().numpy(), q.scales[:n].cpu().numpy())
        step = np.repeat(np.ldexp(1.0, q.scales[:n].cpu().numpy().astype(int) - 127), 32, axis=1)
        over = np.maximum(np.abs(want) - 448 * step, 0.0)
        lim = np.maximum(2.0 ** -4 * np.abs(want), 2.0 ** -10 * step) + bound(u64) * np.abs(want) + over
        assert (np.abs(v - want) <= lim * 1.001).all()
        top = np.abs(want).reshape(n, want.shape[1] // 32, 32).max(2)
        off = block.mxfp8_quantize(want)[1] != q.scales[:n].cpu().numpy()
        m = np.frexp(top)[0]
        assert not off.any() or (np.minimum(np.abs(m[off] - 0.5), 1 - m[off]) <= 60 * U).all()
        if u.dtype == torch.float32:
            q2 = nv.MXFP8Rows.empty(*a.shape)
            nv.moe_mxfp8_quantize(a, q2.codes, q2.scales)
            assert torch.equal(q.codes[:n], q2.codes[:n]) and torch.equal(q.scales[:n], q2.scales[:n])
    return a, q, kept


@pytest.mark.parametrize("dtype", FLOATS)
@pytest.mark.parametrize("M,F", [(1, 1), (5, 7), (3, 8), (4, 9), (300, 100), (7, 65535), (1000, 515)])
def test_swiglu(dtype, M, F):
    require_gpu()
    log(f"swiglu {dtype} {M}x{F}")
    u = draw(M, 2 * F, dtype, M + F)
    check_forward(u, mx=False)
    check_forward(u, live=M // 2, mx=False, pad=3)


@pytest.mark.parametrize("dtype", FLOATS)
@pytest.mark.parametrize("M,F", [(1, 32), (512, 1024), (257, 96), (3, 65536), (4001, 160)])
def test_swiglu_to_mxfp8(dtype, M, F):
    require_gpu()
    log(f"swiglu mxfp8 {dtype} {M}x{F}")
    u = draw(M, 2 * F, dtype, M + F)
    for live in (None, M * 2 // 3, 0):
        check_forward(u, live, pad=5 if live else 0)


@pytest.mark.parametrize("dtype", FLOATS)
def test_specials(dtype):
    """Gates far from 0 both ways; Inf and NaN reach their own element (and, as MXFP8, their block)."""
    require_gpu()
    log(f"swiglu specials {dtype}")
    u = draw(4, 128, dtype, 1)
    u[0, :64] = torch.linspace(-120, 120, 64).to(dtype)
    u[1, :32] = -0.0
    u[1, 64:96] = 5.0
    check_forward(u)
    u[2, 3], u[2, 64 + 40], u[3, 7] = float("inf"), float("nan"), float("nan")
    a, q, kept = forward(u)
    bad = torch.isnan(a) | torch.isinf(a)
    assert bad.sum() == 3 and bad[2, 3] and bad[2, 40] and bad[3, 7]
    assert (q.scales == 255).sum() == 3 and (kept.scales == 255).sum() == 3


def check_backward(u, da, live=None, pad=0, mx=False):
    M, F = da.shape
    p = nv.make_swiglu_problem(M, F, 3, u.dtype)
    off = None if live is None else offsets_of(M, live, 3)
    n = M if live is None else live
    if mx:
        src = nv.MXFP8Rows.empty(M, 2 * F)
        nv.moe_mxfp8_quantize(u.cuda(), src.codes, src.scales)
        src.codes[n:] = 0x7F                                     # rows of no group are not looked at
        u64 = block.mxfp8_dequantize(src.codes[:n].cpu().numpy(), src.scales[:n].cpu().numpy())
    else:
        src, u64 = view(u, pad), u[:n].double().numpy()
    du = view(torch.full((M, 2 * F), 7.0, dtype=u.dtype), pad)
    nv.moe_swiglu_backward(p, src, off, view(da, pad), du)
    torch.cuda.synchronize()
    assert (du[n:] == 7).all()
    g, up, d = u64[:, :F], u64[:, F:], np.abs(da[:n].double().numpy())
    want = block.swiglu_gradient(u64, da[:n].double().numpy())
    s = block.sigmoid(g)
    rel = (14 + 2 * np.abs(g)) * U
    lim = np.concatenate([rel * d * np.abs(up) * s * (1 + np.abs(g)), rel * d * np.abs(g) * s], axis=1)
    lim += np.where(np.concatenate([g, g], axis=1) < -87, np.abs(want), 0)         # exp(-gate) overflows: 0
    half = torch.finfo(u.dtype).eps / 2
    err = np.abs(du[:n].double().cpu().numpy() - want)
    lim += half * np.abs(want) * 1.01 + float(torch.finfo(u.dtype).tiny) * half * 2
    assert (err <= lim).all(), float((err / lim).max())


@pytest.mark.parametrize("dtype", FLOATS)
@pytest.mark.parametrize("M,F", [(1, 1), (5, 7), (3, 8), (4, 9), (300, 100), (7, 65535), (1000, 515), (600, 1024)])
def test_gradient(dtype, M, F):
    require_gpu()
    log(f"swiglu gradient {dtype} {M}x{F}")
    u, da = draw(M, 2 * F, dtype, M + F), draw(M, F, dtype, M, 0.5)
    u[0, 0] = -100.0
    check_backward(u, da)
    check_backward(u, da, live=M // 2, pad=3)


@pytest.mark.parametrize("dtype", FLOATS)
@pytest.mark.parametrize("M,F", [(1, 32), (512, 1024), (257, 96), (3, 65536), (4001, 160)])
def test_gradient_from_mxfp8(dtype, M, F):
    require_gpu()
    log(f"swiglu gradient mxfp8 {dtype} {M}x{F}")
    u, da = draw(M, 2 * F, dtype, M + F), draw(M, F, dtype, M, 0.5)
    for live in (None, M * 2 // 3, 0):
        check_backward(u, da, live, pad=5 if live else 0, mx=True)


def test_gradient_against_differences():
    require_gpu()
    log("swiglu gradient differences")
    u, da = draw(2, 20, torch.float32, 1, 1.0), draw(2, 10, torch.float32, 2, 1.0)
    p = nv.make_swiglu_problem(2, 10, 1, torch.float32)
    du = torch.empty(2, 20, device="cuda")
    nv.moe_swiglu_backward(p, u.cuda(), None, da.cuda(), du)
    h = 2.0 ** -7
    for r, c in ((0, 0), (0, 13), (1, 9), (1, 19)):
        vals = []
        for sign in (1, -1):
            m = u.clone()
            m[r, c] += sign * h
            vals.append(float((forward(m, mx=False)[0].double().cpu() * da.double()).sum()))
        e = c % 10
        mag = float(da[r, e].abs()) * (1 + float(u[r, 10 + e].abs()))
        # silu's third derivative is below 0.6, a rounds by 12 U of its size (here below 4)
        assert abs((vals[0] - vals[1]) / (2 * h) - float(du[r, c])) <= mag * (0.6 * h * h / 6 + 12 * U * 8 / h)


def test_no_rows_and_far_offsets():
    """No rows; offsets that claim more rows than there are, or fewer than none."""
    require_gpu()
    log("swiglu offsets")
    check_forward(torch.empty(0, 64, dtype=torch.bfloat16), mx=True)
    u = draw(5, 64, torch.bfloat16, 1)
    p = nv.make_swiglu_problem(5, 32, 2)
    whole = torch.zeros(5, 32, dtype=torch.bfloat16, device="cuda")
    nv.moe_swiglu(p, u.cuda(), None, whole, None, None)
    for last, live in ((9, 5), (1 << 30, 5), (-3, 0)):
        a = torch.zeros(5, 32, dtype=torch.bfloat16, device="cuda")
        nv.moe_swiglu(p, u.cuda(), torch.tensor([0, 1, last], dtype=torch.int32, device="cuda"), a, None, None)
        assert torch.equal(a[:live], whole[:live]) and (a[live:] == 0).all()

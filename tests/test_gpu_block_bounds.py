"""What include/moe_block.h states of the operators' ranges: the norm's magnitudes, SwiGLU's far gates, MXFP8's
smallest values; and that a call writes its outputs alone."""
import numpy as np
import pytest
import torch

import nvfp4_expert_layer_amd as nv
from tests.gpu_helpers import log, require_gpu

pytestmark = pytest.mark.gpu

U = 2.0 ** -24                                                   # half a step of fp32, relative


def norm(x, eps):
    T, d = x.shape
    y, rstd = torch.empty_like(x), torch.empty(T, device="cuda")
    nv.moe_norm(nv.make_norm_problem(T, d, eps, x.dtype, torch.float32), x, None, torch.ones(d, device="cuda"), None, y,
                None, rstd)
    return y.double().cpu().numpy(), rstd.double().cpu().numpy()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d", [1, 7, 64, 100, 4096, 10000, 65536])
def test_norm_magnitudes(dtype, d):
    """Rows of alike magnitudes up to 2^64 / sqrt(d), beyond which rstd and y are 0; with eps 0 down to 2^-63, and
    rstd Inf where every square vanishes."""
    require_gpu()
    log(f"norm magnitudes {dtype} d={d}")
    top = 2.0 ** 64 / d ** 0.5
    m = torch.tensor([0.98 * top, 1.01 * top, 2.0 ** -62, 2.0 ** -80]).to(dtype)      # (bf16 rounds by 2^-9)
    sign = torch.where(torch.arange(d) % 3 == 0, -1.0, 1.0).to(dtype)
    x = m.unsqueeze(1) * sign
    y, rstd = norm(x.cuda(), 0.0)
    want = 1 / np.abs(m.double().numpy())
    # up to 64 squares in a row a thread, 6 steps of a wave, 16 waves: 86 roundings, halved by the root; four more
    for i in (0, 2):
        assert abs(rstd[i] - want[i]) <= 50 * U * want[i]
        assert (np.abs(y[i] - sign.double().numpy()) <= 60 * U + torch.finfo(dtype).eps / 2).all()
    assert rstd[1] == 0 and (y[1] == 0).all() and rstd[3] == np.inf
    # beside eps a mean square below 2^-25 of it leaves no trace
    _, rstd = norm(torch.full((1, d), 2.0 ** -24, dtype=dtype, device="cuda"), 2.0 ** -20)
    assert rstd[0] == 2.0 ** 10


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_swiglu_of_far_gates(dtype):
    """From gates of about -88 on a and du are 0, whose values are below 2^-121 of |up|, |da up| and |da|."""
    require_gpu()
    log(f"swiglu far gates {dtype}")
    F = 64
    gate = torch.linspace(-120.0, -70.0, F).to(dtype)
    u = torch.cat([gate, torch.linspace(-4, 4, F).to(dtype)]).unsqueeze(0)
    da = torch.linspace(-2, 2, F).to(dtype).unsqueeze(0)
    p = nv.make_swiglu_problem(1, F, 1, dtype)
    a, du = torch.empty(1, F, dtype=dtype, device="cuda"), torch.empty(1, 2 * F, dtype=dtype, device="cuda")
    nv.moe_swiglu(p, u.cuda(), None, a, None, None)
    nv.moe_swiglu_backward(p, u.cuda(), None, da.cuda(), du)
    g, up, d = gate.double(), u[0, F:].double(), da[0].double()
    s = torch.sigmoid(g)
    want = torch.stack([g * s * up, d * up * s * (1 + g * (1 - s)), d * g * s])
    mag = torch.stack([up.abs(), (d * up).abs(), d.abs()])
    got = torch.cat([a, du[:, :F], du[:, F:]]).double().cpu()
    far = g < -88.8
    assert (got[:, far] == 0).all() and (want[:, far].abs() <= 2.0 ** -121 * mag[:, far]).all()
    near = g > -87
    half, tiny = torch.finfo(dtype).eps / 2, float(torch.finfo(dtype).smallest_normal) * torch.finfo(dtype).eps
    lim = ((14 + 2 * g[near].abs()) * U * (1 + g[near].abs()) / g[near].abs() * 1.1 + half) * want[:, near].abs() + tiny
    assert ((got - want)[:, near].abs() <= lim).all()


def test_dequantizer_below_bf16():
    """Exact in f32 for every scale byte; in bf16 from byte 3 on, below it to nearest, ties to even."""
    require_gpu()
    log("mxfp8 smallest values")
    codes = torch.arange(256, dtype=torch.uint8).repeat(8, 1).cuda()
    scales = torch.arange(8, dtype=torch.uint8).unsqueeze(1).repeat(1, 8).cuda()
    f, b = torch.empty(8, 256, device="cuda"), torch.empty(8, 256, dtype=torch.bfloat16, device="cuda")
    nv.moe_mxfp8_dequantize(codes, scales, f)
    nv.moe_mxfp8_dequantize(codes, scales, b)
    fine = ~torch.isnan(f)
    assert fine.sum() == 8 * 254
    # f32 by the format's own fields
    c = torch.arange(256).double()
    e, m = (c.int() >> 3 & 15).double(), (c.int() & 7).double()
    v = torch.where(e == 0, m / 8 * 2.0 ** -6, (1 + m / 8) * torch.exp2(e - 7)) * torch.where(c >= 128, -1.0, 1.0)
    want = v * torch.exp2(torch.arange(8).double() - 127).unsqueeze(1)
    assert torch.equal(f.double().cpu()[fine.cpu()], want[fine.cpu()])
    same = b.double() == f.double()
    assert same[3:][fine[3:]].all() and not same[:3][fine[:3]].all()
    step = 2.0 ** -133                                              # bf16's smallest value: its step down here
    low = fine & (f.abs() < 2.0 ** -126)
    err = (b.double() - f.double()).abs() / step
    assert (err[low] <= 0.5).all()
    tie = low & (err == 0.5)
    assert tie.any() and ((b.double()[tie] / step) % 2 == 0).all()


@pytest.mark.parametrize("T,d,dtype", [(40, 96, torch.bfloat16), (3, 4096, torch.float32), (700, 32, torch.float16)])
def test_norm_writes_what_is_asked_for(T, d, dtype):
    """Every choice of outputs, each between neighbours of one buffer: no byte beside them changes."""
    require_gpu()
    log(f"norm outputs between neighbours {dtype} {T}x{d}")
    x, r = torch.randn(T, d, device="cuda").to(dtype), torch.randn(T, d, device="cuda").to(dtype)
    w, es = torch.ones(d, device="cuda"), x.element_size()
    p = nv.make_norm_problem(T, d, 1e-6, dtype, torch.float32)
    sizes = [T * d * es, T * d * es, T * d, T * (d // 32), T * 4]
    starts, at = [], 64
    for n in sizes:
        starts.append(at)
        at += (n + 63) // 16 * 16 + 16                              # 32 to 48 bytes between
    first = None
    for skip in range(16):
        buf = torch.full((at,), 0x5A, dtype=torch.uint8, device="cuda")
        part = [buf[s:s + n] for s, n in zip(starts, sizes)]
        h, y = (part[i].view(dtype).view(T, d) for i in (0, 1))
        q, rstd = nv.MXFP8Rows(part[2].view(T, d), part[3].view(T, d // 32)), part[4].view(torch.float32)
        kept = [None if skip >> i & 1 else v for i, v in enumerate((h, y, q, rstd))]
        nv.moe_norm(p, x, r, w, *kept)
        wrote = torch.zeros(at, dtype=torch.bool, device="cuda")
        for i, s in enumerate((0, 1, 2, 2, 3)):
            if kept[s] is not None:
                wrote[starts[i]:starts[i] + sizes[i]] = True
        assert (buf[~wrote] == 0x5A).all()
        first = buf if first is None else first                     # all four outputs
        assert torch.equal(buf[wrote], first[wrote])
    assert (first != 0x5A).any()

"""The operators' C entry points on the CPU: every declared symbol is exported, and
every refusal comes back as its status before anything is enqueued (the pointers
are never followed)."""
import ctypes
import os
import re

import pytest

import nvfp4_expert_layer_amd as nv
from nvfp4_expert_layer_amd import ops

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
INV, SHAPE, SMALL = nv.ERR_INVALID_ARG, nv.ERR_UNSUPPORTED_SHAPE, nv.ERR_WORKSPACE_TOO_SMALL


def test_library_exports_every_declared_symbol():
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "moe_ops.h")).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(moe_\w+)\s*\(", text)))
    assert len(names) == 9
    for n in names:
        assert hasattr(nv.lib(), n) and getattr(ops._lib(), n).argtypes is not None, n


def dp(**kw):
    a = dict(T=64, d=4096, E=320, k=8, offset=0, L=160)
    a.update(kw)
    dt = a.pop("dtype", 0)
    p = nv.make_dispatch_problem(**a)
    p.dtype = dt
    return ctypes.byref(p)


G = 1 << 32          # made-up device addresses, 4 GiB apart


def at(i, off=0):
    return (i + 1) * G + off


def dispatch(p=None, ids=at(0), x=at(1), xs=4096, counts=at(2), offsets=at(3), perm=at(4), inv=at(5), rows=at(6),
             rs=4096, ws=at(7), wb=1 << 30):
    return ops._lib().moe_dispatch(dp() if p is None else p, ids, x, xs, counts, offsets, perm, inv, rows, rs, ws, wb,
                                   None)


def well_formed(status):
    """Past every check there is no gfx950 device here."""
    return status in (nv.ERR_HIP, nv.ERR_ARCH, nv.OK)


def test_dispatch_workspace_size():
    assert nv.moe_dispatch_workspace_size(nv.make_dispatch_problem(64, 8, 320, 8, 0, 160)) == 0
    big = nv.make_dispatch_problem(1 << 17, 8, 320, 8, 0, 160)
    n = nv.moe_dispatch_workspace_size(big)
    assert n > 160 * 4
    assert dispatch(ctypes.byref(big), wb=n - 1) == SMALL
    assert dispatch(ctypes.byref(big), ws=None) == INV
    assert ops._lib().moe_dispatch_workspace_size(ctypes.byref(big), None) == INV


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), INV), (dict(k=0), INV), (dict(k=33), INV), (dict(E=1025), SHAPE), (dict(E=0), SHAPE),
    (dict(L=0), INV), (dict(offset=-1), INV), (dict(offset=200), INV), (dict(d=0), SHAPE), (dict(d=65537), SHAPE),
    (dict(dtype=4), INV), (dict(dtype=-1), INV), (dict(T=1 << 25), SHAPE),
])
def test_dispatch_problem_refusals(kw, status):
    assert dispatch(dp(**kw)) == status
    assert nv.moe_nvfp4_last_error() != ""
    if kw.get("dtype") is None:
        assert combine(dp(**kw)) == status and combine_backward(dp(**kw)) == status


@pytest.mark.parametrize("kw", [
    dict(ids=None), dict(ids=at(0, 2)), dict(counts=at(2, 1)), dict(offsets=at(3, 2)), dict(perm=at(4, 3)),
    dict(inv=at(5, 2)), dict(x=None), dict(rows=None), dict(x=at(1, 1)), dict(rows=at(6, 1)), dict(xs=4095),
    dict(rs=0), dict(rows=at(1, 64 * 4096 * 2 - 2)), dict(perm=at(5, 64 * 8 * 4 - 4)), dict(counts=at(3, 4)),
    dict(inv=at(0)), dict(offsets=at(1)),
])
def test_dispatch_argument_refusals(kw):
    assert dispatch(**kw) == INV
    assert well_formed(dispatch())
    assert well_formed(dispatch(x=None, rows=None, perm=None, counts=None))
    # byte rows need no alignment; a last row reaches only to its width
    assert well_formed(dispatch(dp(dtype=3), x=at(1, 1), rows=at(6, 3)))
    assert well_formed(dispatch(rows=at(1, 64 * 4096 * 2)))
    # no token: token pointers are not looked at
    assert well_formed(dispatch(dp(T=0), ids=None, x=None, rows=at(6), inv=None, perm=None))


def combine(p=None, inv=at(0), w=at(1), rows=at(2), rs=4096, out=at(3), os_=4096):
    return ops._lib().moe_combine(dp() if p is None else p, inv, w, rows, rs, out, os_, None)


@pytest.mark.parametrize("kw", [
    dict(inv=None), dict(w=None), dict(rows=None), dict(out=None), dict(inv=at(0, 2)), dict(w=at(1, 1)),
    dict(rows=at(2, 1)), dict(out=at(3, 1)), dict(rs=4000), dict(os_=4095), dict(out=at(2, 64)), dict(out=at(0)),
    dict(out=at(1, 8)), dict(p=dp(dtype=3)),
])
def test_combine_argument_refusals(kw):
    assert combine(**kw) == INV
    assert well_formed(combine())
    if "w" not in kw and kw.get("out") != at(1, 8):
        back = dict(p=dp(), inv=at(0), rows=at(2), rs=4096, out=at(3), os_=4096)
        back.update(kw)
        assert ops._lib().moe_dispatch_backward(back["p"], back["inv"], back["rows"], back["rs"], back["out"],
                                                back["os_"], None) == INV


def combine_backward(p=None, inv=at(0), w=at(1), rows=at(2), rs=4096, dout=at(3), dos=4096, drows=at(4), drs=4096,
                     dw=at(5)):
    return ops._lib().moe_combine_backward(dp() if p is None else p, inv, w, rows, rs, dout, dos, drows, drs, dw, None)


@pytest.mark.parametrize("kw", [
    dict(inv=None), dict(w=None), dict(rows=None), dict(dout=None), dict(dw=at(5, 2)), dict(drows=at(4, 1)),
    dict(dos=1), dict(drs=4095), dict(rs=2), dict(drows=at(2)), dict(drows=at(3, 128)), dict(dw=at(1)),
    dict(dw=at(4, 4096)), dict(p=dp(dtype=3)),
])
def test_combine_backward_argument_refusals(kw):
    assert combine_backward(**kw) == INV
    assert well_formed(combine_backward())
    assert well_formed(combine_backward(rows=None, dw=None))
    assert well_formed(combine_backward(drows=None))


def quantize(dtype=0, R=8, C=64, xs=64, x=at(0), codes=at(1), scales=at(2)):
    return ops._lib().moe_mxfp4_quantize(x, dtype, R, C, xs, codes, scales, None)


def dequantize(dtype=0, R=8, C=64, xs=64, x=at(0), codes=at(1), scales=at(2)):
    return ops._lib().moe_mxfp4_dequantize(codes, scales, R, C, dtype, x, xs, None)


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=3), INV), (dict(R=-1), INV), (dict(C=-32), INV), (dict(C=48), SHAPE), (dict(R=1 << 40), SHAPE),
    (dict(xs=63), INV), (dict(x=None), INV), (dict(codes=None), INV), (dict(scales=None), INV),
    (dict(codes=at(1, 8)), INV), (dict(x=at(0, 1)), INV), (dict(x=at(1)), INV), (dict(xs=1 << 40), SHAPE),
])
def test_mxfp4_refusals(kw, status):
    for f in (quantize, dequantize):
        assert f(**kw) == status, f
        assert well_formed(f()) and well_formed(f(R=0, x=None, codes=None, scales=None))
        assert well_formed(f(R=1, xs=0)) and well_formed(f(x=at(0, 2), scales=at(2, 1)))
    assert quantize(codes=at(2)) == INV


def product(M=64, N=100, K=96, groups=4, a=at(0), a_s=None, as_=96, w=at(2), w_s=at(3), off=at(4), out=at(5), od=0,
            os_=100):
    p = nv.make_product_problem(M, N, K, groups)
    return ops._lib().moe_mxfp4_product(ctypes.byref(p), a, a_s, as_, w, w_s, off, out, od, os_, None)


def product_backward(M=64, N=100, K=96, groups=4, a=at(0), as_=100, w=at(2), w_s=at(3), off=at(4), out=at(5), od=0,
                     os_=96):
    p = nv.make_product_problem(M, N, K, groups)
    return ops._lib().moe_mxfp4_product_backward(ctypes.byref(p), a, as_, w, w_s, off, out, od, os_, None)


@pytest.mark.parametrize("kw,status", [
    (dict(M=-1), INV), (dict(N=0), SHAPE), (dict(N=65537, os_=1 << 17), SHAPE), (dict(K=48), SHAPE), (dict(K=0), SHAPE),
    (dict(K=65568), SHAPE), (dict(groups=0), SHAPE), (dict(groups=1025), SHAPE), (dict(a=None), INV),
    (dict(w=None), INV), (dict(w_s=None), INV), (dict(off=None), INV), (dict(out=None), INV), (dict(w=at(2, 8)), INV),
    (dict(off=at(4, 2)), INV), (dict(od=3), INV), (dict(os_=95), INV), (dict(out=at(5, 1)), INV), (dict(out=at(0)), INV),
    (dict(out=at(2)), INV), (dict(out=at(4)), INV), (dict(as_=95), INV),
])
def test_product_refusals(kw, status):
    assert product(**kw) == status
    assert product_backward(**kw) == status
    assert well_formed(product()) and well_formed(product_backward())
    for f in (product, product_backward):
        assert well_formed(f(off=None, groups=1)) and well_formed(f(M=0, a=None, out=None))
    # row operand: 16-byte rows forward, any element alignment backward
    assert product(as_=100) == INV and product(a=at(0, 2)) == INV
    assert well_formed(product_backward(as_=101, a=at(0, 2)))
    assert product(a_s=at(1), a=at(0, 8)) == INV and well_formed(product(a_s=at(1, 1), as_=0))


@pytest.mark.parametrize("kw,msg", [
    (dict(a="f32"), "a: dtype"), (dict(a="short"), "a: shape"), (dict(a="strided"), "a: elements"),
    (dict(out="short"), "out: shape"), (dict(off="short"), "offsets: shape"), (dict(w="short"), "w.codes: shape"),
    (dict(a="codes"), "a.scales: shape"), (dict(), "must be on the GPU"),
])
def test_binding_checks_tensors(kw, msg):
    import torch
    p = nv.make_product_problem(6, 10, 64, 2)
    bf = torch.bfloat16
    a = {"f32": torch.zeros(6, 64), "short": torch.zeros(5, 64, dtype=bf),
         "strided": torch.zeros(64, 6, dtype=bf).t(), "codes": nv.MXFP4Rows(torch.zeros(6, 32, dtype=torch.uint8),
                                                                        torch.zeros(6, 1, dtype=torch.uint8)),
         None: torch.zeros(6, 64, dtype=bf)}[kw.get("a")]
    w = nv.MXFP4Weights.empty(1 if "w" in kw else 2, 10, 64, device="cpu")
    off = torch.zeros(2 if "off" in kw else 3, dtype=torch.int32)
    out = torch.zeros(6, 9 if "out" in kw else 10)
    with pytest.raises(ValueError, match=msg):
        nv.moe_mxfp4_product(p, a, w, off, out)


def test_binding_checks_dispatch_tensors():
    import torch
    p = nv.make_dispatch_problem(4, 16, 8, 2, 0, 8, torch.float16)
    i32 = torch.int32
    ok = dict(ids=torch.zeros(4, 2, dtype=i32), x=torch.zeros(4, 16, dtype=torch.float16), counts=None, offsets=None,
              perm=None, inv=None, rows=torch.zeros(8, 16, dtype=torch.float16),
              workspace=torch.zeros(0, dtype=torch.uint8))
    for bad, msg in ((dict(ids=torch.zeros(4, 2, dtype=torch.int64)), "ids: dtype"),
                     (dict(x=torch.zeros(4, 16)), "x: dtype"), (dict(rows=torch.zeros(7, 16, dtype=torch.float16)),
                                                                "rows: shape"),
                     (dict(counts=torch.zeros(7, dtype=i32)), "counts: shape"), (dict(), "must be on the GPU")):
        with pytest.raises(ValueError, match=msg):
            nv.moe_dispatch(p, **{**ok, **bad})
    with pytest.raises(ValueError, match="dtype"):
        nv.make_dispatch_problem(4, 16, 8, 2, 0, 8, torch.float64)

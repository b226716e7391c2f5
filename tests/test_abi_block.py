"""The C entry points of include/moe_block.h on the CPU: every declared symbol is exported,
and every refusal comes back as its status before anything is enqueued (the pointers are
never followed); the binding refuses tensors of another dtype, shape, layout or device."""
import ctypes
import os
import re

import pytest
import torch

import nvfp4_expert_layer_amd as nv
from nvfp4_expert_layer_amd import block

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
INV, SHAPE, SMALL = nv.ERR_INVALID_ARG, nv.ERR_UNSUPPORTED_SHAPE, nv.ERR_WORKSPACE_TOO_SMALL
G = 1 << 36          # made-up device addresses


def at(i, off=0):
    return (i + 1) * G + off


def well_formed(status):
    """Past every check there is no gfx950 device here."""
    return status in (nv.ERR_HIP, nv.ERR_ARCH, nv.OK)


def test_library_exports_every_declared_symbol():
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "moe_block.h")).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(moe_\w+)\s*\(", text)))
    assert len(names) == 10
    for n in names:
        assert hasattr(nv.lib(), n) and getattr(block._lib(), n).argtypes is not None, n


# ------------------------------------------------------------------------ route
def rp(**kw):
    late = {n: kw.pop(n) for n in ("dtype", "scale", "renormalize") if n in kw}
    p = nv.make_route_problem(**{**dict(T=64, E=320, k=8), **kw})
    for n, v in late.items():
        setattr(p, n, v)
    return ctypes.byref(p)


def route(p=None, logits=at(0), ls=320, bias=at(1), ids=at(2), w=at(3)):
    return block._lib().moe_route(p or rp(), logits, ls, bias, ids, w, None)


def route_backward(p=None, logits=at(0), ls=320, ids=at(1), dw=at(2), dl=at(3), ds=320):
    return block._lib().moe_route_backward(p or rp(), logits, ls, ids, dw, dl, ds, None)


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), INV), (dict(E=0), SHAPE), (dict(E=1025), SHAPE), (dict(k=0), INV), (dict(k=33), INV),
    (dict(E=4, k=5), INV), (dict(scores=2), INV), (dict(scores=-1), INV), (dict(groups=0), SHAPE),
    (dict(groups=65, E=650), SHAPE), (dict(groups=7), INV), (dict(groups=8, top_groups=0), INV),
    (dict(groups=8, top_groups=9), INV), (dict(groups=160, E=320), SHAPE), (dict(group_keys=0), INV),
    (dict(group_keys=3), INV), (dict(groups=64, top_groups=1, k=6), INV), (dict(renormalize=2), INV),
    (dict(dtype=3), INV), (dict(dtype=-1), INV), (dict(scale=float("nan")), INV), (dict(scale=float("inf")), INV),
    (dict(T=1 << 25), SHAPE),
])
def test_route_problem_refusals(kw, status):
    assert route(rp(**kw)) == status and nv.moe_nvfp4_last_error() != ""
    assert route_backward(rp(**kw)) == status


def test_route_argument_refusals():
    for kw in (dict(logits=None), dict(ids=None), dict(w=None), dict(ids=at(2, 2)), dict(w=at(3, 1)), dict(bias=at(1, 2)),
               dict(logits=at(0, 2)), dict(ls=319), dict(ids=at(3)), dict(ids=at(0, 64)), dict(w=at(1, 4 * 319)),
               dict(w=at(2, 64 * 8 * 4 - 4))):
        assert route(**kw) == INV, kw
    for kw in (dict(logits=None), dict(ids=None), dict(dw=None), dict(dl=None), dict(ds=300), dict(dl=at(0)),
               dict(dl=at(0, 63 * 1280)), dict(dl=at(1)), dict(dl=at(2)), dict(dw=at(2, 3))):
        assert route_backward(**kw) == INV, kw
    assert block._lib().moe_route(None, at(0), 320, None, at(2), at(3), None) == INV
    assert well_formed(route()) and well_formed(route(bias=None)) and well_formed(route(ls=1000))
    assert well_formed(route(rp(groups=64, top_groups=2))) and well_formed(route_backward())
    # logits and their gradient in different columns of one buffer; no token: nothing is looked at
    assert well_formed(route_backward(ls=640, dl=at(0, 1280), ds=640))
    assert well_formed(route(rp(T=0), None, 0, None, None, None)) and well_formed(route_backward(rp(T=0), *[None, 0] * 3))


# ------------------------------------------------------------------------- norm
def np_(**kw):
    late = {n: kw.pop(n) for n in ("dtype", "weight_dtype", "eps") if n in kw}
    p = nv.make_norm_problem(**{**dict(T=64, d=4096), **kw})
    for n, v in late.items():
        setattr(p, n, v)
    return ctypes.byref(p)


def norm(p=None, x=at(0), xs=4096, r=at(1), rs=4096, w=at(2), h=at(3), hs=4096, y=at(4), ys=4096, c=at(5), s=at(6),
         rstd=at(7)):
    return block._lib().moe_norm(p or np_(), x, xs, r, rs, w, h, hs, y, ys, c, s, rstd, None)


def norm_backward(p=None, h=at(0), hs=4096, w=at(1), rstd=at(2), dy=at(3), dys=4096, dh=at(4), dhs=4096, dx=at(5),
                  dxs=4096, dw=at(6), ws=at(7), wb=1 << 30):
    return block._lib().moe_norm_backward(p or np_(), h, hs, w, rstd, dy, dys, dh, dhs, dx, dxs, dw, ws, wb, None)


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), INV), (dict(T=(1 << 27) + 1), INV), (dict(d=0), SHAPE), (dict(d=65537), SHAPE), (dict(dtype=3), INV),
    (dict(weight_dtype=3), INV), (dict(weight_dtype=-1), INV), (dict(eps=-1e-6), INV), (dict(eps=float("nan")), INV),
    (dict(eps=float("inf")), INV),
])
def test_norm_problem_refusals(kw, status):
    assert norm(np_(**kw)) == status and norm_backward(np_(**kw)) == status
    assert block._lib().moe_norm_workspace_size(np_(**kw), ctypes.byref(ctypes.c_size_t())) == status


def test_norm_argument_refusals():
    for kw in (dict(x=None), dict(w=None), dict(xs=4095), dict(rs=1), dict(hs=4000), dict(ys=4095), dict(x=at(0, 1)),
               dict(h=at(3, 1)), dict(y=at(4, 1)), dict(w=at(2, 1)), dict(c=None), dict(s=None), dict(c=at(5, 8)),
               dict(rstd=at(7, 2)), dict(h=at(1)), dict(h=at(0)), dict(y=at(3, 64)), dict(c=at(4)), dict(s=at(5, 64)),
               dict(rstd=at(2, 4)), dict(y=at(2, 4096))):
        assert norm(**kw) == INV, kw
    assert norm(np_(d=4008)) == SHAPE                                        # no whole blocks
    assert well_formed(norm(np_(d=4008), c=None, s=None))
    assert well_formed(norm()) and well_formed(norm(r=None, h=None, y=None))
    assert well_formed(norm(np_(T=0), **{n: None for n in ("x", "r", "w", "h", "y", "c", "s", "rstd")}))
    for kw in (dict(h=None), dict(rstd=None), dict(dy=None), dict(w=None), dict(hs=1), dict(dys=4095), dict(dhs=9),
               dict(dxs=4095), dict(dw=at(6, 2)), dict(dx=at(0)), dict(dx=at(3)), dict(dx=at(4)), dict(dw=at(1)),
               dict(ws=at(5)), dict(ws=None), dict(ws=at(7, 2)), dict(dw=at(7, 64))):
        assert norm_backward(**kw) == INV, kw
    p = nv.make_norm_problem(64, 4096)
    n = nv.moe_norm_workspace_size(p)
    assert n >= 4 * 4096 and norm_backward(wb=n - 1) == SMALL and well_formed(norm_backward(wb=n))
    assert well_formed(norm_backward(dw=None, ws=None, wb=0)) and well_formed(norm_backward(dx=None, w=None, dh=None))
    assert nv.moe_norm_workspace_size(nv.make_norm_problem(0, 4096)) == 0
    assert block._lib().moe_norm_workspace_size(np_(), None) == INV


# ----------------------------------------------------------------------- SwiGLU
def sp(**kw):
    dt = kw.pop("dtype", 0)
    p = nv.make_swiglu_problem(**{**dict(M=512, F=1024, groups=160), **kw})
    p.dtype = dt
    return ctypes.byref(p)


def swiglu(p=None, u=at(0), us=2048, off=at(1), a=at(2), as_=1024, c=at(3), s=at(4), k=at(5), ks=at(6)):
    return block._lib().moe_swiglu(p or sp(), u, us, off, a, as_, c, s, k, ks, None)


def swiglu_backward(p=None, u=at(0), us=2048, ks=at(1), off=at(2), da=at(3), das=1024, du=at(4), dus=2048):
    return block._lib().moe_swiglu_backward(p or sp(), u, us, ks, off, da, das, du, dus, None)


@pytest.mark.parametrize("kw,status", [
    (dict(M=-1), INV), (dict(M=(1 << 27) + 1), INV), (dict(F=0), SHAPE), (dict(F=65537), SHAPE), (dict(groups=0), SHAPE),
    (dict(groups=1025), SHAPE), (dict(dtype=3), INV), (dict(dtype=-1), INV),
])
def test_swiglu_problem_refusals(kw, status):
    assert swiglu(sp(**kw)) == status and swiglu_backward(sp(**kw)) == status


def test_swiglu_argument_refusals():
    for kw in (dict(u=None), dict(us=2047), dict(as_=1000), dict(u=at(0, 1)), dict(a=at(2, 1)), dict(c=None), dict(s=None),
               dict(c=at(3, 4)), dict(k=None), dict(ks=None), dict(k=at(5, 8)), dict(off=at(1, 2)), dict(a=at(0)),
               dict(k=at(0, 16)), dict(a=at(1)), dict(c=at(2, 16)), dict(s=at(3, 1)), dict(ks=at(6), k=at(6))):
        assert swiglu(**kw) == INV, kw
    assert swiglu(sp(F=1000)) == SHAPE and well_formed(swiglu(sp(F=1000), c=None, s=None, k=None, ks=None))
    assert well_formed(swiglu()) and well_formed(swiglu(off=None)) and well_formed(swiglu(a=None, c=None, s=None))
    for kw in (dict(u=None), dict(u=at(0, 8)), dict(da=None), dict(du=None), dict(das=1), dict(dus=2047),
               dict(off=at(2, 1)), dict(du=at(0)), dict(du=at(3)), dict(du=at(1)), dict(du=at(2))):
        assert swiglu_backward(**kw) == INV, kw
    assert swiglu_backward(sp(F=1000)) == SHAPE and well_formed(swiglu_backward(sp(F=1000), ks=None, us=2000))
    assert swiglu_backward(ks=None, us=2047) == INV
    assert well_formed(swiglu_backward()) and well_formed(swiglu_backward(us=0)) and well_formed(swiglu_backward(off=None))
    none = {n: None for n in ("u", "off", "a", "c", "s", "k", "ks")}
    assert well_formed(swiglu(sp(M=0), **none))
    assert well_formed(swiglu_backward(sp(M=0), **{n: None for n in ("u", "ks", "off", "da", "du")}))


# ------------------------------------------------------------------------ MXFP8
def quantize(x=at(0), dt=0, R=64, C=4096, xs=4096, c=at(1), s=at(2)):
    return block._lib().moe_mxfp8_quantize(x, dt, R, C, xs, c, s, None)


def dequantize(c=at(0), s=at(1), R=64, C=4096, dt=0, out=at(2), os_=4096):
    return block._lib().moe_mxfp8_dequantize(c, s, R, C, dt, out, os_, None)


def test_mxfp8_refusals():
    for kw, st in ((dict(x=None), INV), (dict(c=None), INV), (dict(s=None), INV), (dict(dt=3), INV), (dict(R=-1), INV),
                   (dict(C=-32), INV), (dict(C=40, xs=40), SHAPE), (dict(R=1 << 36), SHAPE), (dict(xs=4095), INV),
                   (dict(c=at(1, 8)), INV), (dict(x=at(0, 1)), INV), (dict(c=at(0, 32)), INV), (dict(s=at(1, 5)), INV)):
        assert quantize(**kw) == st, kw
    for kw, st in ((dict(c=None), INV), (dict(s=None), INV), (dict(out=None), INV), (dict(dt=-1), INV),
                   (dict(C=100, os_=100), SHAPE), (dict(os_=1), INV), (dict(out=at(0)), INV), (dict(out=at(1)), INV),
                   (dict(c=at(0, 4)), INV)):
        assert dequantize(**kw) == st, kw
    assert well_formed(quantize()) and well_formed(dequantize()) and well_formed(quantize(R=0, x=None, c=None, s=None))


def product(p=None, a=at(0), as_=at(1), w=at(2), ws=at(3), off=at(4), out=at(5), dt=0, os_=2048):
    p = p or nv.make_product_problem(512, 2048, 4096, 160)
    return block._lib().moe_mxfp8_product(ctypes.byref(p), a, as_, w, ws, off, out, dt, os_, None)


def test_product_refusals():
    mk = nv.make_product_problem
    for p, st in ((mk(-1, 8, 32), INV), (mk(8, 0, 32), SHAPE), (mk(8, 65537, 32), SHAPE), (mk(8, 8, 40), SHAPE),
                  (mk(8, 8, 0), SHAPE), (mk(8, 8, 65568), SHAPE), (mk(8, 8, 32, 0), SHAPE), (mk(8, 8, 32, 1025), SHAPE)):
        assert product(p) == st
    for kw in (dict(a=None), dict(as_=None), dict(w=None), dict(ws=None), dict(off=None), dict(out=None), dict(dt=3),
               dict(os_=2047), dict(a=at(0, 8)), dict(w=at(2, 4)), dict(off=at(4, 2)), dict(out=at(5, 1)),
               dict(out=at(0, 64)), dict(out=at(1)), dict(out=at(2)), dict(out=at(3)), dict(out=at(4))):
        assert product(**kw) == INV, kw
    assert well_formed(product()) and well_formed(product(mk(512, 2048, 4096), off=None))
    assert well_formed(product(mk(0, 8, 32), a=None, as_=None, out=None, off=None))


# ---------------------------------------------------------------------- binding
def test_binding_refusals():
    bf, f32 = torch.bfloat16, torch.float32
    e = lambda *s, t=bf: torch.empty(*s, dtype=t)  # noqa: E731
    with pytest.raises(ValueError, match="must be on the GPU"):
        nv.moe_mxfp8_quantize(e(4, 64), e(4, 64, t=torch.uint8), e(4, 2, t=torch.uint8))
    with pytest.raises(ValueError, match="scales: shape"):
        nv.moe_mxfp8_quantize(e(4, 64), e(4, 64, t=torch.uint8), e(4, 3, t=torch.uint8))
    with pytest.raises(ValueError, match="out: dtype"):
        nv.moe_mxfp8_dequantize(e(4, 64, t=torch.uint8), e(4, 2, t=torch.uint8), e(4, 64, t=torch.int32))
    p = nv.make_route_problem(4, 16, 2, dtype=bf)
    ids, w = e(4, 2, t=torch.int32), e(4, 2, t=f32)
    with pytest.raises(ValueError, match="logits: dtype"):
        nv.moe_route(p, e(4, 16, t=f32), None, ids, w)
    with pytest.raises(ValueError, match="bias: shape"):
        nv.moe_route(p, e(4, 16), e(15, t=f32), ids, w)
    with pytest.raises(ValueError, match="ids: dtype"):
        nv.moe_route(p, e(4, 16), None, e(4, 2, t=torch.int64), w)
    with pytest.raises(ValueError, match="contiguous"):
        nv.moe_route(p, e(16, 4).t(), None, ids, w)
    with pytest.raises(ValueError, match="dlogits: shape"):
        nv.moe_route_backward(p, e(4, 16), ids, w, e(4, 17))
    with pytest.raises(ValueError, match="dtype torch.uint8"):
        nv.make_route_problem(4, 16, 2, dtype=torch.uint8)
    p = nv.make_norm_problem(4, 48, dtype=bf, weight_dtype=f32)
    with pytest.raises(ValueError, match="whole blocks of 32"):
        nv.moe_norm(p, e(4, 48), None, e(48, t=f32), None, None, nv.MXFP8Rows(e(4, 48, t=torch.uint8),
                                                                              e(4, 1, t=torch.uint8)), None)
    with pytest.raises(ValueError, match="weight: dtype"):
        nv.moe_norm(p, e(4, 48), None, e(48), None, e(4, 48), None, None)
    with pytest.raises(ValueError, match="residual: shape"):
        nv.moe_norm(p, e(4, 48), e(3, 48), e(48, t=f32), None, e(4, 48), None, None)
    with pytest.raises(ValueError, match="dweight: dtype"):
        nv.moe_norm_backward(p, e(4, 48), e(48, t=f32), e(4, t=f32), e(4, 48), None, e(4, 48), e(48), None)
    p = nv.make_swiglu_problem(4, 48, 2)
    with pytest.raises(ValueError, match="whole blocks of 32"):
        nv.moe_swiglu_backward(p, nv.MXFP8Rows(e(4, 96, t=torch.uint8), e(4, 3, t=torch.uint8)), None, e(4, 48), e(4, 96))
    with pytest.raises(ValueError, match="offsets: shape"):
        nv.moe_swiglu(p, e(4, 96), e(2, t=torch.int32), e(4, 48), None, None)
    p = nv.make_product_problem(4, 8, 64)
    w = nv.MXFP4Weights(e(1, 8, 32, t=torch.uint8), e(1, 8, 2, t=torch.uint8))
    with pytest.raises(ValueError, match="a.codes: shape"):
        nv.moe_mxfp8_product(p, nv.MXFP8Rows(e(4, 32, t=torch.uint8), e(4, 2, t=torch.uint8)), w, None, e(4, 8))

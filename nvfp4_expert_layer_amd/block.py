"""Binding of the operators in include/moe_block.h (route, norm, SwiGLU, MXFP8), on torch
tensors and the current torch stream, under the rules of the operators in ops.py:
argument marshalling only, no fallback, every tensor's dtype, shape, device and layout
checked before its pointer reaches the library.

Rows may be strided (views of wider rows, also of unaligned start); the elements of a row
must be contiguous.  MXFP8 codes and scales are dense.
"""
import ctypes
from dataclasses import dataclass

import torch

from . import _check, lib
from .ops import _DTYPE, _FLOATS, _TORCH, _stream_of, _tensors, _weight_specs, moe_product_problem

ROUTE_SOFTMAX, ROUTE_SIGMOID = 0, 1


class moe_route_problem(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in (
        "num_tokens", "num_experts", "top_k", "scores", "num_groups", "top_groups", "group_keys", "renormalize",
        "dtype")] + [("scale", ctypes.c_float)]


class moe_norm_problem(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("rows", "width", "dtype", "weight_dtype")] + [("eps", ctypes.c_float)]


class moe_swiglu_problem(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("rows", "width", "groups", "dtype")]


_typed = None


def _lib():
    """The shared library with the argument types of this header's entry points set."""
    global _typed
    if _typed is None:
        L = lib()
        P, vp = ctypes.POINTER, ctypes.c_void_p
        i32, i64, sz = ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
        rp, np_, sp, pp = P(moe_route_problem), P(moe_norm_problem), P(moe_swiglu_problem), P(moe_product_problem)
        L.moe_route.argtypes = [rp, vp, i64, vp, vp, vp, vp]
        L.moe_route_backward.argtypes = [rp, vp, i64, vp, vp, vp, i64, vp]
        L.moe_norm.argtypes = [np_, vp, i64, vp, i64, vp, vp, i64, vp, i64, vp, vp, vp, vp]
        L.moe_norm_workspace_size.argtypes = [np_, P(sz)]
        L.moe_norm_backward.argtypes = [np_, vp, i64, vp, vp, vp, i64, vp, i64, vp, i64, vp, vp, sz, vp]
        L.moe_swiglu.argtypes = [sp, vp, i64, vp, vp, i64, vp, vp, vp, vp, vp]
        L.moe_swiglu_backward.argtypes = [sp, vp, i64, vp, vp, vp, i64, vp, i64, vp]
        L.moe_mxfp8_quantize.argtypes = [vp, i32, i64, i32, i64, vp, vp, vp]
        L.moe_mxfp8_dequantize.argtypes = [vp, vp, i64, i32, i32, vp, i64, vp]
        L.moe_mxfp8_product.argtypes = [pp, vp, vp, vp, vp, vp, vp, i32, i64, vp]
        for f in ("route", "route_backward", "norm", "norm_workspace_size", "norm_backward", "swiglu",
                  "swiglu_backward", "mxfp8_quantize", "mxfp8_dequantize", "mxfp8_product"):
            getattr(L, "moe_" + f).restype = ctypes.c_int
        _typed = L
    return _typed


def _code(dtype):
    if dtype not in _FLOATS:
        raise ValueError(f"dtype {dtype}: expected one of {_FLOATS}")
    return _DTYPE[dtype]


# ------------------------------------------------------------------------ MXFP8
@dataclass
class MXFP8Rows:
    """Rows held as MXFP8 (device tensors)."""
    codes: torch.Tensor       # uint8 [M, K]
    scales: torch.Tensor      # uint8 [M, K/32]

    @staticmethod
    def empty(M, K, device="cuda"):
        u8 = dict(dtype=torch.uint8, device=device)
        return MXFP8Rows(torch.empty(M, K, **u8), torch.empty(M, K // 32, **u8))


def _mx8_specs(q, R, C, name):
    """Specs of an MXFP8Rows of R rows of C elements (None: both pointers NULL)."""
    u8 = torch.uint8
    codes, scales = (None, None) if q is None else (q.codes, q.scales)
    return (codes, name + ".codes", u8, (R, C)), (scales, name + ".scales", u8, (R, C // 32))


def _wide(q, width, name):
    """MXFP8 rows hold whole blocks of 32."""
    if q is not None and width % 32:
        raise ValueError(f"{name}: rows of {width} elements are not whole blocks of 32")


def moe_mxfp8_quantize(x, codes, scales, stream=None):
    """x [R, C] (bfloat16, float16 or float32) -> codes uint8 [R, C], scales uint8 [R, C/32].
    Returns (codes, scales)."""
    if x.dim() != 2:
        raise ValueError(f"x: shape {tuple(x.shape)}, expected (R, C)")
    R, C = x.shape
    (px, xs), (pc, ps), dev = _tensors(((x, "x", _FLOATS, (R, C)),),
                                       ((codes, "codes", torch.uint8, (R, C)),
                                        (scales, "scales", torch.uint8, (R, C // 32))))
    _check(_lib().moe_mxfp8_quantize(px, _DTYPE[x.dtype], R, C, xs, pc, ps, _stream_of(stream, dev)))
    return codes, scales


def moe_mxfp8_dequantize(codes, scales, out, stream=None):
    """out [R, C] (bfloat16, float16 or float32) = the values of codes uint8 [R, C] and
    scales uint8 [R, C/32]."""
    if out.dim() != 2:
        raise ValueError(f"out: shape {tuple(out.shape)}, expected (R, C)")
    R, C = out.shape
    (po, os_), (pc, ps), dev = _tensors(((out, "out", _FLOATS, (R, C)),),
                                        ((codes, "codes", torch.uint8, (R, C)),
                                         (scales, "scales", torch.uint8, (R, C // 32))))
    _check(_lib().moe_mxfp8_dequantize(pc, ps, R, C, _DTYPE[out.dtype], po, os_, _stream_of(stream, dev)))
    return out


def moe_mxfp8_product(problem, a, w, offsets, out, stream=None):
    """out[r] = a[r] . w[group of r]^T for the rows of every group (W4A8); other rows of
    out stay as they were.  a: MXFP8Rows [M, K]; w: MXFP4Weights; offsets int32 [G + 1]
    (None: one group of all rows); out [M, N] (bfloat16, float16 or float32).  Its
    gradient is moe_mxfp4_product_backward."""
    p = problem
    (po, os_), (pa, pas, pw, ps, pf), dev = _tensors(
        ((out, "out", _FLOATS, (p.rows, p.n)),), (*_mx8_specs(a, p.rows, p.k, "a"), *_weight_specs(p, w, offsets)))
    _check(_lib().moe_mxfp8_product(ctypes.byref(p), pa, pas, pw, ps, pf, po, _DTYPE[out.dtype], os_,
                                    _stream_of(stream, dev)))
    return out


# ------------------------------------------------------------------------ route
def make_route_problem(T, E, k, scores=ROUTE_SOFTMAX, groups=1, top_groups=1, group_keys=2, renormalize=True, scale=1.0,
                       dtype=torch.float32):
    """T tokens' logits over E experts (rows of a torch dtype), k chosen by ROUTE_SOFTMAX
    or ROUTE_SIGMOID scores out of the top_groups of `groups` groups."""
    return moe_route_problem(T, E, k, scores, groups, top_groups, group_keys, int(bool(renormalize)), _code(dtype),
                             float(scale))


def moe_route(problem, logits, bias, ids, weights, stream=None):
    """logits [T, E], bias float32 [E] (None: none) -> ids int32 [T, k], highest key first
    (-1 where fewer experts have keys), weights float32 [T, k].  Returns (ids, weights)."""
    p = problem
    T, E, k = p.num_tokens, p.num_experts, p.top_k
    (pl, ls), (pb, pi, pw), dev = _tensors(
        ((logits, "logits", (_TORCH[p.dtype],), (T, E)),),
        ((bias, "bias", torch.float32, (E,)), (ids, "ids", torch.int32, (T, k)),
         (weights, "weights", torch.float32, (T, k))))
    _check(_lib().moe_route(ctypes.byref(p), pl, ls, pb, pi, pw, _stream_of(stream, dev)))
    return ids, weights


def moe_route_backward(problem, logits, ids, dweights, dlogits, stream=None):
    """dlogits [T, E] from dweights float32 [T, k], the ids int32 [T, k] held fixed."""
    p = problem
    T, E, k, dt = p.num_tokens, p.num_experts, p.top_k, (_TORCH[p.dtype],)
    (pl, ls, pd, ds), (pi, pw), dev = _tensors(
        ((logits, "logits", dt, (T, E)), (dlogits, "dlogits", dt, (T, E))),
        ((ids, "ids", torch.int32, (T, k)), (dweights, "dweights", torch.float32, (T, k))))
    _check(_lib().moe_route_backward(ctypes.byref(p), pl, ls, pi, pw, pd, ds, _stream_of(stream, dev)))
    return dlogits


# ------------------------------------------------------------------------- norm
def make_norm_problem(T, d, eps=1e-6, dtype=torch.bfloat16, weight_dtype=None):
    """T rows of d elements of a torch dtype; the weight's dtype is the rows' unless given."""
    return moe_norm_problem(T, d, _code(dtype), _code(weight_dtype or dtype), eps)


def moe_norm(problem, x, residual, weight, h, y, q, rstd, stream=None):
    """h = x + residual, y = h * rstd * weight, rstd = 1 / sqrt(mean(h^2) + eps).
    x, residual (None: none), h, y [T, d]; weight [d]; q MXFP8Rows [T, d]: y as MXFP8;
    rstd float32 [T].  h, y, q and rstd may each be None to skip that output.
    Returns (h, y, q, rstd)."""
    p = problem
    T, d, dt = p.rows, p.width, (_TORCH[p.dtype],)
    _wide(q, d, "q")
    (px, xs, pr, rs, ph, hs, py, ys), (pw, pc, ps, pt), dev = _tensors(
        ((x, "x", dt, (T, d)), (residual, "residual", dt, (T, d)), (h, "h", dt, (T, d)), (y, "y", dt, (T, d))),
        ((weight, "weight", _TORCH[p.weight_dtype], (d,)), *_mx8_specs(q, T, d, "q"),
         (rstd, "rstd", torch.float32, (T,))))
    _check(_lib().moe_norm(ctypes.byref(p), px, xs, pr, rs, pw, ph, hs, py, ys, pc, ps, pt, _stream_of(stream, dev)))
    return h, y, q, rstd


def moe_norm_workspace_size(problem):
    n = ctypes.c_size_t(0)
    _check(_lib().moe_norm_workspace_size(ctypes.byref(problem), ctypes.byref(n)))
    return n.value


def alloc_norm_workspace(problem, device="cuda"):
    return torch.empty(moe_norm_workspace_size(problem), dtype=torch.uint8, device=device)


def moe_norm_backward(problem, h, weight, rstd, dy, dh, dx, dweight, workspace=None, stream=None):
    """Gradients of moe_norm from dy [T, d] and dh [T, d] (what else arrives at h; None:
    nothing): dx [T, d], of x and the residual alike, and dweight float32 [d]; either may
    be None.  workspace uint8 (moe_norm_workspace_size bytes; None without dweight).
    Returns (dx, dweight)."""
    p = problem
    T, d, dt = p.rows, p.width, (_TORCH[p.dtype],)
    have = 0 if workspace is None else workspace.numel()
    (ph, hs, py, ys, pg, gs, px, xs), (pw, pt, pd, pk), dev = _tensors(
        ((h, "h", dt, (T, d)), (dy, "dy", dt, (T, d)), (dh, "dh", dt, (T, d)), (dx, "dx", dt, (T, d))),
        ((weight, "weight", _TORCH[p.weight_dtype], (d,)), (rstd, "rstd", torch.float32, (T,)),
         (dweight, "dweight", torch.float32, (d,)), (workspace, "workspace", torch.uint8, (have,))))
    _check(_lib().moe_norm_backward(ctypes.byref(p), ph, hs, pw, pt, py, ys, pg, gs, px, xs, pd, pk, have,
                                    _stream_of(stream, dev)))
    return dx, dweight


# ----------------------------------------------------------------------- SwiGLU
def make_swiglu_problem(M, F, groups=1, dtype=torch.bfloat16):
    """M buffer rows of gate | up, F columns each, sorted into groups."""
    return moe_swiglu_problem(M, F, groups, _code(dtype))


def moe_swiglu(problem, u, offsets, a, q, kept, stream=None):
    """silu(gate) * up of u [M, 2F] (gate first) -> a [M, F] and as MXFP8 q (MXFP8Rows
    [M, F]); kept (MXFP8Rows [M, 2F]): u as MXFP8, for the way back.  a, q and kept may
    each be None.  offsets int32 [groups + 1] (None: all rows): rows from its last entry
    on stay as they were.  Returns (a, q, kept)."""
    p = problem
    M, F, dt = p.rows, p.width, (_TORCH[p.dtype],)
    _wide(q, F, "q")
    _wide(kept, F, "kept")
    (pu, us, pa, as_), (pf, pc, ps, pk, pks), dev = _tensors(
        ((u, "u", dt, (M, 2 * F)), (a, "a", dt, (M, F))),
        ((offsets, "offsets", torch.int32, (p.groups + 1,)), *_mx8_specs(q, M, F, "q"),
         *_mx8_specs(kept, M, 2 * F, "kept")))
    _check(_lib().moe_swiglu(ctypes.byref(p), pu, us, pf, pa, as_, pc, ps, pk, pks, _stream_of(stream, dev)))
    return a, q, kept


def moe_swiglu_backward(problem, u, offsets, da, du, stream=None):
    """du [M, 2F] from da [M, F] and u: the rows [M, 2F] or what moe_swiglu kept of them
    (MXFP8Rows [M, 2F])."""
    p = problem
    M, F, dt = p.rows, p.width, (_TORCH[p.dtype],)
    rows, off = ((da, "da", dt, (M, F)), (du, "du", dt, (M, 2 * F))), (offsets, "offsets", torch.int32, (p.groups + 1,))
    if isinstance(u, MXFP8Rows):
        _wide(u, F, "u")
        (pa, as_, pd, ds), (pf, pu, ps), dev = _tensors(rows, (off, *_mx8_specs(u, M, 2 * F, "u")))
        us = 2 * F
    else:
        (pa, as_, pd, ds, pu, us), (pf,), dev = _tensors((*rows, (u, "u", dt, (M, 2 * F))), (off,))
        ps = None
    _check(_lib().moe_swiglu_backward(ctypes.byref(p), pu, us, ps, pf, pa, as_, pd, ds, _stream_of(stream, dev)))
    return du

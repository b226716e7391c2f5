"""Binding of the operators in include/moe_ops.h (dispatch, combine, MXFP4), on
torch tensors and the current torch stream.  As for the fused layer: argument
marshalling only, no fallback, every tensor's dtype, shape, device and layout
checked before its pointer reaches the library.

Token and expert rows may be strided (views of wider rows, also of unaligned
start); the elements of a row must be contiguous.
"""
import ctypes
from dataclasses import dataclass

import torch

from . import _check, _stream, lib

BF16, F16, F32, U8 = 0, 1, 2, 3
_DTYPE = {torch.bfloat16: BF16, torch.float16: F16, torch.float32: F32, torch.uint8: U8}
_TORCH = {v: k for k, v in _DTYPE.items()}
_FLOATS = (torch.bfloat16, torch.float16, torch.float32)


class moe_dispatch_problem(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in (
        "num_tokens", "top_k", "num_experts", "local_expert_offset", "num_local_experts", "width", "dtype")]


class moe_product_problem(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("rows", "n", "k", "groups")]


_typed = None


def _lib():
    """The shared library with the argument types of this header's entry points set."""
    global _typed
    if _typed is None:
        L = lib()
        P, vp = ctypes.POINTER, ctypes.c_void_p
        i32, i64, sz = ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
        dp, pp = P(moe_dispatch_problem), P(moe_product_problem)
        L.moe_dispatch_workspace_size.argtypes = [dp, P(sz)]
        L.moe_dispatch.argtypes = [dp, vp, vp, i64, vp, vp, vp, vp, vp, i64, vp, sz, vp]
        L.moe_dispatch_backward.argtypes = [dp, vp, vp, i64, vp, i64, vp]
        L.moe_combine.argtypes = [dp, vp, vp, vp, i64, vp, i64, vp]
        L.moe_combine_backward.argtypes = [dp, vp, vp, vp, i64, vp, i64, vp, i64, vp, vp]
        L.moe_mxfp4_quantize.argtypes = [vp, i32, i64, i32, i64, vp, vp, vp]
        L.moe_mxfp4_dequantize.argtypes = [vp, vp, i64, i32, i32, vp, i64, vp]
        L.moe_mxfp4_product.argtypes = [pp, vp, vp, i64, vp, vp, vp, vp, i32, i64, vp]
        L.moe_mxfp4_product_backward.argtypes = [pp, vp, i64, vp, vp, vp, vp, i32, i64, vp]
        for f in ("dispatch_workspace_size", "dispatch", "dispatch_backward", "combine", "combine_backward",
                  "mxfp4_quantize", "mxfp4_dequantize", "mxfp4_product", "mxfp4_product_backward"):
            getattr(L, "moe_" + f).restype = ctypes.c_int
        _typed = L
    return _typed


def _mismatch(t, name, dtypes, shape):
    if t.dtype not in dtypes:
        raise ValueError(f"{name}: dtype {t.dtype}, expected " + " or ".join(str(d) for d in dtypes))
    raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")


def _tensors(rows, dense):
    """Checks the row tensors `rows` (tensor, name, dtypes, shape) and the dense tensors
    `dense` (tensor, name, dtype, shape), dtypes and shapes first; None passes as NULL.
    Returns (pointer, row stride) of each row tensor, flattened, the dense pointers and
    the device.  One pass with few attribute reads: small calls cost what this costs."""
    out, ptrs, device, stray = [], [], None, None
    for t, name, dtypes, shape in rows:
        if t is None:
            out += (None, 0)
            continue
        if t.dtype not in dtypes or t.shape != shape:
            _mismatch(t, name, dtypes, shape)
        many, width = shape[0] > 1, shape[1]
        step, inner = t.stride()
        if inner != 1 and width > 1 and shape[0] > 0:
            raise ValueError(f"{name}: elements of a row must be contiguous (strides {t.stride()})")
        dev = t.get_device()
        if device is None:
            device = dev
        if dev != device or dev < 0:
            stray = stray or (t, name)
        out += (t.data_ptr(), step if many else width)
    for t, name, dtype, shape in dense:
        if t is None:
            ptrs.append(None)
            continue
        if t.dtype is not dtype or t.shape != shape:
            _mismatch(t, name, (dtype,), shape)
        if not t.is_contiguous():
            raise ValueError(f"{name}: tensor must be contiguous")
        dev = t.get_device()
        if device is None:
            device = dev
        if dev != device or dev < 0:
            stray = stray or (t, name)
        ptrs.append(t.data_ptr())
    if stray is not None and not stray[0].is_cuda:
        raise ValueError(f"{stray[1]}: tensor must be on the GPU")
    # the library launches on the current device (and its stream)
    cur = torch._C._cuda_getDevice()
    if stray is not None or device != cur:
        t, name = stray or next((t, n) for t, n, *_ in (*rows, *dense) if t is not None)
        raise ValueError(f"{name}: tensor is on {t.device}, the current device is cuda:{cur}")
    return out, ptrs, cur


def _stream_of(stream, device):
    """The raw handle of `stream`, by default the device's current stream."""
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(device)
    return _stream(stream)


# ------------------------------------------------------------ dispatch, combine
def make_dispatch_problem(T, d, E, k, offset, L, dtype=torch.bfloat16):
    """T tokens of k slots over E experts, of which [offset, offset + L) are local;
    rows of d elements of a torch dtype (bfloat16, float16, float32; uint8 for the
    dispatch alone)."""
    if dtype not in _DTYPE:
        raise ValueError(f"dtype {dtype}: expected one of {tuple(_DTYPE)}")
    return moe_dispatch_problem(T, k, E, offset, L, d, _DTYPE[dtype])


def moe_dispatch_workspace_size(problem):
    n = ctypes.c_size_t(0)
    _check(_lib().moe_dispatch_workspace_size(ctypes.byref(problem), ctypes.byref(n)))
    return n.value


def alloc_dispatch_workspace(problem, device="cuda"):
    return torch.empty(moe_dispatch_workspace_size(problem), dtype=torch.uint8, device=device)


def moe_dispatch(problem, ids, x, counts, offsets, perm, inv, rows, workspace, stream=None):
    """Sorts the pairs of ids int32 [T, k] by local expert and gathers the token rows.
    x [T, d] -> rows [T k, d] (both None: the plan alone); counts int32 [L], offsets
    int32 [L + 1], perm int32 [T k], inv int32 [T, k] (each may be None); workspace
    uint8 (moe_dispatch_workspace_size bytes; may be None where that is 0).  perm and
    rows past the kept pairs stay as they were.  Returns rows."""
    p, i32 = problem, torch.int32
    T, k, L, dt = p.num_tokens, p.top_k, p.num_local_experts, (_TORCH[p.dtype],)
    have = 0 if workspace is None else workspace.numel()
    (px, xs, pr, rs), (pi, pc, po, pp, pv, pw), dev = _tensors(
        ((x, "x", dt, (T, p.width)), (rows, "rows", dt, (T * k, p.width))),
        ((ids, "ids", i32, (T, k)), (counts, "counts", i32, (L,)), (offsets, "offsets", i32, (L + 1,)),
         (perm, "perm", i32, (T * k,)), (inv, "inv", i32, (T, k)),
         (workspace, "workspace", torch.uint8, (have,))))
    _check(_lib().moe_dispatch(ctypes.byref(p), pi, px, xs, pc, po, pp, pv, pr, rs, pw, have,
                               _stream_of(stream, dev)))
    return rows


def moe_dispatch_backward(problem, inv, drows, dx, stream=None):
    """dx [T, d] = the sum of each token's kept rows of drows [T k, d]."""
    p = problem
    T, k, dt = p.num_tokens, p.top_k, (_TORCH[p.dtype],)
    (pr, rs, px, xs), (pv,), dev = _tensors(((drows, "drows", dt, (T * k, p.width)), (dx, "dx", dt, (T, p.width))),
                                       ((inv, "inv", torch.int32, (T, k)),))
    _check(_lib().moe_dispatch_backward(ctypes.byref(p), pv, pr, rs, px, xs, _stream_of(stream, dev)))
    return dx


def moe_combine(problem, inv, weights, rows, out, stream=None):
    """out [T, d] = each token's kept rows [T k, d] times weights fp32 [T, k], summed."""
    p = problem
    T, k, dt = p.num_tokens, p.top_k, (_TORCH[p.dtype],)
    (pr, rs, po, os_), (pv, pw), dev = _tensors(
        ((rows, "rows", dt, (T * k, p.width)), (out, "out", dt, (T, p.width))),
        ((inv, "inv", torch.int32, (T, k)), (weights, "weights", torch.float32, (T, k))))
    _check(_lib().moe_combine(ctypes.byref(p), pv, pw, pr, rs, po, os_, _stream_of(stream, dev)))
    return out


def moe_combine_backward(problem, inv, weights, rows, dout, drows, dweights, stream=None):
    """Gradients of moe_combine from dout [T, d]: drows [T k, d] (rows of no pair stay
    as they were) and dweights fp32 [T, k]; either may be None (rows too, without
    dweights).  Returns (drows, dweights)."""
    p = problem
    T, k, dt = p.num_tokens, p.top_k, (_TORCH[p.dtype],)
    (pr, rs, po, os_, pg, gs), (pv, pw, pd), dev = _tensors(
        ((rows, "rows", dt, (T * k, p.width)), (dout, "dout", dt, (T, p.width)), (drows, "drows", dt, (T * k, p.width))),
        ((inv, "inv", torch.int32, (T, k)), (weights, "weights", torch.float32, (T, k)),
         (dweights, "dweights", torch.float32, (T, k))))
    _check(_lib().moe_combine_backward(ctypes.byref(p), pv, pw, pr, rs, po, os_, pg, gs, pd, _stream_of(stream, dev)))
    return drows, dweights


# ------------------------------------------------------------------------ MXFP4
@dataclass
class MXFP4Rows:
    """Rows held as MXFP4 (device tensors)."""
    codes: torch.Tensor       # uint8 [M, K/2]
    scales: torch.Tensor      # uint8 [M, K/32]

    @staticmethod
    def empty(M, K, device="cuda"):
        u8 = dict(dtype=torch.uint8, device=device)
        return MXFP4Rows(torch.empty(M, K // 2, **u8), torch.empty(M, K // 32, **u8))


@dataclass
class MXFP4Weights:
    """MXFP4 weights of G experts (device tensors)."""
    codes: torch.Tensor       # uint8 [G, N, K/2]
    scales: torch.Tensor      # uint8 [G, N, K/32]

    def slice(self, start, count):
        """Experts [start, start + count) (views)."""
        return MXFP4Weights(self.codes[start:start + count], self.scales[start:start + count])

    @staticmethod
    def empty(G, N, K, device="cuda"):
        u8 = dict(dtype=torch.uint8, device=device)
        return MXFP4Weights(torch.empty(G, N, K // 2, **u8), torch.empty(G, N, K // 32, **u8))


def _mx_specs(codes, scales, *shape, name=""):
    lead, C = shape[:-1], shape[-1]
    return ((codes, name + "codes", torch.uint8, (*lead, C // 2)), (scales, name + "scales", torch.uint8, (*lead, C // 32)))


def moe_mxfp4_quantize(x, codes, scales, stream=None):
    """x [R, C] (bfloat16, float16 or float32) -> codes uint8 [R, C/2], scales uint8 [R, C/32].
    Returns (codes, scales)."""
    if x.dim() != 2:
        raise ValueError(f"x: shape {tuple(x.shape)}, expected (R, C)")
    R, C = x.shape
    (px, xs), (pc, ps), dev = _tensors(((x, "x", _FLOATS, (R, C)),), _mx_specs(codes, scales, R, C))
    _check(_lib().moe_mxfp4_quantize(px, _DTYPE[x.dtype], R, C, xs, pc, ps, _stream_of(stream, dev)))
    return codes, scales


def moe_mxfp4_dequantize(codes, scales, out, stream=None):
    """out [R, C] (bfloat16, float16 or float32) = the values of codes uint8 [R, C/2] and
    scales uint8 [R, C/32]."""
    if out.dim() != 2:
        raise ValueError(f"out: shape {tuple(out.shape)}, expected (R, C)")
    R, C = out.shape
    (po, os_), (pc, ps), dev = _tensors(((out, "out", _FLOATS, (R, C)),), _mx_specs(codes, scales, R, C))
    _check(_lib().moe_mxfp4_dequantize(pc, ps, R, C, _DTYPE[out.dtype], po, os_, _stream_of(stream, dev)))
    return out


def quantize_mxfp4_weights(w, out=None, start=0):
    """Quantizes expert weights w [n, N, K] (bfloat16, float16 or float32, contiguous)
    into `out` (an MXFP4Weights, experts [start, start + n)) on the GPU."""
    n, N, K = w.shape
    if not w.is_contiguous():
        raise ValueError("w must be contiguous")
    if out is None:
        out, start = MXFP4Weights.empty(n, N, K, device=w.device), 0
    part = out.slice(start, n)
    _tensors((), _mx_specs(part.codes, part.scales, n, N, K, name="out."))
    moe_mxfp4_quantize(w.view(n * N, K), part.codes.view(n * N, K // 2), part.scales.view(n * N, K // 32))
    return out


def make_product_problem(M, N, K, groups=1):
    """M buffer rows, weights [groups, N, K]."""
    return moe_product_problem(M, N, K, groups)


def _weight_specs(p, w, offsets):
    return (*_mx_specs(w.codes, w.scales, p.groups, p.n, p.k, name="w."),
            (offsets, "offsets", torch.int32, (p.groups + 1,)))


def moe_mxfp4_product(problem, a, w, offsets, out, stream=None):
    """out[r] = a[r] . w[group of r]^T for the rows of every group; other rows of out
    stay as they were.  a: bfloat16 [M, K] (W4A16) or MXFP4Rows (W4A4); w:
    MXFP4Weights; offsets int32 [G + 1] (None: one group of all rows); out [M, N]
    (bfloat16, float16 or float32)."""
    p = problem
    M, N, K = p.rows, p.n, p.k
    specs, rows = _weight_specs(p, w, offsets), ((out, "out", _FLOATS, (M, N)),)
    if isinstance(a, MXFP4Rows):
        (po, os_), (pa, pas, pw, ps, pf), dev = _tensors(rows, (*_mx_specs(a.codes, a.scales, M, K, name="a."), *specs))
        as_ = K
    else:
        (po, os_, pa, as_), (pw, ps, pf), dev = _tensors((*rows, (a, "a", (torch.bfloat16,), (M, K))), specs)
        pas = None
    _check(_lib().moe_mxfp4_product(ctypes.byref(p), pa, pas, as_, pw, ps, pf, po, _DTYPE[out.dtype], os_,
                                    _stream_of(stream, dev)))
    return out


def moe_mxfp4_product_backward(problem, dout, w, offsets, drows, stream=None):
    """drows[r] = dout[r] . w[group of r] for the rows of every group; other rows stay
    as they were.  dout bfloat16 [M, N]; drows [M, K] (bfloat16, float16 or float32)."""
    p = problem
    (pd, ds, po, os_), (pw, ps, pf), dev = _tensors(
        ((dout, "dout", (torch.bfloat16,), (p.rows, p.n)), (drows, "drows", _FLOATS, (p.rows, p.k))),
        _weight_specs(p, w, offsets))
    _check(_lib().moe_mxfp4_product_backward(ctypes.byref(p), pd, ds, pw, ps, pf, po, _DTYPE[drows.dtype], os_,
                                             _stream_of(stream, dev)))
    return drows

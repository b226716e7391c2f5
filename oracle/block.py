"""What stands round the expert layer's products, in plain numpy fp64 (test infrastructure;
shares nothing with the GPU path): the router's choice and its gradient, the
root-mean-square norm, SwiGLU, and MXFP8.

MXFP8 (the Open Compute Project's microscaling format): a block is 32 elements, its scale
2^(floor(log2 amax) - 8) held as a power-of-two byte (E8M0, bias 127, 255 = NaN), its
elements E4M3, each the nearest of that format's values (ties to the even code, beyond
448 saturating).  Codes are found by searching the value set.
"""
import numpy as np

BLOCK = 32
# E4M3 magnitudes of codes 0 .. 126: exponent field e (bias 7), three fraction bits
E4M3 = np.array([(m / 8 * 2.0 ** -6) if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
                 for e in range(16) for m in range(8)][:127])


def e4m3_codes(q):
    """Nearest E4M3 codes of fp64 q: by search among the midpoints, halves to the even code."""
    a = np.abs(q)
    mid = (E4M3[1:] + E4M3[:-1]) / 2
    lo = np.searchsorted(mid, a, side="left")            # midpoints below a
    hi = np.searchsorted(mid, a, side="right")           # ... and those it equals
    code = np.where(lo % 2 == 0, lo, hi)                 # on a midpoint lo and hi = lo + 1 are as near
    return (np.minimum(code, 126) | (np.signbit(q) * 128)).astype(np.uint8)


def mxfp8_quantize(x):
    """x [R, C] -> codes uint8 [R, C], scales uint8 [R, C/32]."""
    x = np.asarray(x, dtype=np.float64)
    R, C = x.shape
    b = x.reshape(R, C // BLOCK, BLOCK)
    bad = ~np.isfinite(b).all(axis=2)
    b = np.where(bad[:, :, None], 0.0, b)
    amax = np.abs(b).max(axis=2)
    e = np.where(amax > 0, np.frexp(amax)[1] - 1 - 8, -127).clip(-127, 127)
    codes = e4m3_codes(np.ldexp(b, -e[:, :, None]))
    codes = np.where(bad[:, :, None], 0, codes).astype(np.uint8).reshape(R, C)
    return codes, np.where(bad, 255, e + 127).astype(np.uint8)


def mxfp8_dequantize(codes, scales):
    """fp64 values of codes [..., C] and scales [..., C/32] (NaN where a scale is 255; codes 127
    and 255 are NaN)."""
    codes, scales = np.asarray(codes), np.asarray(scales)
    v = np.where(codes & 128, -1.0, 1.0) * np.append(E4M3, np.nan)[codes & 127]
    s = np.where(scales == 255, np.nan, np.ldexp(1.0, scales.astype(int) - 127))
    return v * np.repeat(s, BLOCK, axis=-1)


def sigmoid(x):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-np.asarray(x, dtype=np.float64)))


def _sane(logits):
    """NaN counts as -Inf, +Inf as the largest finite fp32."""
    l = np.asarray(logits, dtype=np.float64)
    return np.where(np.isnan(l), -np.inf, np.minimum(l, float(np.finfo(np.float32).max)))


def scores(logits, kind):
    l = _sane(logits)
    if kind == "sigmoid":
        return sigmoid(l)
    top = l.max()
    if top == -np.inf:
        return np.zeros_like(l)
    e = np.exp(l - top)
    return e / e.sum()


def route_token(logits, k, kind="softmax", bias=None, groups=1, top_groups=1, group_keys=2, renormalize=True, scale=1.0):
    """One token: (ids int [k], -1 where fewer have keys; weights fp64 [k]; keys fp64 [E])."""
    l = _sane(logits)
    s = scores(logits, kind)
    E = len(l)
    if bias is None and top_groups == groups:
        key = l.copy()                                   # the logits' own order
    else:
        key = s + (0.0 if bias is None else np.asarray(bias, dtype=np.float64))
    key = np.where((l == -np.inf) | np.isnan(key), -np.inf, key)
    allowed = np.ones(E, dtype=bool)
    if top_groups < groups:
        n = E // groups
        own = []
        for g in range(groups):
            best = sorted((v for v in key[g * n:(g + 1) * n] if v > -np.inf), reverse=True)[:group_keys]
            own.append(sum(best) if best else -np.inf)
        first = sorted(range(groups), key=lambda g: (-own[g], g))[:top_groups]
        allowed = np.isin(np.arange(E) // n, first)
    order = sorted((e for e in range(E) if allowed[e] and key[e] > -np.inf), key=lambda e: (-key[e], e))[:k]
    ids = np.full(k, -1)
    ids[:len(order)] = order
    w = np.zeros(k)
    w[:len(order)] = s[order]
    if renormalize:
        if kind == "softmax" and order:                  # the sum over all experts cancels
            w[:len(order)] = np.exp(l[order] - l[order].max())
        w = w / w.sum() if w.sum() > 0 else np.zeros(k)
    return ids, scale * w, key


def route_gradient(logits, ids, dweights, kind="softmax", renormalize=True, scale=1.0):
    """dlogits [E] of one token's weights, by the chain rule through the scores' Jacobian."""
    l = _sane(logits)
    E = len(l)
    at = [(e, float(g) * scale) for e, g in zip(ids, dweights) if 0 <= e < E]
    if not at:
        return np.zeros(E)
    idx, g = np.array([a[0] for a in at]), np.array([a[1] for a in at])
    if kind == "softmax" and renormalize:                # a softmax over the chosen ones
        z = np.exp(l[idx] - l[idx].max()) if l[idx].max() > -np.inf else np.zeros(len(idx))
        p = z / z.sum() if z.sum() > 0 else z
        out = np.zeros(E)
        np.add.at(out, idx, p * (g - (p * g).sum()))
        return out
    s = scores(logits, kind)
    if renormalize:
        total = s[idx].sum()
        if total == 0:
            return np.zeros(E)
        p = s[idx] / total
        # p (1 - s) (g - sum): the score cancels against the total, which may be tiny
        out = np.zeros(E)
        np.add.at(out, idx, p * sigmoid(-l[idx]) * (g - (p * g).sum()))
        return out
    ds = np.zeros(E)
    np.add.at(ds, idx, g)
    if kind == "sigmoid":
        return ds * s * sigmoid(-l)
    return s * (ds - (s * ds).sum())


def norm(h, weight, eps):
    """(y, rstd) of fp64 rows h [T, d]."""
    r = 1.0 / np.sqrt((h * h).mean(axis=1) + eps)
    return h * r[:, None] * weight, r


def norm_gradient(h, weight, rstd, dy, dh=None):
    """(dx, dweight)."""
    n = h * rstd[:, None]
    g = dy * weight
    dx = rstd[:, None] * (g - n * (g * n).mean(axis=1)[:, None])
    return (dx if dh is None else dx + dh), (dy * n).sum(axis=0)


def swiglu(u):
    """a [M, F] of fp64 rows gate | up [M, 2F]."""
    F = u.shape[1] // 2
    return u[:, :F] * sigmoid(u[:, :F]) * u[:, F:]


def swiglu_gradient(u, da):
    """du [M, 2F]."""
    F = u.shape[1] // 2
    g, up = u[:, :F], u[:, F:]
    s = sigmoid(g)
    return np.concatenate([da * up * s * (1.0 + g * sigmoid(-g)), da * g * s], axis=1)

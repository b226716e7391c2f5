"""Dispatch, combine and the grouped product in plain numpy fp64 (test
infrastructure; shares nothing with the GPU path)."""
import numpy as np


def plan(ids, offset, L):
    """counts [L], offsets [L+1], perm [P], inv [T, k] of the pairs (t, j) whose expert lies
    in [offset, offset + L), sorted by (expert, t, j)."""
    ids = np.asarray(ids, dtype=np.int64)
    T, k = ids.shape
    kept = [(int(ids[t, j]) - offset, t * k + j) for t in range(T) for j in range(k)
            if offset <= ids[t, j] < offset + L]
    kept.sort()
    counts = np.zeros(L, dtype=np.int64)
    for e, _ in kept:
        counts[e] += 1
    perm = np.array([p for _, p in kept], dtype=np.int64)
    inv = np.full(T * k, -1, dtype=np.int64)
    inv[perm] = np.arange(len(perm))
    return counts, np.concatenate([[0], np.cumsum(counts)]), perm, inv.reshape(T, k)


def combine(inv, weights, rows):
    """(sum over slots of weight * row, the same sum of magnitudes); weights None: ones."""
    T, k = inv.shape
    out, mag = np.zeros((T, rows.shape[1])), np.zeros((T, rows.shape[1]))
    for t in range(T):
        for j in range(k):
            if inv[t, j] >= 0:
                term = (1.0 if weights is None else weights[t, j]) * rows[inv[t, j]]
                out[t] += term
                mag[t] += np.abs(term)
    return out, mag


def combine_backward(inv, weights, rows, dout):
    """(drows [T k, d] with NaN where no pair's row lies, dweights, dweights' sum of magnitudes)."""
    T, k = inv.shape
    drows = np.full((T * k, dout.shape[1]), np.nan)
    dw, mag = np.zeros((T, k)), np.zeros((T, k))
    for t in range(T):
        for j in range(k):
            r = inv[t, j]
            if r >= 0:
                drows[r] = weights[t, j] * dout[t]
                dw[t, j] = np.dot(dout[t], rows[r])
                mag[t, j] = np.dot(np.abs(dout[t]), np.abs(rows[r]))
    return drows, dw, mag


def product(a, w, offsets, backward=False):
    """(rows of each group times its weight, the same of magnitudes); NaN in rows of no group.
    w fp64 [G, N, K]; backward: a [M, N] -> [M, K]."""
    M = a.shape[0]
    out = np.full((M, w.shape[2] if backward else w.shape[1]), np.nan)
    mag = out.copy()
    for g in range(w.shape[0]):
        s = slice(int(offsets[g]), int(offsets[g + 1]))
        m = w[g] if backward else w[g].T
        out[s] = a[s] @ m
        mag[s] = np.abs(a[s]) @ np.abs(m)
    return out, mag

"""Plain 64-bit implementations of the FP8 and balance-loss operators, on the CPU, and the
error bounds that the GPU tests hold the kernels to."""
from __future__ import annotations

import numpy as np
import torch

BLK, TOP = 128, 448.0
U32 = 2.0 ** -24          # half a step of binary32, relative
U16 = 2.0 ** -8           # of bf16


def e4m3_values():
    """The 256 E4M3FN values from the format (bias 7, no infinities, 0x7f / 0xff NaN)."""
    v = np.empty(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        x = m * 2.0 ** -9 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        v[c] = np.nan if c & 127 == 127 else (-x if c & 128 else x)
    return v


_V = e4m3_values()
_POS = _V[:127]           # codes 0 .. 126: ascending


def e4m3_codes(u):
    """Codes of u (binary64, |u| <= 448), nearest, ties to the even code, the sign kept."""
    a = np.abs(u)
    hi = np.clip(np.searchsorted(_POS, a), 1, 126)
    lo = hi - 1
    dl, dh = a - _POS[lo], _POS[hi] - a
    c = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    return (c | np.where(np.signbit(u), 128, 0)).astype(np.uint8)


def values(codes):
    return _V[np.asarray(codes)]


def block(x):
    """(codes, scale) of one block x (any shape, binary32 values): every step one correctly
    rounded binary32 operation."""
    x = np.asarray(x, np.float32)
    if not np.isfinite(x).all():
        return np.where(np.signbit(x), 128, 0).astype(np.uint8), np.float32(np.nan)
    s = np.float32(np.abs(x).max(initial=0)) / np.float32(TOP)
    with np.errstate(over="ignore"):
        u = x / s if s > 0 else np.copysign(np.float32(0), x)
    return e4m3_codes(np.clip(u.astype(np.float64), -TOP, TOP)), np.float32(s)


def quantize_rows(x):
    x = np.asarray(x, np.float32)
    n = -(-x.shape[1] // BLK)
    q, s = np.empty(x.shape, np.uint8), np.empty((x.shape[0], n), np.float32)
    for r in range(x.shape[0]):
        for b in range(n):
            q[r, b * BLK:(b + 1) * BLK], s[r, b] = block(x[r, b * BLK:(b + 1) * BLK])
    return q, s


def quantize_weights(w):
    w = np.asarray(w, np.float32)
    E, N, K = w.shape
    q, s = np.empty(w.shape, np.uint8), np.empty((E, -(-N // BLK), -(-K // BLK)), np.float32)
    for e in range(E):
        for i in range(s.shape[1]):
            for j in range(s.shape[2]):
                at = (e, slice(i * BLK, (i + 1) * BLK), slice(j * BLK, (j + 1) * BLK))
                q[at], s[e, i, j] = block(w[at])
    return q, s


def quantize_tokens(x, off, rows=None):
    """Codes [blocks, C, 128] and scales [blocks, C] of the used blocks."""
    x = np.asarray(x, np.float32)
    q, s = [], []
    for lo, hi in zip(off[:-1], off[1:]):
        for p in range(lo, hi, BLK):
            at = np.arange(p, min(p + BLK, hi))
            v = np.zeros((BLK, x.shape[1]), np.float32)
            v[:len(at)] = x[at if rows is None else rows[at]]
            cols = [block(v[:, c]) for c in range(v.shape[1])]
            q.append(np.stack([c for c, _ in cols]))
            s.append(np.array([t for _, t in cols], np.float32))
    C = x.shape[1]
    return (np.stack(q), np.stack(s)) if q else (np.empty((0, C, BLK), np.uint8), np.empty((0, C), np.float32))


def rows_value(q, s):
    return values(q) * np.repeat(np.asarray(s, np.float64), BLK, 1)[:, :q.shape[1]]


def weights_value(q, s):
    s = np.repeat(np.repeat(np.asarray(s, np.float64), BLK, 1)[:, :q.shape[1]], BLK, 2)[:, :, :q.shape[2]]
    return values(q) * s


def sum_error(K):
    """Relative to sum |a b|: a block's 128 products are added in binary32 in an order of the
    matrix core's choosing, perhaps cut off rather than rounded (a whole step each), the
    scales' product is rounded once, the blocks' sums are added by one fma each."""
    return (2 * BLK + 2 + -(-K // BLK)) * U32


def core_error(K):
    """The same for the FP8 matrix core: it adds the products of 8 consecutive elements after
    aligning them to the largest one's exponent and cutting each off at 2^-13 of that power of
    two, so 7 of 8 products lose less than 2^-13 of a value that the sum of the 8 magnitudes
    exceeds (the largest, 8 bits long, loses nothing)."""
    return 7 * 2.0 ** -13 + sum_error(K)


def product(a, w, off, rows=None):
    """(y, sum |a w|) of values a [rows_A, K], w [E, N, K] over the groups, binary64."""
    R, N = int(off[-1]), w.shape[1]
    y, m = np.zeros((R, N)), np.zeros((R, N))
    for e, (lo, hi) in enumerate(zip(off[:-1], off[1:])):
        g = a[np.arange(lo, hi) if rows is None else rows[lo:hi]]
        y[lo:hi], m[lo:hi] = g @ w[e].T, np.abs(g) @ np.abs(w[e]).T
    return y, m


def tokens_value(q, s):
    return values(q) * np.asarray(s, np.float64)[:, :, None]


def wgrad(yv, xv, off):
    """(dW, sum |dy x|) from token-block values yv [blocks, N, 128], xv [blocks, K, 128]."""
    E = len(off) - 1
    d = np.zeros((E, yv.shape[1], xv.shape[1]))
    m = np.zeros_like(d)
    b = 0
    for e in range(E):
        for _ in range(-(-(off[e + 1] - off[e]) // BLK)):
            d[e] += yv[b] @ xv[b].T
            m[e] += np.abs(yv[b]) @ np.abs(xv[b]).T
            b += 1
    return d, m


def swiglu(y):
    g, u = np.split(y, 2, axis=1)
    with np.errstate(over="ignore"):
        return g / (1 + np.exp(-g)) * u


# ---- balance loss ---------------------------------------------------------------------------

def softmax(z):
    with np.errstate(invalid="ignore"):
        m = z.max(1, keepdims=True)
        p = np.exp(z - np.where(m == -np.inf, 0, m))
    s = p.sum(1, keepdims=True)
    return np.divide(p, s, out=np.zeros_like(p), where=s != 0)


def balance(logits, ids, off, mask=None):
    """loss, counts [S, E], coef [S, E], p [T, E] in binary64."""
    z = np.asarray(logits, np.float64)
    T, E = z.shape
    k, S = ids.shape[1], len(off) - 1
    keep = np.ones(T, bool) if mask is None else np.asarray(mask) != 0
    p = np.zeros((T, E))
    p[keep] = softmax(z[keep])
    counts, coef, loss = np.zeros((S, E), np.int64), np.zeros((S, E)), 0.0
    for s in range(S):
        rows = [t for t in range(off[s], off[s + 1]) if keep[t]]
        for t in rows:
            for e in ids[t]:
                if 0 <= e < E:
                    counts[s, e] += 1
        if rows:
            coef[s] = E * counts[s] / (k * len(rows) ** 2 * S)
            loss += (coef[s] * p[rows].sum(0)).sum()
    return loss, counts, coef, p


def balance_grad(p, off, coef, grad, mask=None, ids=None, w=None, dw=None):
    """(dlogits, magnitude of what was added up) for rows inside a sequence; NaN elsewhere."""
    T, E = p.shape
    d, m = np.full((T, E), np.nan), np.zeros((T, E))
    for s in range(len(off) - 1):
        a = grad * coef[s]
        for t in range(off[s], off[s + 1]):
            if mask is not None and not mask[t]:
                d[t] = 0
                continue
            dot = (p[t] * a).sum()
            d[t] = p[t] * (a - dot)
            m[t] = p[t] * (np.abs(a) + np.abs(p[t] * a).sum())
            if dw is not None:
                wd = np.float64(w[t]) * dw[t]
                v = np.float64(w[t]) * (dw[t] - wd.sum())
                mag = np.abs(w[t]) * (np.abs(dw[t]) + np.abs(wd).sum())
                for j, e in enumerate(ids[t]):
                    if 0 <= e < E:
                        d[t, e] += v[j]
                        m[t, e] += mag[j]
    return d, m


def softmax_error(logits, mask=None):
    """Relative error of a binary32 softmax: the exponent's argument (x - max) log2(e) is rounded
    three times (difference, constant, product), exp2 is off by a step, the sum of up to 1024
    terms is taken over 16 terms a lane and 6 levels, then a reciprocal and a product."""
    z = np.asarray(logits, np.float64)
    z = z if mask is None else z[np.asarray(mask) != 0]
    z = np.where(np.isfinite(z), z, np.nan)
    with np.errstate(all="ignore"):
        span = np.nan_to_num(np.nanmax(z, 1) - np.nanmin(z, 1)).max(initial=0) if z.size else 0.0
    return (2 * 3 * span + 2 * 2 + 2 * (16 + 6) + 4) * U32


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()

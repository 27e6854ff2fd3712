"""64-bit references of the bf16 expert products, their epilogues and gradients, and of products with
NVFP4 weights, in torch (any device), with the bounds that the tests hold the kernels to."""
import torch

U32, U16 = 2.0 ** -24, 2.0 ** -8    # half a step of binary32 and of bf16, relative
E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def groups(off):
    b = [int(v) for v in off]
    return list(zip(range(len(b) - 1), b, b[1:]))


def product(a, w, off, rows=None):
    """(y, sum |a w|) [R, N] of a [rows_A, K], w [E, N, K] in binary64; zeros behind the last group."""
    R = int(off[-1])
    y = torch.zeros(R, w.shape[1], dtype=torch.double, device=a.device)
    m = torch.zeros_like(y)
    for e, lo, hi in groups(off):
        if hi > lo:
            v = (a[lo:hi] if rows is None else a[rows[lo:hi].long()]).double()
            b = w[e].double()
            y[lo:hi], m[lo:hi] = v @ b.T, v.abs() @ b.abs().T
    return y, m


def wgrad(dy, x, off, rows=None):
    """(dW, sum |dy x|) [E, N, K]."""
    E = len(off) - 1
    d = torch.zeros(E, dy.shape[1], x.shape[1], dtype=torch.double, device=x.device)
    m = torch.zeros_like(d)
    for e, lo, hi in groups(off):
        if hi > lo:
            v = (x[lo:hi] if rows is None else x[rows[lo:hi].long()]).double()
            g = dy[lo:hi].double()
            d[e], m[e] = g.T @ v, g.abs().T @ v.abs()
    return d, m


def sum_error(n):
    """Relative to sum |a b|, for n products added in binary32 in any order, each sum perhaps cut off
    rather than rounded (a whole step)."""
    return 2 * (n + 2) * U32


def swiglu(y):
    g, u = y.chunk(2, 1)
    return g * torch.sigmoid(g) * u


def swiglu_error(y):
    """Of silu(g) u in binary32: the exponent's argument g log2(e) is rounded (|g| steps of the result),
    hardware exp2 and reciprocal are good to a step each, two products and a sum are rounded."""
    g, _ = y.chunk(2, 1)
    return (8 + 2 * g.abs()) * 2 * U32 * swiglu(y).abs()


def swiglu_backward(da, z):
    """(dz, bound of its binary32 error) from the activations' gradient and the pre-activations."""
    g, u = z.chunk(2, 1)
    s = torch.sigmoid(g)
    dz = torch.cat([da * u * s * (1 + g * (1 - s)), da * g * s], 1)
    # s as above; in 1 + g (1 - s) the terms may cancel, so its error goes by their magnitudes
    mag = torch.cat([(da * u).abs() * s * (1 + g.abs()), (da * g).abs() * s], 1)
    return dz, (12 + 4 * g.abs()).repeat(1, 2) * 2 * U32 * mag


def bf16(v):
    """v (binary64) rounded to bf16 once: nearest, ties to even."""
    e = ((v.view(torch.int64) >> 52) & 0x7ff).clamp(min=1023 - 126)   # of the value, at least bf16's least normal one
    step = ((e - 7) << 52).view(torch.double)
    return torch.round(v / step) * step


def close(got, want, err):
    """|got - want| is within `err` and the rounding of got to bf16."""
    d = (got.double() - want).abs()
    return bool((d <= U16 * want.abs() + (1 + U16) * err + 1e-37).all())


def nvfp4_values(q, sf, gs):
    """Values [E, N, K] in binary64 of codes [E, N, K/2], E4M3 scales [E, N, K/16] and gs [E]."""
    table = torch.tensor(E2M1 + [-v for v in E2M1], dtype=torch.double, device=q.device)
    v = torch.stack([table[(q & 15).long()], table[(q >> 4).long()]], -1).flatten(-2)
    return v * sf.view(torch.float8_e4m3fn).double().repeat_interleave(16, -1) * gs.double()[:, None, None]


def gemv(x, w, ids):
    """(y, sum |x w|) [T * k, N] of x [T or T * k, K], w [E, N, K], ids [T, k]; zeros in dropped slots."""
    T, k = ids.shape
    at = torch.arange(T * k, device=x.device)
    rows = x.double()[at if x.shape[0] == T * k else at // k]
    y = torch.zeros(T * k, w.shape[1], dtype=torch.double, device=x.device)
    m = torch.zeros_like(y)
    flat = ids.flatten()
    for e in sorted({int(v) for v in flat if 0 <= int(v) < w.shape[0]}):
        p = (flat == e).nonzero().flatten()
        y[p], m[p] = rows[p] @ w[e].T, rows[p].abs() @ w[e].abs().T
    return y, m

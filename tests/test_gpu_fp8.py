"""FP8 quantisers, grouped product and weight gradient on the GPU against plain 64-bit
implementations: quantisers bit for bit, products within bounds that count their roundings."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import block_scaled_fp4_02_amd as moe
from tests import fp8_ref as ref
from tests.fp8_ref import U16, U32, dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    moe.lib()
    yield
    torch.cuda.synchronize()


def _x(rng, shape, bf16=True, special=True):
    """Values over a wide range with zeros, tiny and huge blocks, and one NaN and one infinity."""
    x = (rng.standard_normal(shape) * 2.0 ** rng.integers(-6, 7, shape)).astype(np.float32)
    x[rng.random(shape) < 0.05] = 0
    if special and x.size >= 4096:
        f = x.reshape(-1)
        f[:256] = 0                      # whole blocks of zeros
        f[1] = -0.0
        f[256:400] *= 2.0 ** -130        # scales near and below the smallest normal number
        f[512:768] *= 2.0 ** 115
        f[900], f[1500] = np.nan, -np.inf
    t = torch.from_numpy(x)
    return t.to(torch.bfloat16) if bf16 else t


def _bits(t):
    """Bytes of u8 codes, bits of f32 with every NaN the same."""
    if t.dtype == torch.uint8:
        return t.cpu().numpy()
    a = t.cpu().numpy()
    return np.where(np.isnan(a), np.float32(np.nan), a).view(np.uint32)


def _same(got, want, what):
    w = np.where(np.isnan(want), np.float32(np.nan), want).view(np.uint32) if want.dtype == np.float32 else want
    assert np.array_equal(_bits(got), w), (what, int((_bits(got) != w).sum()))


# codes of non-finite blocks carry no value (their scale is NaN)
def _same_codes(got, want, scale_is_nan, what):
    g = got.cpu().numpy()
    assert np.array_equal(g[~scale_is_nan], want[~scale_is_nan]), what


@pytest.mark.parametrize("rows, C, bf16", [(1, 16, True), (1, 128, False), (3, 144, True), (37, 2064, True), (64, 6144, True),
                                           (37, 2064, False), (5, 112, False), (513, 1040, True)])
def test_quantize_rows(rows, C, bf16):
    x = _x(np.random.default_rng(rows * C), (rows, C), bf16)
    got = moe.quantize_fp8_alloc(x.cuda())
    q, s = ref.quantize_rows(x.float().numpy())
    _same(got.sf, s, "scales")
    nan = np.repeat(np.isnan(s), 128, 1)[:, :C]
    _same_codes(got.q, q, nan, "codes")
    again = moe.quantize_fp8_alloc(x.cuda())
    assert torch.equal(got.q, again.q)


def test_quantize_rows_none():
    got = moe.quantize_fp8_alloc(torch.empty(0, 64, dtype=torch.bfloat16, device="cuda"))
    assert got.q.shape == (0, 64) and got.sf.shape == (0, 1)


@pytest.mark.parametrize("E, N, K, bf16", [(1, 16, 16, True), (2, 128, 256, False), (3, 144, 1040, True), (2, 272, 112, False)])
@pytest.mark.parametrize("transposed", [False, True])
def test_quantize_weights(E, N, K, bf16, transposed):
    w = _x(np.random.default_rng(E * N * K), (E, N, K), bf16)
    got = moe.quantize_fp8_weights_alloc(w.cuda(), transposed)
    q, s = ref.quantize_weights(w.float().numpy())
    nan = np.repeat(np.repeat(np.isnan(s), 128, 1)[:, :N], 128, 2)[:, :, :K]
    if transposed:
        got, t = got
        _same(t.sf, s.transpose(0, 2, 1).copy(), "transposed scales")
        _same_codes(t.q, q.transpose(0, 2, 1), nan.transpose(0, 2, 1), "transposed codes")
    _same(got.sf, s, "scales")
    _same_codes(got.q, q, nan, "codes")


@pytest.mark.parametrize("sizes, C, gather, bf16", [
    ([1], 16, False, True), ([0, 128, 0, 129], 144, True, True), ([5, 300, 0, 1, 127], 400, True, True), ([64] * 40, 48, False, False),
    ([0, 0], 32, False, True), ([1, 0, 2] * 100, 32, True, True)])
def test_quantize_tokens(sizes, C, gather, bf16):
    rng = np.random.default_rng(sum(sizes) + C)
    off = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
    R = int(off[-1])
    rows_x = max(1, R // 2) if gather else R + 3
    x = _x(rng, (rows_x, C), bf16)
    rows = rng.integers(0, rows_x, max(R, 1)).astype(np.int32) if gather else None
    blocks = moe.moe_fp8_token_blocks(R, len(sizes))
    q = torch.full((blocks + 1, C, 128), 0x5A, dtype=torch.uint8, device="cuda")
    sf = torch.full((blocks + 1, C), -3.0, device="cuda")
    moe.moe_quantize_fp8_tokens(x.cuda(), dev(off), R, q, sf, None if rows is None else dev(rows))
    wq, ws = ref.quantize_tokens(x.float().numpy(), off, rows)
    n = len(wq)
    _same(sf[:n], ws, "scales")
    _same_codes(q[:n], wq, np.repeat(np.isnan(ws)[:, :, None], 128, 2), "codes")
    assert (q[n:] == 0x5A).all() and (sf[n:] == -3.0).all()   # blocks that no group has stay as they were
    for b, (lo, hi) in _blocks(off):                          # rows behind a group are zero codes
        assert (q[b, :, hi - lo:] == 0).all()


def _blocks(off):
    b = 0
    for lo, hi in zip(off[:-1], off[1:]):
        for p in range(lo, hi, 128):
            yield b, (p, min(p + 128, hi))
            b += 1


# ---- products -------------------------------------------------------------------------------

GROUPS = {
    "one row": [1], "one group": [200], "empty ones": [0, 5, 0, 0, 33, 0], "all empty": [0, 0, 0],
    "decode": [32, 17, 40, 8, 64, 0, 31, 1], "many": [1, 0, 2, 3] * 80, "long": [700, 0, 3, 513],
}


def _operands(rng, sizes, N, K, gather, extra=0):
    off = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
    R = int(off[-1])
    rows_A = max(1, R // 3 + 1) if gather else R + extra
    rows = rng.integers(0, rows_A, R).astype(np.int32) if gather else None
    a = moe.quantize_fp8_alloc((torch.from_numpy(rng.standard_normal((max(rows_A, 1), K)).astype(np.float32))).to(torch.bfloat16).cuda())
    w = moe.quantize_fp8_weights_alloc((0.05 * torch.from_numpy(rng.standard_normal((len(sizes), N, K)).astype(np.float32))).cuda())
    return off, R, rows, a, w


def _near(got, want, bound, what):
    err = np.abs(got.astype(np.float64) - want)
    bad = ~(err <= bound)
    assert not bad.any(), (what, int(bad.sum()), float((err / np.maximum(bound, 1e-300)).max()))


@pytest.mark.parametrize("groups", GROUPS)
@pytest.mark.parametrize("N, K, gather", [(16, 16, False), (144, 2064, True), (512, 512, True), (272, 128, False)])
def test_product(groups, N, K, gather):
    rng = np.random.default_rng(len(groups) * N + K)
    off, R, rows, a, w = _operands(rng, GROUPS[groups], N, K, gather)
    D = torch.full((R + 2, N), 7.0, dtype=torch.bfloat16, device="cuda")
    moe.moe_grouped_gemm_fp8(moe.make_gemm_fp8_args(a.q, a.sf, w.q, w.sf, dev(off), R, moe.MOE_EPI_NONE, D,
                                                    A_rows=None if rows is None or R == 0 else dev(rows)))
    av, wv = ref.rows_value(a.q.cpu().numpy(), a.sf.cpu().numpy()), ref.weights_value(w.q.cpu().numpy(), w.sf.cpu().numpy())
    y, mag = ref.product(av, wv, off, rows)
    _near(D[:R].float().cpu().numpy(), y, U16 * np.abs(y) + (1 + U16) * ref.core_error(K) * mag, groups)
    assert (D[R:] == 7.0).all()


def test_product_rows_behind_the_last_group_stay():
    rng = np.random.default_rng(5)
    off, R, _, a, w = _operands(rng, [40, 3], 64, 256, False, extra=10)
    D = torch.full((R + 10, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    moe.moe_grouped_gemm_fp8(moe.make_gemm_fp8_args(a.q, a.sf, w.q, w.sf, dev(off), R + 10, moe.MOE_EPI_NONE, D))
    assert (D[R:] == 7.0).all() and not (D[:R] == 7.0).all(1).any()


def test_product_exact_integers():
    """Small whole numbers under power-of-two scales: every product and sum is exact."""
    rng = np.random.default_rng(6)
    N, K, sizes = 160, 1008, [33, 0, 130]
    off = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
    R = int(off[-1])
    codes = {v: int(ref.e4m3_codes(np.float64(v))) for v in range(-3, 4)}
    pick = lambda *s: rng.integers(-3, 4, s)
    enc = np.vectorize(codes.get, otypes=[np.uint8])
    av, wv = pick(R, K), pick(3, N, K)
    asf = 2.0 ** rng.integers(-1, 2, (R, 8)).astype(np.float32)
    wsf = 2.0 ** rng.integers(-1, 2, (3, 2, 8)).astype(np.float32)
    D = torch.empty(R, N, dtype=torch.bfloat16, device="cuda")
    moe.moe_grouped_gemm_fp8(moe.make_gemm_fp8_args(dev(enc(av)), dev(asf), dev(enc(wv)), dev(wsf), dev(off), R, moe.MOE_EPI_NONE, D))
    y, _ = ref.product(ref.rows_value(enc(av), asf), ref.weights_value(enc(wv), wsf), off)
    assert torch.equal(D.cpu(), torch.from_numpy(y).to(torch.bfloat16))


def test_product_carries_nan_to_its_own_row_and_columns_only():
    rng = np.random.default_rng(7)
    off, R, _, a, w = _operands(rng, [70, 50], 256, 384, False)
    a.sf[3, 1] = float("nan")
    w.sf[1, 1, 2] = float("nan")
    a.q[5, 0] = 0x7F                 # a NaN code
    D = moe.grouped_gemm_fp8_alloc(a, w, dev(off), R)
    nan = torch.isnan(D).cpu().numpy()
    want = np.zeros((R, 256), bool)
    want[[3, 5]] = True
    want[70:, 128:] = True
    assert np.array_equal(nan, want)


@pytest.mark.parametrize("groups", GROUPS)
@pytest.mark.parametrize("I, K, gather", [(128, 144, True), (384, 1024, False)])
def test_swiglu_quantized(groups, I, K, gather):
    rng = np.random.default_rng(len(groups) * I + K)
    off, R, rows, a, w = _operands(rng, GROUPS[groups], 2 * I, K, gather)
    act = moe.grouped_gemm_fp8_alloc(a, w, dev(off), R, moe.MOE_EPI_SWIGLU_FP8, None if rows is None or R == 0 else dev(rows))
    av, wv = ref.rows_value(a.q.cpu().numpy(), a.sf.cpu().numpy()), ref.weights_value(w.q.cpu().numpy(), w.sf.cpu().numpy())
    y, mag = ref.product(av, wv, off, rows)
    want = ref.swiglu(y)
    # act: the sums' errors through silu (slope at most 1.1) and up, and 8 steps for exp2, the
    # reciprocal and the products; the exponent's argument is rounded: |gate| 2^-24 relative
    e = ref.core_error(K) * mag
    g, u = np.split(y, 2, 1)
    silu = np.divide(want, u, out=np.zeros_like(u), where=u != 0)
    err = 1.1 * np.abs(u) * e[:, :I] + (np.abs(silu) + e[:, :I]) * e[:, I:] + (8 + 2 * np.abs(g)) * 2 * U32 * np.abs(want)
    s = act.sf.cpu().numpy().astype(np.float64)
    peak = np.abs(want).reshape(R, I // 128, 128)
    tol = err.reshape(R, I // 128, 128).max(2, initial=0)
    if R:
        _near(s * 448, peak.max(2), tol + 4 * U32 * (peak.max(2) + tol), "scales")
    # a code is off by half a step of E4M3: 2^-4 of the value, or 2^-10 of the scale
    got = ref.rows_value(act.q.cpu().numpy(), act.sf.cpu().numpy())
    _near(got, want, (np.abs(want) + err) * 2.0 ** -4 + np.repeat(s, 128, 1) * 2.0 ** -10 + err + 4 * U32 * np.abs(want), "values")


@pytest.mark.parametrize("groups", GROUPS)
@pytest.mark.parametrize("N, K", [(16, 16), (144, 272), (256, 400)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_weight_gradient(groups, N, K, dtype):
    rng = np.random.default_rng(len(groups) * N + K)
    sizes = GROUPS[groups]
    off = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
    R = int(off[-1])
    if len(sizes) * N * K > 1 << 22:
        sizes, off = sizes[:40], off[:41]
        R = int(off[-1])
    dy = torch.from_numpy(rng.standard_normal((max(R, 1), N)).astype(np.float32)).to(torch.bfloat16).cuda()
    x = torch.from_numpy(rng.standard_normal((max(1, R // 2), K)).astype(np.float32)).cuda()
    rows = rng.integers(0, x.shape[0], max(R, 1)).astype(np.int32)
    o = dev(off)
    Y, X = moe.quantize_fp8_tokens_alloc(dy, o, R), moe.quantize_fp8_tokens_alloc(x, o, R, dev(rows))
    D = torch.full((len(sizes), N, K), float("nan"), dtype=dtype, device="cuda")
    moe.moe_grouped_wgrad_fp8(moe.make_wgrad_fp8_args(Y.q, Y.sf, X.q, X.sf, o, R, D))
    n = sum(-(-s // 128) for s in sizes)
    yv, xv = (ref.tokens_value(t.q[:n].cpu().numpy(), t.sf[:n].cpu().numpy()) for t in (Y, X))
    want, mag = ref.wgrad(yv, xv, off)
    half = U16 if dtype == torch.bfloat16 else U32
    _near(D.float().cpu().numpy(), want, half * np.abs(want) + (1 + half) * ref.sum_error(max(sizes)) * mag, groups)


def test_weight_gradient_of_half_blocks():
    """Groups whose last token block is up to half full, just over and full."""
    rng = np.random.default_rng(12)
    N, K, sizes = 144, 272, [1, 63, 64, 65, 127, 128, 129, 191, 192, 193, 0, 256]
    off = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
    R = int(off[-1])
    o = dev(off)
    Y, X = (moe.quantize_fp8_tokens_alloc(torch.from_numpy(rng.standard_normal((R, C)).astype(np.float32)).cuda(), o, R) for C in (N, K))
    D = moe.grouped_wgrad_fp8_alloc(Y, X, o, R)
    n = sum(-(-s // 128) for s in sizes)
    yv, xv = (ref.tokens_value(t.q[:n].cpu().numpy(), t.sf[:n].cpu().numpy()) for t in (Y, X))
    want, mag = ref.wgrad(yv, xv, off)
    _near(D.float().cpu().numpy(), want, U32 * np.abs(want) + (1 + U32) * ref.sum_error(max(sizes)) * mag, "half blocks")


def test_input_gradient_is_the_transposed_product():
    rng = np.random.default_rng(11)
    N, K, sizes = 272, 144, [50, 0, 7, 140]
    off = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
    R = int(off[-1])
    w, wt = moe.quantize_fp8_weights_alloc(torch.from_numpy(rng.standard_normal((4, N, K)).astype(np.float32)).cuda(), True)
    dy = moe.quantize_fp8_alloc(torch.from_numpy(rng.standard_normal((R, N)).astype(np.float32)).cuda())
    dx = moe.grouped_gemm_fp8_alloc(dy, wt, dev(off), R)
    wv = ref.weights_value(w.q.cpu().numpy(), w.sf.cpu().numpy()).transpose(0, 2, 1)
    want, mag = ref.product(ref.rows_value(dy.q.cpu().numpy(), dy.sf.cpu().numpy()), wv, off)
    _near(dx.float().cpu().numpy(), want, U16 * np.abs(want) + (1 + U16) * ref.core_error(N) * mag, "dx")


def test_product_gradients_match_differences():
    """The sum c . y of the product over operands that FP8 holds exactly (small whole numbers), against
    differences in x and in w: exact, because the product is linear in each."""
    rng = np.random.default_rng(12)
    N, K, sizes = 48, 80, [5, 0, 9]
    off = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
    R = int(off[-1])
    whole = lambda *s: torch.from_numpy(rng.integers(-3, 4, s).astype(np.float32))
    top = lambda t, d: t.index_fill(d, torch.zeros(1, dtype=torch.long), 7.0)   # every block's maximum is 7: scale 2^-6
    x, w, c = top(whole(R, K), 1), top(whole(3, N, K), 2), whole(R, N)
    w[:, 0, 0] = 7.0
    c[:, 0] = 7.0
    o = dev(off)
    f = lambda x, w: moe.grouped_gemm_fp8_alloc(moe.quantize_fp8_alloc(x.cuda()), moe.quantize_fp8_weights_alloc(w.cuda()), o, R).double().cpu()
    cols = c.clone()
    cols[off[:-1][np.array(sizes) > 0]] = 7.0          # for the weight gradient every column's maximum is 7 too
    xc = x.clone()
    xc[off[:-1][np.array(sizes) > 0]] = 7.0
    dx = moe.grouped_gemm_fp8_alloc(moe.quantize_fp8_alloc(c.cuda()), moe.quantize_fp8_weights_alloc(w.cuda(), True)[1], o, R).double().cpu()
    dw = moe.grouped_wgrad_fp8_alloc(moe.quantize_fp8_tokens_alloc(cols.cuda(), o, R), moe.quantize_fp8_tokens_alloc(xc.cuda(), o, R), o, R).double().cpu()
    for p, k in [(0, 3), (4, 79), (7, 16), (13, 40)]:
        up = x.clone()
        up[p, k] = 5.0 if x[p, k] != 5.0 else 4.0
        want = ((f(up, w) - f(x, w)) * c).sum() / (up[p, k] - x[p, k])
        assert abs(want - dx[p, k]) <= 2 * U16 * (f(up, w).abs() + f(x, w).abs() + dx.abs().max()).sum()
    for e, n, k in [(0, 3, 5), (2, 47, 79), (0, 0, 7), (1, 5, 5)]:
        up = w.clone()
        up[e, n, k] = 5.0
        want = ((f(xc, up) - f(xc, w)) * cols).sum() / (5.0 - w[e, n, k])
        y = (f(xc, up).abs() + f(xc, w).abs())[:, n]
        assert abs(want - dw[e, n, k]) <= U16 * (y * cols[:, n].abs()).sum() / abs(5.0 - w[e, n, k]) + U32 * 1e3


# ---- every kernel behind the product ----------------------------------------------------------

def _values_gpu(q, s, per_tile):
    v = torch.from_numpy(ref.e4m3_values()).cuda()[q.long()]
    s = s.double().repeat_interleave(128, -1)[..., :q.shape[-1]]
    if per_tile:
        s = s.repeat_interleave(128, -2)[..., :q.shape[-2], :]
    return v * s


def _uneven(rng, E, mean, empty=0.1):
    sizes = rng.integers(0, 2 * mean + 1, E) * (rng.random(E) >= empty)
    sizes[E // 2] = 5 * mean      # one long group
    return [int(s) for s in sizes]


KERNELS = {
    "few tiles, up to 16 rows": (6, 9, 272, 2064), "few tiles, up to 32 rows": (4, 26, 240, 1104),
    "few tiles, more rows": (3, 80, 400, 656), "many tiles, short": (90, 12, 528, 400), "many tiles, long": (90, 20, 528, 1552),
    "middle": (8, 220, 1648, 368), "large": (70, 70, 1040, 528), "large, four steps": (70, 60, 1024, 400),
    "large, whole steps": (64, 200, 1024, 1024), "weights past the caches": (40, 6, 2048, 2064),
    "weights past the caches, large": (72, 90, 2048, 1040),
}


@pytest.mark.parametrize("case", KERNELS)
@pytest.mark.parametrize("gather", [False, True])
def test_product_kernels(case, gather):
    E, mean, N, K = KERNELS[case]
    rng = np.random.default_rng(E * N + K)
    g = torch.Generator(device="cuda").manual_seed(E + N)
    sizes = _uneven(rng, E, mean)
    off = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
    R = int(off[-1])
    a = moe.quantize_fp8_alloc(torch.randn(R // 2 + 1 if gather else R, K, generator=g, device="cuda").to(torch.bfloat16))
    w = moe.quantize_fp8_weights_alloc(torch.randn(E, N, K, generator=g, device="cuda").to(torch.bfloat16))
    rows = torch.randint(0, a.q.shape[0], (R,), generator=g, device="cuda", dtype=torch.int32) if gather else None
    D = torch.full((R + 3, N), 7.0, dtype=torch.bfloat16, device="cuda")
    moe.moe_grouped_gemm_fp8(moe.make_gemm_fp8_args(a.q, a.sf, w.q, w.sf, dev(off), R, moe.MOE_EPI_NONE, D, A_rows=rows))
    av = _values_gpu(a.q, a.sf, False)
    av = av if rows is None else av[rows.long()]
    swiglu = N % 256 == 0 and moe.grouped_gemm_fp8_alloc(a, w, dev(off), R, moe.MOE_EPI_SWIGLU_FP8, rows)
    for e in range(E):
        lo, hi = int(off[e]), int(off[e + 1])
        wv = _values_gpu(w.q[e], w.sf[e], True)
        y, mag = av[lo:hi] @ wv.T, av[lo:hi].abs() @ wv.abs().T
        err = (D[lo:hi].double() - y).abs()
        bound = U16 * y.abs() + (1 + U16) * ref.core_error(K) * mag
        assert (err <= bound).all(), (case, e, (err / bound).max().item())
        if N % 256 == 0:
            # as in test_swiglu_quantized
            I = N // 2
            gate, up, eb = y[:, :I], y[:, I:], ref.core_error(K) * mag
            silu = gate / (1 + torch.exp(-gate))
            want = silu * up
            tol = 1.1 * up.abs() * eb[:, :I] + (silu.abs() + eb[:, :I]) * eb[:, I:] + (8 + 2 * gate.abs()) * 2 * U32 * want.abs()
            s = swiglu.sf[lo:hi].double().repeat_interleave(128, 1)
            got = _values_gpu(swiglu.q[lo:hi], swiglu.sf[lo:hi], False)
            lim = (want.abs() + tol) * 2.0 ** -4 + s * 2.0 ** -10 + tol + 4 * U32 * want.abs()
            assert ((got - want).abs() <= lim).all(), (case, e, "swiglu")
    assert (D[R:] == 7.0).all()
    again = torch.empty_like(D)
    moe.moe_grouped_gemm_fp8(moe.make_gemm_fp8_args(a.q, a.sf, w.q, w.sf, dev(off), R, moe.MOE_EPI_NONE, again, A_rows=rows))
    assert torch.equal(D[:R].view(torch.int16), again[:R].view(torch.int16))

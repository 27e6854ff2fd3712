"""The FP8 products on operands for which every sum is exact in any order, so a single lost, doubled
or misplaced element shows in every kernel behind moe_grouped_gemm_fp8, and the gradients against
differences without a tolerance."""
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


def kernel_of(R, E, N, K, swiglu=False):
    """The kernel that the library's rule takes, which follows the sizes alone."""
    hit = min(R, E)
    mean = R // hit
    tiles = lambda q, c: (R // q + hit) * -(-N // c)
    large = mean > 44 and K > 384 and tiles(256, 256) >= 192
    one_round = lambda q, c: hit * -(-mean // q) * -(-N // c) <= 256
    if large:
        return "256 x 256"
    if swiglu:
        return "32 rows" if one_round(32, 256) else "64 rows"
    q = 64 if mean > 32 else 32 if mean > 16 else 16
    if K >= 512 and q == 16 and one_round(16, 16):
        return "split 16, 16 columns"
    if K >= 512 and one_round(q, 32):
        return f"split {q}"
    if mean > 88 and tiles(128, 128) >= 192:
        return "128 x 128"
    if K <= 256 and tiles(64, 512) >= 768:
        return "64 rows, four tiles"
    return "64 rows, two stages" if K <= 512 else "64 rows"


def _sizes(E, mean):
    """E groups with an empty one, a short one and a long one, `mean` rows each in all."""
    sizes = np.full(E, mean)
    if E >= 3 and mean > 1:
        sizes[0], sizes[1], sizes[E // 2] = 0, 1, mean + mean + mean - 1
    return sizes


def _integers(E, mean, N, K, gather, wide):
    """Codes of -1, 0, 1 (wide: with two products of +-100352 that cancel in front of every sum) and scales
    of 1 and 2, 1/2 and 1: (offsets, R, A, B, rows, a's values, a function of e for B's values)."""
    g = torch.Generator(device="cuda").manual_seed(E * N + K)
    off = np.concatenate([[0], np.cumsum(_sizes(E, mean))]).astype(np.int32)
    R = int(off[-1])
    rows_A = R // 2 + 1 if gather else R
    code = {v: int(ref.e4m3_codes(np.float64(v))) for v in (-1, 0, 1, 448, 224, -224)}
    small = torch.tensor([code[-1], code[0], code[1]], dtype=torch.uint8, device="cuda")
    pick = lambda *s: small[torch.randint(0, 3, s, generator=g, device="cuda")]
    kb, nb = -(-K // 128), -(-N // 128)
    power = lambda lo, *s: 2.0 ** torch.randint(lo, lo + 2, s, generator=g, device="cuda").float()
    A, B = moe.FP8Tensor(pick(rows_A, K), power(0, rows_A, kb)), moe.FP8Tensor(pick(E, N, K), power(-1, E, nb, kb))
    if wide:
        A.q[:, :2] = code[448]
        B.q[..., 0], B.q[..., 1] = code[224], code[-224]
    rows = torch.randint(0, rows_A, (R,), generator=g, device="cuda", dtype=torch.int32) if gather else None
    table = torch.from_numpy(ref.e4m3_values()).cuda()
    up = lambda s, n, d: s.double().repeat_interleave(128, d).narrow(d, 0, n)
    a = table[A.q.long()] * up(A.sf, K, 1)
    return off, R, A, B, rows, a if rows is None else a[rows.long()], lambda e: table[B.q[e].long()] * up(up(B.sf[e], N, 0), K, 1)


PRODUCTS = {
    "split 16, 16 columns": [(6, 9, 272, 2064), (1, 1, 16, 528)],
    "split 16": [(8, 10, 784, 1040), (7, 16, 1040, 512)],
    "split 32": [(4, 26, 240, 1104), (9, 17, 528, 2064)],
    "split 64": [(3, 80, 400, 656), (2, 33, 1040, 1040)],
    "64 rows, four tiles": [(200, 12, 1616, 240), (256, 3, 2576, 16), (200, 70, 1024, 144)],
    "64 rows, two stages": [(90, 12, 528, 400), (5, 7, 48, 272)],
    "64 rows": [(90, 20, 528, 1552), (40, 6, 2048, 2064), (5, 48, 2064, 1040), (9, 1, 1040, 528)],      # the second one past the caches
    "128 x 128": [(8, 220, 1648, 368), (20, 130, 1040, 144)],
    "256 x 256": [(70, 70, 1040, 528), (64, 200, 1024, 1024), (72, 90, 2048, 1040), (30, 300, 1296, 400)],
}


@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("kernel, size", [(k, s) for k, sizes in PRODUCTS.items() for s in sizes])
def test_product(kernel, size, gather):
    E, mean, N, K = size
    off, R, A, B, rows, a, b = _integers(E, mean, N, K, gather, False)
    assert kernel_of(R, E, N, K) == kernel
    D = torch.full((R + 3, N), 7.5, dtype=torch.bfloat16, device="cuda")
    moe.moe_grouped_gemm_fp8(moe.make_gemm_fp8_args(A.q, A.sf, B.q, B.sf, dev(off), R, moe.MOE_EPI_NONE, D, A_rows=rows))
    for e in range(E):
        lo, hi = int(off[e]), int(off[e + 1])
        assert torch.equal(D[lo:hi].double(), (a[lo:hi] @ b(e).T).bfloat16().double()), e
    assert (D[R:] == 7.5).all()


def _check_act(act, y, what):
    """act = silu(gate) up of exact sums y: 8 steps for exp2, the reciprocal and the products, the rounded
    exponent's |gate| 2^-24, and the code's half step, 2^-4 of the value or 2^-10 of the scale."""
    I = y.shape[1] // 2
    gate, up = y[:, :I], y[:, I:]
    want = gate / (1 + torch.exp(-gate)) * up
    err = (8 + 2 * gate.abs()) * 2 * U32 * want.abs()
    s = act.sf.double()
    peak, tol = want.abs().unflatten(1, (I // 128, 128)).amax(2), err.unflatten(1, (I // 128, 128)).amax(2)
    assert ((s * 448 - peak).abs() <= tol + 4 * U32 * (peak + tol)).all(), what
    table = torch.from_numpy(ref.e4m3_values()).cuda()
    s = s.repeat_interleave(128, 1)
    lim = (want.abs() + err) * 2.0 ** -4 + s * 2.0 ** -10 + err + 4 * U32 * want.abs()
    assert ((table[act.q.long()] * s - want).abs() <= lim).all(), what


SWIGLU = {
    "32 rows": [(8, 5, 512, 1040), (3, 70, 256, 144), (1, 1, 256, 16)],
    "64 rows": [(150, 20, 512, 528), (9, 100, 2048, 144), (40, 6, 2048, 2064)],
    "256 x 256": [(70, 70, 1024, 528), (64, 200, 1024, 1024), (72, 90, 2048, 1040)],
}


@pytest.mark.parametrize("kernel, size, wide", [(k, s, w) for k, sizes in SWIGLU.items() for s in sizes for w in (False, True)
                                                if not (w and k == "256 x 256")])
def test_swiglu(kernel, size, wide):
    """wide: the smaller tiles sum whole products, so two that cancel leave the small ones as they are (the
    256 x 256 tile may cut them at 2^-13 of the large ones: not asked of it)."""
    E, mean, N, K = size
    off, R, A, B, rows, a, b = _integers(E, mean, N, K, True, wide)
    assert kernel_of(R, E, N, K, True) == kernel
    act = moe.grouped_gemm_fp8_alloc(A, B, dev(off), R, moe.MOE_EPI_SWIGLU_FP8, rows)
    for e in range(E):
        lo, hi = int(off[e]), int(off[e + 1])
        if hi > lo:
            _check_act(moe.FP8Tensor(act.q[lo:hi], act.sf[lo:hi]), a[lo:hi] @ b(e).T, e)


def test_gradients_equal_differences():
    """f = sum c . y over operands that FP8 holds exactly (-1, 0, 1 and a 7 in every block, so every scale is
    2^-6) and results that bf16 holds exactly (whole numbers up to 256): f's differences in x and in w
    are dx and dw without any rounding, and dx is c w."""
    rng = np.random.default_rng(41)
    N, K, sizes = 48, 144, [5, 0, 9]
    off = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
    R, o, e_of = int(off[-1]), dev(off), np.repeat(np.arange(3), sizes)
    whole = lambda *s: torch.from_numpy(rng.integers(-1, 2, s).astype(np.float32))
    x, w, c = whole(R, K), whole(3, N, K), whole(R, N)
    x[:, 0] = x[:, 128] = w[..., 0] = c[:, 0] = 7.0
    w[..., 128] = -7.0
    xc, cc = x.clone(), c.clone()
    first = [int(off[e]) for e in range(3) if sizes[e]]
    xc[first], cc[first] = 7.0, 7.0                       # a 7 in every column of every group
    exact = lambda x, w: torch.stack([w[e_of[p]].double() @ x[p].double() for p in range(R)])

    def y(x, w):
        got = moe.grouped_gemm_fp8_alloc(moe.quantize_fp8_alloc(x.cuda()), moe.quantize_fp8_weights_alloc(w.cuda()), o, R).double().cpu()
        want = exact(x, w)
        assert want.abs().max() <= 256 and torch.equal(got, want)
        return got

    dx = moe.grouped_gemm_fp8_alloc(moe.quantize_fp8_alloc(c.cuda()), moe.quantize_fp8_weights_alloc(w.cuda(), True)[1], o, R).double().cpu()
    assert torch.equal(dx, torch.stack([c[p].double() @ w[e_of[p]].double() for p in range(R)]).bfloat16().double())
    changed = 0
    for p in range(R):
        for k in rng.choice(np.arange(1, 128), 3, replace=False):
            up = x.clone()
            up[p, k] += 2 if x[p, k] < 1 else -2
            slope = (((y(up, w) - y(x, w)) * c).sum() / (up[p, k] - x[p, k])).item()
            assert slope == dx[p, k].item()
            changed += slope != 0
    assert changed > R
    dw = moe.grouped_wgrad_fp8_alloc(moe.quantize_fp8_tokens_alloc(cc.cuda(), o, R), moe.quantize_fp8_tokens_alloc(xc.cuda(), o, R), o, R).double().cpu()
    assert (dw[1] == 0).all()
    for e, n, k in [(0, 3, 5), (2, 47, 143), (0, 0, 7), (1, 5, 5), (2, 0, 127), (0, 47, 129)]:
        up = w.clone()
        up[e, n, k] += 2 if w[e, n, k] < 1 else -2
        assert (((y(xc, up) - y(xc, w)) * cc).sum() / (up[e, n, k] - w[e, n, k])).item() == dw[e, n, k].item()


def test_codes_in_their_own_type():
    """float8_e4m3fn codes in and out of every call: the bytes of the u8 ones."""
    g = torch.Generator(device="cuda").manual_seed(5)
    f8 = torch.float8_e4m3fn
    R, E, I, K, o = 40, 2, 128, 144, dev(np.array([0, 15, 40], np.int32))
    x, w = torch.randn(R, K, generator=g, device="cuda").bfloat16(), torch.randn(E, 2 * I, K, generator=g, device="cuda").bfloat16()
    typed = lambda t: moe.FP8Tensor(torch.empty_like(t.q).view(f8), torch.empty_like(t.sf))
    same = lambda a, b: torch.equal(a.q.view(torch.uint8), b.q) and torch.equal(a.sf, b.sf)
    a, (b, bt), t = moe.quantize_fp8_alloc(x), moe.quantize_fp8_weights_alloc(w, True), moe.quantize_fp8_tokens_alloc(x, o, R)
    a8, b8, bt8, t8 = typed(a), typed(b), typed(bt), typed(t)
    t8.q.view(torch.uint8).copy_(t.q)      # (blocks that no group has are not written)
    t8.sf.copy_(t.sf)
    moe.moe_quantize_fp8(x, a8.q, a8.sf)
    moe.moe_quantize_fp8_weights(w, b8.q, b8.sf, bt8.q, bt8.sf)
    moe.moe_quantize_fp8_tokens(x, o, R, t8.q, t8.sf)
    assert same(a8, a) and same(b8, b) and same(bt8, bt) and same(t8, t)
    y, act = (moe.grouped_gemm_fp8_alloc(a, b, o, R, e) for e in (moe.MOE_EPI_NONE, moe.MOE_EPI_SWIGLU_FP8))
    assert torch.equal(moe.grouped_gemm_fp8_alloc(a8, b8, o, R), y)
    act8 = typed(act)
    moe.moe_grouped_gemm_fp8(moe.make_gemm_fp8_args(a8.q, a8.sf, b8.q, b8.sf, o, R, moe.MOE_EPI_SWIGLU_FP8, act8.q, act8.sf))
    assert same(act8, act)
    assert torch.equal(moe.grouped_wgrad_fp8_alloc(t8, t8, o, R), moe.grouped_wgrad_fp8_alloc(t, t, o, R))


# ---- whole sums asked for ---------------------------------------------------------------------

WHOLE = {"64 rows": [(1, 1, 16, 16), (6, 9, 272, 2064), (90, 12, 528, 400), (40, 6, 2048, 2064)],
         "128 rows": [(8, 220, 1648, 368), (64, 200, 1024, 1024), (30, 300, 1296, 400)]}


@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("size", [s for sizes in WHOLE.values() for s in sizes])
def test_whole_product(size, gather):
    """Two products of 100352 that cancel in front of every sum take nothing from the others."""
    E, mean, N, K = size
    off, R, A, B, rows, a, b = _integers(E, mean, N, K, gather, True)
    D = torch.full((R + 3, N), 7.5, dtype=torch.bfloat16, device="cuda")
    moe.moe_grouped_gemm_fp8(moe.make_gemm_fp8_args(A.q, A.sf, B.q, B.sf, dev(off), R, moe.MOE_EPI_NONE | moe.MOE_SUMS_WHOLE, D, A_rows=rows))
    for e in range(E):
        lo, hi = int(off[e]), int(off[e + 1])
        assert torch.equal(D[lo:hi].double(), (a[lo:hi] @ b(e).T).bfloat16().double()), e
    assert (D[R:] == 7.5).all()


@pytest.mark.parametrize("size", [s for sizes in SWIGLU.values() for s in sizes])
def test_whole_swiglu(size):
    E, mean, N, K = size
    off, R, A, B, rows, a, b = _integers(E, mean, N, K, True, True)
    act = moe.grouped_gemm_fp8_alloc(A, B, dev(off), R, moe.MOE_EPI_SWIGLU_FP8 | moe.MOE_SUMS_WHOLE, rows)
    for e in range(E):
        lo, hi = int(off[e]), int(off[e + 1])
        if hi > lo:
            _check_act(moe.FP8Tensor(act.q[lo:hi], act.sf[lo:hi]), a[lo:hi] @ b(e).T, e)


@pytest.mark.parametrize("E, mean, N, K", [(3, 20, 272, 2064), (8, 220, 1648, 368), (20, 400, 1040, 1040)])
def test_whole_product_of_random_operands(E, mean, N, K):
    """Within binary32 sums' bound and bf16's half step."""
    g = torch.Generator(device="cuda").manual_seed(E)
    off = np.concatenate([[0], np.cumsum(_sizes(E, mean))]).astype(np.int32)
    R = int(off[-1])
    A = moe.quantize_fp8_alloc(torch.randn(R, K, generator=g, device="cuda").bfloat16())
    B = moe.quantize_fp8_weights_alloc(torch.randn(E, N, K, generator=g, device="cuda").bfloat16())
    D = moe.grouped_gemm_fp8_alloc(A, B, dev(off), R, moe.MOE_EPI_NONE | moe.MOE_SUMS_WHOLE)
    table = torch.from_numpy(ref.e4m3_values()).cuda()
    up = lambda s, n, d: s.double().repeat_interleave(128, d).narrow(d, 0, n)
    a = table[A.q.long()] * up(A.sf, K, 1)
    for e in range(E):
        lo, hi = int(off[e]), int(off[e + 1])
        w = table[B.q[e].long()] * up(up(B.sf[e], N, 0), K, 1)
        y, mag = a[lo:hi] @ w.T, a[lo:hi].abs() @ w.abs().T
        assert ((D[lo:hi].double() - y).abs() <= U16 * y.abs() + (1 + U16) * ref.sum_error(K) * mag).all(), e


def test_whole_sums_do_not_depend_on_the_other_rows():
    """A layer's output for its first tokens, alone and in a prompt, with a graph's replays between."""
    E, k, H, I = 8, 2, 528, 256
    g = torch.Generator(device="cuda").manual_seed(9)
    randn = lambda *s: torch.randn(*s, generator=g, device="cuda")
    W1, W2 = (moe.quantize_fp8_weights_alloc((0.05 * randn(*s)).bfloat16()) for s in ((E, 2 * I, H), (E, H, I)))
    logits, x = randn(3000, E), randn(3000, H).bfloat16()
    run = lambda T: moe.MoEFP8LayerPlan(T, E, k, H, I, W1, W2, whole_sums=True).forward(logits[:T].contiguous(), x[:T].contiguous())
    want = run(3000).view(torch.int16)
    for T in (1, 7, 300):
        assert torch.equal(run(T).view(torch.int16), want[:T]), T
    plan = moe.MoEFP8LayerPlan(7, E, k, H, I, W1, W2, whole_sums=True)
    l, y = logits[:7].clone(), x[:7].clone()
    graph = plan.graph(l, y)
    for first in (0, 40, 2000):
        l.copy_(logits[first:first + 7])
        y.copy_(x[first:first + 7])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(plan.out.view(torch.int16), want[first:first + 7]), first
        run(300)


def test_layer_refuses_a_stream_of_another_device_before_its_first_launch():
    class Elsewhere:
        device_index, cuda_stream = 1, 0
    E, k, H, I = 4, 2, 256, 128
    g = torch.Generator(device="cuda").manual_seed(2)
    W1, W2 = (moe.quantize_fp8_weights_alloc(torch.randn(*s, generator=g, device="cuda")) for s in ((E, 2 * I, H), (E, H, I)))
    plan = moe.MoEFP8LayerPlan(5, E, k, H, I, W1, W2)
    for t in (plan.ids, plan.off):
        t.fill_(-5)
    logits, x = torch.randn(5, E, generator=g, device="cuda"), torch.randn(5, H, generator=g, device="cuda")
    with pytest.raises(moe.MoeError):
        plan.forward(logits, x, Elsewhere())
    torch.cuda.synchronize()
    assert (plan.ids == -5).all() and (plan.off == -5).all()
    assert not (plan.forward(logits, x, torch.cuda.current_stream()) != plan.forward(logits, x)).any()


def test_layer_of_no_tokens():
    z = lambda *s: moe.quantize_fp8_weights_alloc(torch.zeros(*s, device="cuda"))
    for whole in (False, True):
        plan = moe.MoEFP8LayerPlan(0, 4, 2, 256, 128, z(4, 256, 256), z(4, 256, 128), whole_sums=whole)
        out = plan.forward(torch.empty(0, 4, device="cuda"), torch.empty(0, 256, device="cuda"))
        torch.cuda.synchronize()
        assert out.shape == (0, 256) and (plan.off == 0).all()

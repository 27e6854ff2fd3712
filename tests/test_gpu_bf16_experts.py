"""The gated experts in bf16 (products, SwiGLU epilogue and its backward pass, weight gradients) on the
GPU against 64 bits.  Products of small whole numbers have exact sums, so there every result has to equal
the reference rounded once; where the operands are random the bounds are those of binary32 sums in any
order.  Rows behind the last group, rows that no group reads and the weights of empty experts hold NaN
or a pattern, which has to stay out of, or in, every result."""
from __future__ import annotations

import pytest
import torch

import block_scaled_fp4_02_amd as moe
from tests import experts_ref as ref

pytestmark = pytest.mark.gpu

BF16, TR = torch.bfloat16, moe.MOE_LAYOUT_TRANSPOSED
MARK = -77.0   # what outputs hold before a call


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    moe.lib()
    yield
    torch.cuda.synchronize()


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _ints(g, *s, most=3, scale=1.0):
    return (torch.randint(-most, most + 1, s, generator=g, device="cuda").float() * scale).to(BF16)


def _randn(g, *s, scale=1.0):
    return (scale * torch.randn(*s, generator=g, device="cuda")).to(BF16)


def _offsets(sizes):
    off = torch.zeros(len(sizes) + 1, dtype=torch.int32)
    off[1:] = torch.tensor(sizes).cumsum(0)
    return off.cuda()


def _operand(g, sizes, K, gather, pad, make=_ints, **kw):
    """(A, A_rows or None, R): rows of the groups, `pad` more permuted rows behind the last, NaN where nothing reads."""
    R = sum(sizes)
    if not gather:
        A = torch.full((R + pad, K), float("nan"), dtype=BF16, device="cuda")
        A[:R] = make(g, R, K, **kw)
        return A, None, R + pad
    T = R // 2 + 3
    A = make(g, T, K, **kw)
    rows = torch.randint(0, T - 2, (R + pad,), generator=g, device="cuda", dtype=torch.int32)
    A[T - 2:] = float("nan")
    rows[R:] = T - 1
    return A, rows, R + pad


def _weights(g, sizes, N, K, make=_ints, **kw):
    W = make(g, len(sizes), N, K, **kw)
    for e, n in enumerate(sizes):
        if n == 0:
            W[e] = float("nan")
    return W


# which kernel takes them, row-major: 16- and 32-row split tiles, 32- and 64-row tiles, 128 and 256 squared, and their edges
PRODUCTS = {
    "one row": ([1], 8, 8), "split 16": ([1, 0, 3], 24, 264), "split 16, two chunks": ([30, 0, 2], 40, 520), "split 32": ([5], 4808, 512),
    "split 32, two chunks": ([40, 20, 0], 2056, 136), "split 32, short": ([20, 0, 40, 7], 1000, 72), "32 rows": ([64, 128, 1], 2600, 64),
    "64 rows": ([20] * 40 + [0, 70], 1024, 136), "full chunks": ([64, 128, 1], 13000, 64), "many small": ([3] * 90 + [0] * 30, 72, 136),
    "middle": ([130, 200, 0, 95], 6400, 136), "middle, one step": ([256, 128], 12800, 40), "large": ([300, 0, 517, 45], 12808, 200),
    "large, one step": ([600, 90], 16392, 8), "large, halves": ([256, 512, 100], 22528, 64), "large, two steps": ([256, 512], 12288, 128), "1024 experts": ([1] * 1000 + [0] * 20 + [50] * 4, 16, 72),
}


@pytest.mark.parametrize("gather", [False, True], ids=["own rows", "gathered"])
@pytest.mark.parametrize("transposed", [False, True], ids=["row-major", "transposed"])
@pytest.mark.parametrize("name", PRODUCTS)
def test_product(name, transposed, gather):
    sizes, N, K = PRODUCTS[name]
    g, off = _gen(len(name) + 2 * gather), _offsets(sizes)
    A, rows, R = _operand(g, sizes, K, gather, 5)
    W = _weights(g, sizes, N, K)
    D = torch.full((R, N), MARK, dtype=BF16, device="cuda")
    B = W.transpose(1, 2).contiguous() if transposed else W
    moe.moe_grouped_gemm_bf16(moe.make_gemm_bf16_args(A, B, off, R, moe.MOE_EPI_NONE, D, A_rows=rows, B_layout=TR if transposed else 0))
    want, _ = ref.product(A, W, off, rows)   # whole numbers below 2^24: exact in binary32
    assert torch.equal(D[:sum(sizes)].double(), ref.bf16(want))
    assert (D[sum(sizes):] == MARK).all()


GATED = {
    "one row": ([1], 8, 8), "split 16": ([1, 0, 3], 24, 264), "split 16, two chunks": ([30, 0, 2], 40, 520), "split 32": ([5], 2408, 512),
    "split 32, two chunks": ([40, 0, 20], 1032, 72), "64 rows": ([20] * 40 + [0, 70], 1024, 136), "short K": ([9, 100], 136, 8),
    "large": ([300, 0, 517, 45], 6408, 200), "large, one step": ([600, 90], 8200, 64), "large, halves": ([256, 512, 100], 11264, 72),
}


@pytest.mark.parametrize("gather", [False, True], ids=["own rows", "gathered"])
@pytest.mark.parametrize("name", GATED)
def test_gated(name, gather):
    sizes, I, K = GATED[name]
    g, off, n = _gen(len(name) + gather), _offsets(sizes), sum(sizes)
    # sums are multiples of 1/16 below 2^20: exact in binary32
    A, rows, R = _operand(g, sizes, K, gather, 3, scale=0.25)
    W = _weights(g, sizes, 2 * I, K, scale=0.25)
    act, Z = torch.full((R, I), MARK, dtype=BF16, device="cuda"), torch.full((R, 2 * I), MARK, dtype=BF16, device="cuda")
    moe.moe_grouped_gemm_bf16(moe.make_gemm_bf16_args(A, W, off, R, moe.MOE_EPI_SWIGLU, act, Z, rows))
    y, _ = ref.product(A, W, off, rows)
    assert torch.equal(Z[:n].double(), ref.bf16(y))
    assert ref.close(act[:n], ref.swiglu(y), ref.swiglu_error(y))
    assert (act[n:] == MARK).all() and (Z[n:] == MARK).all()
    again = torch.full((R, I), MARK, dtype=BF16, device="cuda")
    moe.moe_grouped_gemm_bf16(moe.make_gemm_bf16_args(A, W, off, R, moe.MOE_EPI_SWIGLU, again, None, rows))
    assert torch.equal(act, again)


BACKWARD = {"one row": ([1], 8, 8), "small": ([20, 0, 40, 7], 200, 72), "32 rows": ([64, 128, 1], 136, 64), "64 rows": ([20] * 40 + [0, 70], 1024, 136),
            "many small": ([3] * 90 + [0] * 30, 72, 136), "middle": ([130, 200, 0, 95], 6400, 136), "large": ([300, 0, 517, 45], 12808, 200), "large, one step": ([600, 90], 16392, 8)}


@pytest.mark.parametrize("name", BACKWARD)
def test_gated_backward(name):
    sizes, I, H = BACKWARD[name]
    g, off, n = _gen(len(name)), _offsets(sizes), sum(sizes)
    dY, _, R = _operand(g, sizes, H, False, 4, scale=0.25)
    W2 = _weights(g, sizes, I, H, scale=0.25).transpose(1, 2).contiguous()   # [E, H, I]
    Z = _randn(g, R, 2 * I, scale=4.0)
    Z[0, :6] = torch.tensor([0.0, -0.0, 100.0, -100.0, 3e38, -3e38], device="cuda")
    dZ = torch.full((R, 2 * I), MARK, dtype=BF16, device="cuda")
    moe.moe_grouped_gemm_bf16(moe.make_gemm_bf16_args(dY, W2, off, R, moe.MOE_EPI_SWIGLU_BACKWARD, dZ, Z, B_layout=TR))
    da, _ = ref.product(dY, W2.transpose(1, 2), off)
    want, err = ref.swiglu_backward(da, Z[:n].double())
    fits = want.abs() < 3e38
    assert fits.float().mean() > 0.9 and torch.isfinite(dZ[:n][fits]).all()
    assert ref.close(dZ[:n][fits], want[fits], err[fits])
    assert (dZ[n:] == MARK).all()
    moe.moe_grouped_gemm_bf16(moe.make_gemm_bf16_args(dY, W2, off, R, moe.MOE_EPI_SWIGLU_BACKWARD, Z, Z, B_layout=TR))   # in place
    assert torch.equal(Z[:n].nan_to_num(7.0), dZ[:n].nan_to_num(7.0))


WGRADS = {"one row": ([1], 8, 8), "small": ([20, 0, 40, 7], 200, 72), "whole steps": ([64, 128, 0, 1], 136, 264), "long": ([3000], 72, 136),
          "many": ([3, 0, 65] * 30, 40, 24), "wide": ([300, 0, 517, 45, 64], 2568, 1032), "large": ([5000, 8, 0, 40, 4609], 2568, 1032), "large, one group": ([2825], 3336, 3592),
          "large, halves": ([1500, 1600], 2816, 4096)}


@pytest.mark.parametrize("gather", [False, True], ids=["own rows", "gathered"])
@pytest.mark.parametrize("dtype", [torch.float32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("name", WGRADS)
def test_weight_gradient(name, dtype, gather):
    sizes, N, K = WGRADS[name]
    g, off, n = _gen(len(name) + gather), _offsets(sizes), sum(sizes)
    X, rows, R = _operand(g, sizes, K, gather, 5)
    Y, _, _ = _operand(g, sizes, N, False, 5)
    D = torch.full((len(sizes), N, K), MARK, dtype=dtype, device="cuda")
    moe.moe_grouped_wgrad_bf16(moe.make_wgrad_bf16_args(Y, X, off, R, D, rows))
    want, _ = ref.wgrad(Y[:n], X, off, None if rows is None else rows[:n])
    assert torch.equal(D.double(), ref.bf16(want) if dtype == BF16 else want)


def test_a_groups_nan_stays_in_it():
    """Tiles end inside their group: what the next group holds does not reach this one's sums."""
    sizes, N, K = [70, 33, 70], 264, 136
    g, off = _gen(1), _offsets(sizes)
    A, W, Y = _ints(g, 173, K), _ints(g, 3, N, K), _ints(g, 173, N)
    want, (dw, _) = ref.product(A, W, off)[0], ref.wgrad(Y, A, off)
    bad = slice(70, 103)
    A[bad], Y[bad] = float("nan"), float("inf")
    for layout, B in ((0, W), (TR, W.transpose(1, 2).contiguous())):
        D = torch.empty(173, N, dtype=BF16, device="cuda")
        moe.moe_grouped_gemm_bf16(moe.make_gemm_bf16_args(A, B, off, 173, 0, D, B_layout=layout))
        assert torch.equal(D[:70].double(), ref.bf16(want[:70])) and torch.equal(D[103:].double(), ref.bf16(want[103:])) and D[bad].isnan().all()
    D = moe.grouped_wgrad_bf16_alloc(Y, A, off, 173)
    assert torch.equal(D[0].double(), dw[0]) and torch.equal(D[2].double(), dw[2]) and D[1].isnan().all()


@pytest.mark.parametrize("sizes", [[3], [40, 20], [700, 900]])
def test_denormals_count(sizes):
    """Elements and weights below the least normal number, and results there."""
    g, off, n, N, K = _gen(5), _offsets(sizes), sum(sizes), 12808, 40
    A, W, Y = _ints(g, n, K), _ints(g, len(sizes), N, K), _ints(g, n, N)
    want, dw = ref.product(A, W, off)[0], ref.wgrad(Y, A, off)[0]
    tiny, big = 2.0 ** -130, 2.0 ** 100
    for a, w in ((tiny, big), (big, tiny), (tiny, 1.0)):
        B = (W.float() * w).to(BF16)
        for layout, V in ((0, B), (TR, B.transpose(1, 2).contiguous())):
            D = torch.empty(n, N, dtype=BF16, device="cuda")
            moe.moe_grouped_gemm_bf16(moe.make_gemm_bf16_args((A.float() * a).to(BF16), V, off, n, 0, D, B_layout=layout))
            assert torch.equal(D.double(), ref.bf16(want * (a * w))), (a, w, layout)
        D = moe.grouped_wgrad_bf16_alloc((Y.float() * w).to(BF16), (A.float() * a).to(BF16), off, n)
        assert torch.equal(D.double(), dw * (a * w)), (a, w)


def test_no_rows():
    g, off = _gen(2), torch.zeros(4, dtype=torch.int32, device="cuda")
    W = _ints(g, 3, 32, 16)
    none = lambda c: torch.empty(0, c, dtype=BF16, device="cuda")  # noqa: E731
    assert moe.grouped_gemm_bf16_alloc(none(16), W, off, 0).shape == (0, 32)
    act, Z = moe.gated_ffn_alloc(none(16), W, off, 0)
    assert act.shape == (0, 16) and Z.shape == (0, 32)
    assert not moe.grouped_wgrad_bf16_alloc(none(32), none(16), off, 0).any()
    # rows that no group has: nothing is written, gradients are zero
    A, D = _ints(g, 9, 16), torch.full((9, 32), MARK, dtype=BF16, device="cuda")
    moe.moe_grouped_gemm_bf16(moe.make_gemm_bf16_args(A, W, off, 9, 0, D))
    assert (D == MARK).all()
    rows = torch.arange(9, dtype=torch.int32, device="cuda")
    assert not moe.grouped_wgrad_bf16_alloc(_ints(g, 9, 32), A, off, 9, X_rows=rows).any()


def test_bad_offsets_and_rows_stay_in_bounds():
    """Offsets that are not monotone or lie outside, and row numbers outside, are clamped: some rows get
    another group's product, none outside [0, R) is touched, and nothing is read outside the operands."""
    g = _gen(3)
    R, N, K = 100, 136, 72
    room = torch.full((R + 64, 2 * N), MARK, dtype=BF16, device="cuda")
    A, W = _ints(g, R, K), _ints(g, 4, N, K)
    rows = torch.randint(-2 ** 31, 2 ** 31 - 1, (R,), generator=g, device="cuda").to(torch.int32)
    for off in ([0, 50, 20, 100, 100], [-5, 30, 2 ** 31 - 1, -2 ** 31, 60], [90, 80, 70, 60, 50], [2 ** 30, 2 ** 30, 0, 10 ** 6, 7]):
        off = torch.tensor(off, dtype=torch.int32, device="cuda")
        for A_rows in (None, rows):
            D = room.view(-1)[:R * N].view(R, N)
            moe.moe_grouped_gemm_bf16(moe.make_gemm_bf16_args(A, W, off, R, 0, D, A_rows=A_rows))
            assert (room.view(-1)[R * N:] == MARK).all() and torch.isfinite(D.float()).all()
            dw = moe.grouped_wgrad_bf16_alloc(_ints(g, R, N), A, off, R, X_rows=A_rows)
            assert torch.isfinite(dw).all()


@pytest.mark.parametrize("T, E, k, I, H", [(1, 8, 2, 64, 256), (150, 6, 2, 136, 400), (1100, 8, 4, 1032, 1544)], ids=["token", "batch", "large"])
def test_training_step(T, E, k, I, H):
    """The operators together as a training loop calls them, each held to 64 bits on what the one before
    gave, and all of them to automatic differentiation of the block in 64 bits."""
    g = _gen(T)
    logits = torch.randn(T, E, generator=g, device="cuda")
    ids, _, off, src, tsr = moe.route_permute_alloc(logits, k)
    R = T * k
    x, w1, w2, dy = _randn(g, T, H), _randn(g, E, 2 * I, H, scale=H ** -0.5), _randn(g, E, H, I, scale=I ** -0.5), _randn(g, R, H)
    act, z = moe.gated_ffn_alloc(x, w1, off, R, A_rows=src)
    y = moe.grouped_gemm_bf16_alloc(act, w2, off, R)
    dz = moe.gated_ffn_backward_alloc(dy, w2, z, off, R)
    dx = moe.grouped_gemm_bf16_alloc(dz, w1, off, R, transposed=True)
    dw1 = moe.grouped_wgrad_bf16_alloc(dz, x, off, R, X_rows=src)
    dw2 = moe.grouped_wgrad_bf16_alloc(dy, act, off, R)
    token_dx = torch.empty(T, H, dtype=BF16, device="cuda")
    moe.moe_finalize(dx, torch.ones(T, k, device="cuda"), tsr, token_dx)

    want, mag = ref.product(x, w1, off, src)
    err = ref.sum_error(H) * mag
    assert ref.close(z, want, err)
    gate, up = want.chunk(2, 1)
    eg, eu = err.chunk(2, 1)   # |silu'| <= 1.1
    assert ref.close(act, ref.swiglu(want), 1.1 * eg * (up.abs() + eu) + (torch.nn.functional.silu(gate).abs() + 1.1 * eg) * eu + 1.01 * ref.swiglu_error(want))
    want, mag = ref.product(act, w2, off)
    assert ref.close(y, want, ref.sum_error(I) * mag)
    da, mag = ref.product(dy, w2.transpose(1, 2), off)
    want, err = ref.swiglu_backward(da, z.double())
    _, slope = ref.swiglu_backward(torch.ones_like(da), z.double())   # per unit of da: the error bound is over it in every factor
    gz, uz = z.double().chunk(2, 1)
    s = torch.sigmoid(gz)
    factor = torch.cat([(uz * s * (1 + gz * (1 - s))).abs(), (gz * s).abs()], 1)
    assert ref.close(dz, want, 1.01 * err + (factor + slope) * (ref.sum_error(H) * mag).repeat(1, 2))
    want, mag = ref.product(dz, w1.transpose(1, 2), off)
    assert ref.close(dx, want, ref.sum_error(2 * I) * mag)
    for got, a, b, rows in ((dw1, dz, x, src), (dw2, dy, act, None)):
        want, mag = ref.wgrad(a, b, off, rows)
        assert ((got.double() - want).abs() <= ref.sum_error(R) * mag).all()

    # the whole: four tensors are rounded to bf16 on the way (z, act, dz, and the result), half a step
    # each relative to a value or, where a formula's terms cancel, to a few times it: 2^-5 of the 2-norm
    leaves = [t.double().requires_grad_() for t in (x, w1, w2)]
    total = 0.0
    for e, lo, hi in ref.groups(off):
        total = total + ((ref.swiglu(leaves[0][src[lo:hi].long()] @ leaves[1][e].T) @ leaves[2][e].T) * dy[lo:hi].double()).sum()
    total.backward()
    for got, leaf in zip((token_dx, dw1, dw2), leaves):
        assert (got.double() - leaf.grad).norm() <= 2.0 ** -5 * leaf.grad.norm()


def test_results_do_not_depend_on_the_stream_and_repeat():
    g = _gen(11)
    sizes, N, K = [300, 0, 517, 45], 2064, 520
    off, R = _offsets(sizes), 862
    A, W = _randn(g, R, K), _randn(g, 4, N, K)
    first = (moe.gated_ffn_alloc(A, W, off, R), moe.grouped_wgrad_bf16_alloc(_randn(_gen(12), R, N), A, off, R))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    second = (moe.gated_ffn_alloc(A, W, off, R, stream=s), None)
    with torch.cuda.stream(s):
        dw = moe.grouped_wgrad_bf16_alloc(_randn(_gen(12), R, N), A, off, R)
    torch.cuda.synchronize()
    assert torch.equal(first[0][0], second[0][0]) and torch.equal(first[0][1], second[0][1]) and torch.equal(first[1], dw)


def test_step_captured_and_replayed():
    """A whole step in a graph, replayed on new inputs with eager work between the replays."""
    g = _gen(21)
    T, E, k, I, H = 90, 6, 2, 136, 264
    R = T * k
    x, dy = _randn(g, T, H), _randn(g, R, H)
    w1, w2 = _randn(g, E, 2 * I, H, scale=0.06), _randn(g, E, H, I, scale=0.08)
    logits = torch.randn(T, E, generator=g, device="cuda")

    def step():
        _, _, off, src, _ = moe.route_permute_alloc(logits, k)
        act, z = moe.gated_ffn_alloc(x, w1, off, R, A_rows=src)
        y = moe.grouped_gemm_bf16_alloc(act, w2, off, R)
        dz = moe.gated_ffn_backward_alloc(dy, w2, z, off, R)
        dx = moe.grouped_gemm_bf16_alloc(dz, w1, off, R, transposed=True)
        grads = [moe.grouped_wgrad_bf16_alloc(dz, x, off, R, X_rows=src), moe.grouped_wgrad_bf16_alloc(dy, act, off, R)]
        norm = moe.clip_grad_norm(grads, 0.5)
        return [act, z, y, dx, *grads, norm]

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for i in range(4):
        for t in (x, dy):
            t.copy_(_randn(g, *t.shape))
        logits.copy_(torch.randn(T, E, generator=g, device="cuda"))
        want = step()
        for t in got:
            t.fill_(MARK)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)), i


def test_offsets_past_32_bits():
    """Weights, rows and results beyond 2^32 bytes: the last expert and the last rows."""
    g = _gen(31)
    E, N, K = 9, 16384, 16384     # 4.8 GB of weights
    W = torch.zeros(E, N, K, dtype=BF16, device="cuda")
    W[-1] = _ints(g, N, K, most=1)
    off = _offsets([0] * (E - 1) + [70])
    A = _ints(g, 70, K, most=1)
    D = moe.grouped_gemm_bf16_alloc(A, W, off, 70)
    assert torch.equal(D.double(), ref.bf16(ref.product(A, W, off)[0]))
    dw = torch.empty(E, N, K, dtype=BF16, device="cuda")
    Y = _ints(g, 70, N, most=1)
    moe.moe_grouped_wgrad_bf16(moe.make_wgrad_bf16_args(Y, A, off, 70, dw))
    assert not dw[:-1].any() and torch.equal(dw[-1].double(), Y.double().T @ A.double())
    del W, dw
    R, C = 70000, 32768           # 4.6 GB of rows, of results, of Y
    big = torch.zeros(R, C, dtype=BF16, device="cuda")
    big[-40:] = _ints(g, 40, C, most=1)
    off = _offsets([R - 40, 40])
    W = _ints(g, 2, 16, C, most=1)
    D = moe.grouped_gemm_bf16_alloc(big, W, off, R)
    assert not D[:-40].any() and torch.equal(D[-40:].double(), ref.bf16(big[-40:].double() @ W[1].double().T))
    x = _ints(g, R, 16, most=1)
    dw = moe.grouped_wgrad_bf16_alloc(big, x, off, R)
    assert not dw[0].any() and torch.equal(dw[1].double(), big[-40:].double().T @ x[-40:].double())
    Wt = _ints(g, 2, 16, C, most=1)   # as the transposed operand: results [R, C]
    moe.moe_grouped_gemm_bf16(moe.make_gemm_bf16_args(x, Wt, off, R, 0, big, B_layout=TR))
    assert torch.equal(big[-40:].double(), ref.bf16(x[-40:].double() @ Wt[1].double()))


def test_sigmoids_far_out():
    """Gates where the sigmoid leaves binary32's normal range, with factors that make it count: below 2^-126 it
    may be zero, everywhere else it keeps its bound; in every kernel that takes one."""
    gates = torch.tensor([-80.0, -86.5, -87.0, -87.5, -88.0, -88.5, -89.0, -95.0, -100.0, -104.0, -120.0, 80.0, 87.5, 89.0, 104.0, 120.0], device="cuda")
    n, I, big = 16, 64, 2.0 ** 100
    for rows in ([n], [n] * 40):
        off, R = _offsets(rows), sum(rows)
        A = torch.zeros(R, 64, dtype=BF16, device="cuda")
        A[:, 0], A[:, 1] = gates.repeat(len(rows)).to(BF16), 1.0
        W = torch.zeros(len(rows), 2 * I, 64, dtype=BF16, device="cuda")
        W[:, :I, 0], W[:, I:, 1] = 1.0, big
        act, z = moe.gated_ffn_alloc(A, W, off, R)
        y, _ = ref.product(A, W, off)
        gate, up = y.chunk(2, 1)
        assert ref.close(act, ref.swiglu(y), ref.swiglu_error(y) + (gate * up).abs() * 2.0 ** -126)
        W2 = torch.zeros(len(rows), 64, I, dtype=BF16, device="cuda")
        W2[:, 1] = 1.0
        dz = moe.gated_ffn_backward_alloc(A, W2, z, off, R)
        want, err = ref.swiglu_backward(torch.ones_like(gate), z.double())
        assert ref.close(dz, want, err + torch.cat([up * (1 + gate.abs()), gate.abs()], 1).abs() * 2.0 ** -126)

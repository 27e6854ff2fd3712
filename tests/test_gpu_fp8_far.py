"""FP8 operands and results whose byte offsets pass 2^31 and 2^32, checked on samples that lie behind
those borders."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import block_scaled_fp4_02_amd as moe
from tests import fp8_ref as ref
from tests.fp8_ref import U16, U32, dev

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.empty_cache()
    yield
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


def _codes(g, *shape):
    """Random codes of every sign and exponent but the NaNs."""
    c = torch.randint(0, 127, shape, generator=g, device="cuda", dtype=torch.uint8)
    return c | (torch.randint(0, 2, shape, generator=g, device="cuda", dtype=torch.uint8) << 7)


def _value(q, s):
    v = torch.from_numpy(ref.e4m3_values()).cuda()[q.long()]
    return v * s.double().repeat_interleave(128, -1)[..., :q.shape[-1]]


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def test_weights_past_32_bits():
    """Three experts of the largest size one descriptor reaches: the second and third start past 2^31
    and 2^32 bytes."""
    E, N, K, sizes = 3, 131056, 16384, [2, 0, 3]
    g = _gen(1)
    B = torch.empty(E, N, K, dtype=torch.uint8, device="cuda")
    for e in range(E):
        for n in range(0, N, 16384):
            B[e, n:n + 16384] = _codes(g, min(16384, N - n), K)
    Bs = torch.rand(E, N // 128 + 1, K // 128, generator=g, device="cuda")[:, :-(-N // 128)].contiguous()
    off = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
    R = int(off[-1])
    A, As = _codes(g, R, K), torch.rand(R, K // 128, generator=g, device="cuda")
    D = torch.empty(R, N, dtype=torch.bfloat16, device="cuda")
    moe.moe_grouped_gemm_fp8(moe.make_gemm_fp8_args(A, As, B, Bs, dev(off), R, moe.MOE_EPI_NONE, D))
    cols = torch.tensor([0, 1, 127, 128, 65535, 65536, N - 17, N - 1], device="cuda")
    for e, (lo, hi) in enumerate(zip(off[:-1], off[1:])):
        w = _value(B[e][cols], Bs[e][cols // 128])
        a = _value(A[lo:hi], As[lo:hi])
        y, mag = a @ w.T, a.abs() @ w.abs().T
        assert ((D[lo:hi][:, cols].double() - y).abs() <= U16 * y.abs() + (1 + U16) * ref.core_error(K) * mag).all(), e


@pytest.mark.parametrize("K", [144, 528])
def test_results_past_32_bits(K):
    """D of 4.6 GB: rows behind 2^31 and 2^32 bytes, in the middle and in the large tile."""
    R, N = 140000, 16400
    g = _gen(2)
    A = moe.quantize_fp8_alloc(torch.randn(R, K, generator=g, device="cuda").bfloat16())
    W = moe.quantize_fp8_weights_alloc(torch.randn(2, N, K, generator=g, device="cuda").bfloat16())
    off = torch.tensor([0, 60001, R], dtype=torch.int32, device="cuda")
    D = moe.grouped_gemm_fp8_alloc(A, W, off, R)
    rows = torch.tensor([0, 60000, 60001, (1 << 31) // (2 * N), (1 << 32) // (2 * N), (1 << 32) // (2 * N) + 1, R - 1], device="cuda")
    for p in rows.tolist():
        e = int(p >= 60001)
        w = torch.from_numpy(ref.e4m3_values()).cuda()[W.q[e].long()] * W.sf[e].double().repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)[:, :K]
        a = _value(A.q[p:p + 1], A.sf[p:p + 1])
        y, mag = a @ w.T, a.abs() @ w.abs().T
        assert ((D[p:p + 1].double() - y).abs() <= U16 * y.abs() + (1 + U16) * ref.core_error(K) * mag).all(), p


def test_quantisers_past_32_bits():
    """4.9 GB of codes from each row and token quantiser."""
    rows, C = 300000, 16384
    x = torch.empty(rows, C, dtype=torch.bfloat16, device="cuda")
    g = _gen(3)
    for r in range(0, rows, 50000):
        x[r:r + 50000] = torch.randn(50000, C, generator=g, device="cuda", dtype=torch.bfloat16)
    q = moe.quantize_fp8_alloc(x)
    at = torch.tensor([0, (1 << 31) // C, (1 << 32) // C - 1, (1 << 32) // C, rows - 1], device="cuda")
    wq, ws = ref.quantize_rows(x[at].float().cpu().numpy())
    assert np.array_equal(q.q[at].cpu().numpy(), wq) and np.array_equal(q.sf[at].cpu().numpy(), ws)
    del q
    off = torch.tensor([0, 100, rows - 5, rows], dtype=torch.int32, device="cuda")
    t = moe.quantize_fp8_tokens_alloc(x, off, rows)
    starts = np.concatenate([[0], 100 + 128 * np.arange(-(-(rows - 105) // 128)), [rows - 5]])
    for b in (0, 1, (1 << 32) // (C * 128), (1 << 32) // (C * 128) + 1, len(starts) - 2, len(starts) - 1):
        lo = int(starts[b])
        hi = min(lo + 128, 100 if b == 0 else rows - 5 if b < len(starts) - 1 else rows)
        cols = [0, 129, C - 1]
        wq, ws = ref.quantize_tokens(x[lo:hi][:, cols].float().cpu().numpy(), [0, hi - lo])
        assert np.array_equal(t.q[b, cols].cpu().numpy(), wq[0]) and np.array_equal(t.sf[b, cols].cpu().numpy(), ws[0]), b


def test_weight_gradient_past_32_bits():
    """dW of 5.4 GB, and token blocks of 0.7 GB."""
    E, N, K = 40, 8192, 4096
    g = _gen(4)
    sizes = [130] * 20 + [0, 7] * 10
    off = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
    R = int(off[-1])
    dy, x = torch.randn(R, N, generator=g, device="cuda").bfloat16(), torch.randn(R, K, generator=g, device="cuda").bfloat16()
    o = dev(off)
    Y, X = moe.quantize_fp8_tokens_alloc(dy, o, R), moe.quantize_fp8_tokens_alloc(x, o, R)
    D = moe.grouped_wgrad_fp8_alloc(Y, X, o, R)
    blocks = np.concatenate([[0], np.cumsum([-(-s // 128) for s in sizes])])
    v = torch.from_numpy(ref.e4m3_values()).cuda()
    for e in (0, 15, 16, 19, 31, 38, 39):
        b = slice(int(blocks[e]), int(blocks[e + 1]))
        y, w = v[Y.q[b][:, :64].long()] * Y.sf[b][:, :64, None].double(), v[X.q[b][:, -64:].long()] * X.sf[b][:, -64:, None].double()
        want = torch.zeros(64, 64, dtype=torch.double, device="cuda")
        mag = torch.zeros_like(want)
        for i in range(y.shape[0]):
            want += y[i] @ w[i].T
            mag += y[i].abs() @ w[i].abs().T
        got = D[e, :64, -64:].double()
        assert ((got - want).abs() <= U32 * want.abs() + (1 + U32) * ref.sum_error(max(sizes)) * mag).all(), e

"""The bf16 expert products, clipping and single-token products at the ends of what they take: the widest and the
longest sizes, the most tokens and slots, tensors beyond 2^32 elements.  Whole numbers, so results are exact."""
from __future__ import annotations

import math

import pytest
import torch

import block_scaled_fp4_02_amd as moe
from tests import experts_ref as ref
from tests.test_gpu_bf16_experts import BF16, MARK, _gen, _ints, _offsets
from tests.test_gpu_gemv import _exact_weights, _ids, _layouts

pytestmark = pytest.mark.gpu
MOST = 1 << 20


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    moe.lib()
    yield
    torch.cuda.synchronize()


@pytest.mark.parametrize("sizes", [[3], [40, 0, 90]], ids=["few rows", "groups"])
@pytest.mark.parametrize("N, K", [(MOST, 8), (8, MOST)], ids=["widest", "longest"])
def test_products(N, K, sizes):
    g, off, R = _gen(K + len(sizes)), _offsets(sizes), sum(sizes)
    A, W, Y = _ints(g, R, K, most=1), _ints(g, len(sizes), N, K, most=1), _ints(g, R, N, most=1)
    want = ref.bf16(ref.product(A, W, off)[0])   # below 2^20: exact in binary32
    for layout, B in ((0, W), (moe.MOE_LAYOUT_TRANSPOSED, W.transpose(1, 2).contiguous())):
        assert torch.equal(moe.grouped_gemm_bf16_alloc(A, B, off, R, transposed=bool(layout)).double(), want)
    assert torch.equal(moe.grouped_wgrad_bf16_alloc(Y, A, off, R).double(), ref.wgrad(Y, A, off)[0])


def test_widest_gated_block():
    g, off, R = _gen(3), _offsets([5, 0, 70]), 75
    A, W = _ints(g, R, 8, scale=0.25), _ints(g, 3, MOST, 8, scale=0.25)
    act, z = moe.gated_ffn_alloc(A, W, off, R)
    y, _ = ref.product(A, W, off)
    assert torch.equal(z.double(), ref.bf16(y)) and ref.close(act, ref.swiglu(y), ref.swiglu_error(y))
    W2 = _ints(g, 3, 8, MOST // 2, scale=0.25)
    dz = moe.gated_ffn_backward_alloc(A, W2, z, off, R)
    da, _ = ref.product(A, W2.transpose(1, 2), off)
    want, err = ref.swiglu_backward(da, z.double())
    assert ref.close(dz, want, err)


def test_most_rows():
    """500 million rows of 8: offsets of rows, tiles and results beyond 2^32 bytes."""
    R = (1 << 29) - 4096
    A = torch.zeros(R, 8, dtype=BF16, device="cuda")
    off, g = _offsets([R - 300, 300]), _gen(5)
    A[-400:] = _ints(g, 400, 8)
    W = _ints(g, 2, 8, 8)
    D = torch.full((R, 8), MARK, dtype=BF16, device="cuda")
    moe.moe_grouped_gemm_bf16(moe.make_gemm_bf16_args(A, W, off, R, moe.MOE_EPI_NONE, D))
    want = torch.cat([A[-400:-300].double() @ W[0].double().T, A[-300:].double() @ W[1].double().T])
    assert torch.equal(D[-400:].double(), ref.bf16(want)) and not D[:-400].any()


@pytest.mark.parametrize("dtype", [torch.float32, BF16], ids=["f32", "bf16"])
def test_clipping_beyond_32_bits(dtype):
    n = (1 << 32) + 12345
    big, small = torch.zeros(n, dtype=dtype, device="cuda"), torch.full((7,), 2.0, dtype=dtype, device="cuda")
    big[0], big[1 << 31], big[-1] = 4.0, -8.0, 16.0
    norm = moe.clip_grad_norm([big, small], 1.0)
    assert norm.item() == pytest.approx(math.sqrt(16 + 64 + 256 + 28), rel=2.0 ** -24)
    s = torch.tensor(1.0, device="cuda") / (norm + 1e-6)
    for i, v in ((0, 4.0), (1 << 31, -8.0), (n - 1, 16.0)):
        assert torch.equal(big[i:i + 1], (v * s).to(dtype)), i
        big[i] = 0
    assert not big.any() and torch.equal(small, (2.0 * s).to(dtype).expand(7))


@pytest.mark.parametrize("N, K", [(MOST, 32), (16, MOST), (32, MOST - 32)], ids=["widest", "longest", "longest, odd"])
@pytest.mark.parametrize("T", [1, 5])
def test_single_token_products(T, N, K):
    g = _gen(N + T)
    W = _exact_weights(g, 2, N, K)
    x, ids = _ints(g, T, K, most=1), _ids(g, T, 2, 2, "any")
    want = ref.bf16(ref.gemv(x, ref.nvfp4_values(W.q, W.sf, W.gs), ids)[0])   # (random signs: sums far below 2^24 halves)
    for B in _layouts(W):
        assert torch.equal(moe.gemv_nvfp4_alloc(x, B, ids).double(), want)


@pytest.mark.parametrize("T, k, E, how", [(16, 32, 40, "any"), (16, 32, 3, "any"), (25, 32, 33, "distinct"), (4096, 2, 6, "any")])
def test_most_slots_and_tokens(T, k, E, how):
    """512 pairs in a workgroup; every token naming few experts many times; 256 workgroups of tokens."""
    g = _gen(T + E)
    N, K = 48, 256
    W = _exact_weights(g, E, N, K)
    x, ids = _ints(g, T, K), _ids(g, T, k, E, how)
    values = ref.nvfp4_values(W.q, W.sf, W.gs)
    y, _ = ref.gemv(x, values, ids)
    w = torch.randint(0, 3, (T, k), generator=g, device="cuda").float()
    summed = (y.view(T, k, N) * w.double()[..., None]).sum(1)   # quarters below 2^20: exact
    for B in _layouts(W):
        assert torch.equal(moe.gemv_nvfp4_alloc(x, B, ids).double(), ref.bf16(y))
        assert torch.equal(moe.gemv_nvfp4_alloc(x, B, ids, w, moe.MOE_EPI_FINALIZE).double(), ref.bf16(summed))

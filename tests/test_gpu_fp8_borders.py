"""The FP8 quantisers bit for bit on elements next to E4M3's rounding borders, in blocks whose scales
lie around the smallest one that the fast quotient serves (2^-92) and below."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import block_scaled_fp4_02_amd as moe
from tests import fp8_ref as ref
from tests.fp8_ref import dev

pytestmark = pytest.mark.gpu

# (block maximum, element): the quotient by the block's scale is a tie, and the fast form misses it
TIES = [("0x1.500004p-89", "0x1.380004p-104"), ("0x1.880008p-91", "0x1.340006p-106"), ("0x1.500008p-91", "0x1.500008p-107"),
        ("0x1.c00036p-92", "0x1.80002cp-109"), ("0x1.bffff2p-91", "0x1.1ffff8p-106"), ("0x1.c0000cp-91", "0x1.800008p-108"),
        ("0x1.c00016p-91", "0x1.c00014p-107"), ("0x1.c00044p-92", "0x1.800038p-109")]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    moe.lib()
    yield
    torch.cuda.synchronize()


def _blocks():
    """Blocks [n, 128]: the maximum first, then ties of TIES or elements on and next to borders."""
    rng = np.random.default_rng(17)
    borders = (ref._POS[:-1] + ref._POS[1:]) / 2
    out = []
    for amax, a in TIES:
        out.append(np.full(128, float.fromhex(a), np.float32))
        out[-1][0] = float.fromhex(amax)
    for e in np.repeat(np.arange(-104, -84), 16):
        s = np.float32(rng.uniform(1, 2) * 2.0 ** e)
        v = (borders[rng.integers(0, np.where(rng.random(128) < 0.7, 8, 126))] * np.float64(s)).astype(np.float32)
        v = (v.view(np.int32) + rng.integers(-2, 3, 128).astype(np.int32)).view(np.float32)
        v[0] = np.float32(s * np.float64(448))
        out.append(v)
    x = np.stack(out)
    return x * rng.choice([-1, 1], x.shape).astype(np.float32)


def _equal(got, want):
    wrong = int((got.cpu().numpy() != want).sum())
    assert wrong == 0, f"{wrong} of {want.size}"


def test_rows():
    x = _blocks()
    q, s = ref.quantize_rows(x)
    got = moe.quantize_fp8_alloc(dev(x))
    _equal(got.sf, s)
    _equal(got.q, q)


def test_tokens():
    x = _blocks()
    q, s = ref.quantize_rows(x)
    n = x.shape[0]
    cols = np.zeros((128, -(-n // 16) * 16), np.float32)      # a block down each column
    cols[:, :n] = x.T
    got = moe.quantize_fp8_tokens_alloc(dev(cols), dev(np.array([0, 128], np.int32)), 128)
    _equal(got.sf[0, :n], s[:, 0])
    _equal(got.q[0, :n], q)


def test_weights():
    """One block's elements as a 16 x 16 tile beside its zeros."""
    x = _blocks()
    w = np.zeros((x.shape[0], 16, 16), np.float32)
    w.reshape(x.shape[0], 256)[:, :128] = x
    q, s = ref.quantize_weights(w)
    got, t = moe.quantize_fp8_weights_alloc(dev(w), True)
    _equal(got.sf, s)
    _equal(t.sf, s)
    _equal(got.q, q)
    _equal(t.q, q.transpose(0, 2, 1))

"""The global gradient norm and its clipping on the GPU: the norm against binary64, the clipped values
bit for bit (one binary32 product and one rounding each), over counts, sizes, types and alignments."""
from __future__ import annotations

import math

import numpy as np
import pytest
import torch

import block_scaled_fp4_02_amd as moe

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    moe.lib()
    yield
    torch.cuda.synchronize()


def _tensors(sizes, seed, scale=1.0, types=(F32, BF16)):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return [(scale * torch.randn(n, generator=g, device="cuda")).to(types[i % len(types)]) for i, n in enumerate(sizes)]


def _norm(ts):
    return math.sqrt(math.fsum(float(t.double().square().sum()) for t in ts))


def _scale(norm, most):
    """As the kernel takes it: every step one binary32 operation."""
    with np.errstate(all="ignore"):
        s = np.float32(most) / (np.float32(norm) + np.float32(1e-6))
    return np.float32(1.0) if s >= 1 or most == math.inf else s


def _check(ts, most, norm, out):
    want = _norm(ts)
    # binary64 sums of up to 2^30 squares are good to 2^-40; the root is rounded to binary32 once
    assert abs(float(norm) - want) <= 2.0 ** -24 * want * 1.001
    s = torch.tensor(_scale(norm.item(), most), device="cuda")
    for t, o in zip(ts, out):
        assert torch.equal(o, (t.float() * s).to(t.dtype))


SIZES = {"one": [1], "none": [], "empty ones": [0, 5, 0, 0, 3], "odd": [1, 7, 8, 9, 15, 16383, 16384, 16385, 3], "all empty": [0, 0],
         "table edge": [5] * 320, "past the table": [3, 40000] * 160 + [1], "three tables": [3, 0, 9] * 300, "large": [3_000_001, 70_000_000]}


@pytest.mark.parametrize("most", [0.5, 1e6, 0.0, math.inf])
@pytest.mark.parametrize("name", SIZES)
def test_norm_and_clip(name, most):
    ts = _tensors(SIZES[name], len(name))
    keep = [t.clone() for t in ts]
    out = [torch.full_like(t, 9.0) for t in ts]
    norm = moe.clip_grad_norm(ts, most, out=out)
    _check(keep, most, norm, out)
    assert all(torch.equal(a, b) for a, b in zip(ts, keep))
    assert torch.equal(moe.clip_grad_norm(ts, most), norm)      # in place
    assert all(torch.equal(a, b) for a, b in zip(ts, out))


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_views_at_any_element(dtype):
    """Tensors that start between 16-byte borders, and whose outputs lie at other ones."""
    base = _tensors([200000], 3, types=(dtype,))[0]
    room = torch.full((210000,), 9.0, dtype=dtype, device="cuda")
    cuts = [(0, 1000), (1001, 1001 + 16387), (20003, 20010), (30000, 99999), (100008, 199999)]
    ts = [base[a:b] for a, b in cuts]
    out = [room[a + 3:b + 3] for a, b in cuts]
    norm = moe.clip_grad_norm(ts, 2.0, out=out)
    _check(ts, 2.0, norm, out)
    touched = torch.zeros_like(room, dtype=torch.bool)
    for a, b in cuts:
        touched[a + 3:b + 3] = True
    assert (room[~touched] == 9.0).all()


@pytest.mark.parametrize("scale", [1e25, 1e-30], ids=["squares overflow", "squares underflow"])
def test_extreme_values(scale):
    ts = _tensors([5000, 37], 4, scale)
    keep = [t.clone() for t in ts]
    norm = moe.clip_grad_norm(ts, 1.0)
    _check(keep, 1.0, norm, ts)


def test_infinities_and_nan():
    for bad in (math.inf, -math.inf, math.nan):
        ts = _tensors([100, 4000], 5)
        ts[1][77] = bad
        out = [torch.empty_like(t) for t in ts]
        norm = moe.clip_grad_norm(ts, 1.0, out=out)
        if math.isnan(bad):
            assert norm.isnan() and all(o.isnan().all() for o in out)
        else:   # 1 / inf = 0: finite values vanish, the infinity becomes NaN
            assert norm.item() == math.inf and not out[0].any() and out[1][77].isnan() and out[1].isnan().sum() == 1
        clipped = moe.clip_grad_norm(ts, math.inf, out=out)
        assert torch.equal(clipped, norm) or clipped.isnan()
        assert all(torch.equal(a.nan_to_num(7.0), b.nan_to_num(7.0)) for a, b in zip(out, ts))


def test_lists_serve_again_and_repeat():
    ts = _tensors([1000, 33, 50000], 6)
    gl = moe.GradList(ts, [torch.empty_like(t) for t in ts])
    a = moe.clip_grad_norm(gl, 1.0)
    first = [o.clone() for o in gl.out]
    ts[0].mul_(2)
    b = moe.clip_grad_norm(gl, 1.0)
    assert b.item() > a.item()
    _check(ts, 1.0, b, gl.out)
    ts[0].mul_(0.5)
    assert torch.equal(moe.clip_grad_norm(gl, 1.0), a) and all(torch.equal(x, y) for x, y in zip(first, gl.out))
    ws = torch.empty(moe.moe_grad_norm_workspace(gl), dtype=torch.uint8, device="cuda")
    norm = torch.empty(1, device="cuda")
    moe.moe_grad_norm(gl, norm, ws)
    assert torch.equal(norm, a)


def test_streams_and_replayed_graphs():
    ts = _tensors([40000, 17, 5000] * 40, 7)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out = [torch.empty_like(t) for t in ts]
    norm = moe.clip_grad_norm(ts, 1.0, out=out, stream=s)
    torch.cuda.synchronize()
    _check(ts, 1.0, norm, out)
    graphs = []
    for most in (1.0, 3.0):      # two graphs at a time, each with memory of its own
        o = [torch.empty_like(t) for t in ts]
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            n = moe.clip_grad_norm(ts, most, out=o)
        graphs.append((g, n, o, most))
    for i in range(4):
        for t in ts:
            t.mul_(1.25)
        want = [moe.clip_grad_norm(ts, most, out=out).clone() for _, _, _, most in graphs]
        torch.cuda.synchronize()
        for g, _, _, _ in graphs:
            g.replay()
        torch.cuda.synchronize()
        for (g, n, o, most), w in zip(graphs, want):
            assert torch.equal(n, w)
            _check(ts, most, n, o)

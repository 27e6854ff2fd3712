"""What clipping writes has to lie apart from everything else of its list: the check of address ranges
against the pairwise definition, and the binding's refusals, on tensors of the host (nothing is launched)."""
from __future__ import annotations

import ctypes as C
import random

import pytest
import torch

import block_scaled_fp4_02_amd as moe


def _apart(src, dst, nbytes):
    """Each written range against each other one, but a src that it replaces."""
    for i, (d, n) in enumerate(zip(dst, nbytes)):
        for j, m in enumerate(nbytes):
            meets = lambda a: n > 0 and m > 0 and d < a + m and a < d + n  # noqa: E731
            if (j != i and meets(dst[j])) or (meets(src[j]) and not (j == i and src[j] == d)):
                return False
    return True


def test_ranges_against_the_definition():
    r, L = random.Random(5), moe.lib()
    seen = {True: 0, False: 0}
    for _ in range(20000):
        n, room = r.randint(0, 5), r.choice([12, 40, 200])
        place = lambda: 0x10000 + 4 * r.randint(0, room)  # noqa: E731
        src, size, types = [place() for _ in range(n)], [r.choice([0, 1, 2, 4, 8]) for _ in range(n)], [r.randint(0, 1) for _ in range(n)]
        dst = [s if r.random() < p else place() for p in [r.choice([0.0, 0.5, 1.0])] for s in src]
        want = _apart(src, dst, [a * (4 if t else 2) for a, t in zip(size, types)])
        items = (moe.moe_tensor * max(n, 1))(*[moe.moe_tensor(s, None if s == d and r.random() < 0.5 else d, a, t) for s, d, a, t in zip(src, dst, size, types)])
        scratch = (C.c_uint64 * (4 * n + 1))(*[0] * 4 * n, 77)
        got = L.moe_grad_clip_can_implement(items, n, scratch)
        assert got == (moe.MOE_OK if want else moe.MOE_ERR_UNSUPPORTED) and scratch[4 * n] == 77, (src, dst, size, types)
        seen[want] += n > 1
    assert min(seen.values()) > 2000


def test_the_check_refuses_what_clipping_does():
    L = moe.lib()
    one, scratch = lambda **kw: (moe.moe_tensor * 1)(moe.moe_tensor(**(dict(src=0x1000, n=4, dtype=1) | kw))), (C.c_uint64 * 4)()  # noqa: E731
    assert L.moe_grad_clip_can_implement(one(), 1, scratch) == moe.MOE_OK == L.moe_grad_clip_can_implement(None, 0, None)
    assert L.moe_grad_clip_can_implement(one(), 1, None) == L.moe_grad_clip_can_implement(None, 1, scratch) == moe.MOE_ERR_NULL
    assert L.moe_grad_clip_can_implement(one(n=-1), 1, scratch) == L.moe_grad_clip_can_implement(one(), -1, scratch) == moe.MOE_ERR_SHAPE
    assert L.moe_grad_clip_can_implement(one(dtype=2), 1, scratch) == L.moe_grad_clip_can_implement(one(src=0x1002), 1, scratch) == moe.MOE_ERR_UNSUPPORTED


def _views():
    a = torch.zeros(64)
    b = torch.zeros(64, dtype=torch.bfloat16)
    h = b.view(torch.int16).view(torch.float32)
    return {
        "outputs are each other's tensors": ([a[:8], a[8:16]], [a[8:16], a[:8]], False),
        "an output is the next tensor": ([a[:8], a[8:16]], [a[8:16], a[16:24]], False),
        "an output reaches into the next tensor": ([a[:8], a[8:16]], [a[1:9], a[24:32]], False),
        "an output reaches into its own tensor": ([a[:8]], [a[4:12]], False),
        "outputs overlap": ([a[:8], a[8:16]], [a[16:24], a[20:28]], False),
        "an output elsewhere, another its tensor": ([a[:32], a[32:34]], [torch.zeros(32), a[32:34]], True),
        "one inside the other": ([a[:32], a[8:10]], None, False),
        "in place, overlapping": ([a[:8], a[4:12]], None, False),
        "in place, of two types": ([b[:8], h[3:5]], None, False),
        "in place, side by side": ([a[:8], a[8:16], b[:8], h[4:6]], None, True),
        "side by side, in another order": ([a[8:16], a[:8], a[16:17]], None, True),
        "outputs are the tensors": ([a[:8], a[8:16]], [a[:8], a[8:16]], True),
        "one output is its tensor": ([a[:8], a[8:16]], [a[:8], a[16:24]], True),
        "only read twice": ([a[:8], a[4:12], a[:8]], [a[16:24], a[24:32], a[32:40]], True),
        "empty ones anywhere": ([a[4:4], a[:8], a[4:4]], [a[20:20], a[16:24], a[20:20]], True),
    }


@pytest.mark.parametrize("name", _views())
def test_views(name):
    tensors, out, good = _views()[name]
    g = moe.GradList(tensors, out)
    assert g.distinct == good
    if not good:
        for call in (lambda: moe.moe_grad_clip(tensors, torch.zeros(1), 1.0, out=out), lambda: moe.moe_grad_clip(g, torch.zeros(1), 1.0)):
            with pytest.raises(moe.MoeError) as e:
                call()
            assert e.value.status == moe.MOE_ERR_UNSUPPORTED and "overlap" in str(e.value)

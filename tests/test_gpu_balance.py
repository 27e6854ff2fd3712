"""The balance loss, its counts and its gradient on the GPU against a plain 64-bit
implementation, over expert counts, sequences, masks and values where they can go wrong."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import block_scaled_fp4_02_amd as moe
from tests import fp8_ref as ref
from tests.fp8_ref import U32, dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    moe.lib()
    yield
    torch.cuda.synchronize()


def _run(z, ids, off, mask, grad, routed, w=None, dw=None):
    d = lambda a: None if a is None else dev(a)
    o = None if off is None else dev(np.asarray(off, np.int32))
    loss, counts, coef = moe.balance_loss_alloc(d(z), d(ids), o, d(mask))
    dl = torch.full(z.shape, 9.0, device="cuda")
    moe.moe_balance_loss_backward(d(z), coef, d(np.array([grad], np.float32)), dl, o, d(mask), d(ids) if routed else None,
                                  d(w), d(dw))
    return loss, counts, coef, dl


def _check(z, ids, off, mask, grad=1.5, routed=False, seed=0):
    rng = np.random.default_rng(seed)
    T, E = z.shape
    k = ids.shape[1]
    w = dw = None
    if routed:
        with np.errstate(invalid="ignore"):
            w = ref.softmax(np.take_along_axis(z, np.clip(ids, 0, E - 1), 1).astype(np.float64)).astype(np.float32)
        dw = rng.standard_normal((T, k)).astype(np.float32)
    bounds = [0, T] if off is None else list(off)
    S = len(bounds) - 1
    loss, counts, coef, dl = _run(z, ids, off, mask, grad, routed, w, dw)
    wl, wc, wf, p = ref.balance(z, ids, bounds, mask)
    assert np.array_equal(counts.cpu().numpy(), wc)
    assert np.abs(coef.cpu().numpy() - wf).max(initial=0) <= 2 * U32 * wf.max(initial=0)
    # sums of probabilities: 8 tokens a wave and 4 waves in binary32, then binary64
    err = ref.softmax_error(z, mask) + 2 * 12 * U32
    assert abs(loss.item() - wl) <= (err + 4 * U32) * abs(wl)
    d, mag = ref.balance_grad(p, bounds, wf, np.float64(np.float32(grad)), mask, ids if routed else None, w, dw)
    inside = ~np.isnan(d)
    got = dl.cpu().numpy()
    # p twice, coef, grad, the dot product over 16 terms a lane and 6 levels, the difference, the
    # product; the routed part: three products, a sum over 6 levels, up to 32 additions
    bound = mag * (2 * err + 2 * (2 + 22 + 4 + 32) * U32)
    # probabilities below the smallest normal number may be flushed to zero
    bound += U32 * np.nan_to_num(np.abs(d)) + 2.0 ** -126 * 4 * np.abs(wf).max(initial=0) * grad
    bad = inside & ~(np.abs(got - d) <= bound)
    assert not bad.any(), [(i, got[tuple(i)], d[tuple(i)], bound[tuple(i)]) for i in np.argwhere(bad)[:5]]
    rows = np.zeros(T, bool)
    for lo, hi in zip(bounds, bounds[1:]):
        rows[lo:hi] = True
    assert (got[~rows] == 9.0).all()
    if mask is not None:
        assert (got[rows & (mask == 0)] == 0).all()
    again = _run(z, ids, off, mask, grad, routed, w, dw)
    for a, b in zip((loss, counts, coef, dl), again):
        assert torch.equal(a.view(torch.int32), b.view(torch.int32))


def _inputs(T, E, k, seed=0):
    rng = np.random.default_rng(seed)
    z = (2 * rng.standard_normal((T, E))).astype(np.float32)
    return z, np.argsort(-z, 1, kind="stable")[:, :k].astype(np.int32)


@pytest.mark.parametrize("T, E, k", [(1, 1, 1), (1, 4, 2), (7, 3, 3), (33, 64, 8), (64, 65, 1), (100, 128, 6), (257, 160, 6),
                                     (1000, 256, 8), (130, 513, 32), (65, 1000, 4), (40, 1024, 8)])
@pytest.mark.parametrize("routed", [False, True])
def test_one_sequence(T, E, k, routed):
    z, ids = _inputs(T, E, k, T + E)
    _check(z, ids, None, None, routed=routed)


@pytest.mark.parametrize("off", [[0, 100], [0, 0, 40, 40, 41, 100], [0] + [100] * 3, [5, 31, 64, 64, 90], list(range(101)),
                                 [0, 32, 64, 96, 100]])
@pytest.mark.parametrize("masked", [0.0, 0.3, 1.0])
def test_sequences_and_masks(off, masked):
    z, ids = _inputs(100, 40, 4, len(off))
    mask = None
    if masked:
        mask = (np.random.default_rng(1).random(100) >= masked).astype(np.uint8)
        if masked < 1:
            mask[mask != 0] = 7     # any non-zero entry keeps
        z[mask == 0] = np.nan
        ids[mask == 0] = 12345
    _check(z, ids, off, mask, routed=masked != 1.0)


def test_many_sequences():
    """More sequences than one round of the lookup covers, most of them empty or short."""
    rng = np.random.default_rng(2)
    sizes = rng.integers(0, 4, 700) * (rng.random(700) < 0.5)
    sizes[650] = 90
    off = np.concatenate([[0], np.cumsum(sizes)])
    z, ids = _inputs(int(off[-1]) + 5, 24, 2, 3)
    _check(z, ids, off, None)


def test_infinities_and_dropped_slots():
    z, ids = _inputs(50, 48, 4, 4)
    z[3, ids[3, 1:]] = -np.inf
    z[7, 1:] = -np.inf                # one expert left
    z[9] = -np.inf                    # none: no probability, the slots still count
    ids[5, 2], ids[6, 0], ids[8] = -1, 48, -7
    ids[11] = ids[11, 0]              # the same expert in every slot
    z[12] = 3.0                       # all equal
    z[13] *= 30                       # far apart
    _check(z, ids, [0, 20, 50], None)


def test_lowest_finite_values():
    z, ids = _inputs(20, 70, 2, 8)
    low = np.finfo(np.float32).min
    z[:, 10:] = low                   # experts masked by the type's lowest value
    ids[:] = [3, 9]
    d = ref.softmax(z.astype(np.float64))
    loss, counts, coef, dl = _run(z, ids, None, None, 1.0, False)
    assert np.isfinite(loss.item()) and torch.isfinite(dl).all() and (dl[:, 10:] == 0).all() and (d[:, 10:] == 0).all()
    z[:] = low                        # every expert: an even row
    loss, *_ = _run(z, ids, None, None, 1.0, False)
    assert abs(loss.item() - 1.0) <= 64 * U32


def test_nan_in_a_kept_row_is_not_hidden():
    z, ids = _inputs(40, 32, 2, 9)
    z[4, 5] = np.nan
    loss, counts, coef, dl = _run(z, ids, [0, 10, 40], None, 1.0, False)
    assert np.isnan(loss.item()) and torch.isnan(dl[4]).all() and not torch.isnan(dl[:4]).any() and not torch.isnan(dl[5:]).any()


def test_no_tokens():
    z, ids = np.empty((0, 16), np.float32), np.empty((0, 2), np.int32)
    for off in (None, [0, 0, 0]):
        loss, counts, coef, dl = _run(z, ids, off, None, 1.0, False)
        assert loss.item() == 0 and (counts == 0).all() and (coef == 0).all()


def test_balanced_router_is_one_and_counts_are_the_routing():
    """Equal logits and an even choice give 1; with moe_route_permute's choice the counts are its
    group sizes."""
    T, E, k = 64, 32, 4
    ids = (np.arange(T)[:, None] * k + np.arange(k)).astype(np.int32) % E
    loss, counts, _, dl = _run(np.zeros((T, E), np.float32), ids, None, None, 1.0, False)
    assert abs(loss.item() - 1) <= 8 * U32 and (counts == T * k // E).all() and dl.abs().max().item() <= 64 * U32 / T
    z, _ = _inputs(300, 96, 6, 5)
    ids, w, off, *_ = moe.route_permute_alloc(dev(z), 6)
    _, counts, _ = moe.balance_loss_alloc(dev(z), ids)
    assert torch.equal(counts[0], off[1:] - off[:-1])


def test_gradient_matches_differences():
    """dlogits against differences of the loss with the counts held, in binary64."""
    T, E, k = 24, 12, 3
    z, ids = _inputs(T, E, k, 6)
    off, mask = [0, 9, 24], (np.arange(T) % 5 != 2).astype(np.uint8)
    _, _, coef, dl = _run(z, ids, off, mask, 2.0, False)
    c = coef.double().cpu().numpy()[[0] * 9 + [1] * 15] * mask[:, None]
    f = lambda v: 2.0 * (c * ref.softmax(v)).sum()
    h = 1e-5
    for t in range(T):
        for e in range(E):
            up, dn = z.astype(np.float64), z.astype(np.float64)
            up[t, e] += h
            dn[t, e] -= h
            # the difference is off by h^2 of the third derivative (at most 6 max c) and by
            # binary64 rounding of the loss over h
            assert abs((f(up) - f(dn)) / (2 * h) - dl[t, e].item()) <= 12 * c.max() * (h * h + 200 * U32) + 1e-15 * f(z) / h


@pytest.mark.parametrize("T, E, k, S", [(4096, 1024, 8, 4), (9000, 96, 4, 1), (8200, 40, 2, 70), (2050, 300, 8, 2)])
def test_sizes_behind_every_variant(T, E, k, S):
    """Tokens per wave and the shape of the second kernel follow T, E and S."""
    rng = np.random.default_rng(T)
    z, ids = _inputs(T, E, k, T)
    cuts = np.sort(rng.integers(0, T + 1, S - 1))
    mask = (rng.random(T) < 0.8).astype(np.uint8)
    _check(z, ids, None if S == 1 else [0, *cuts, T], mask, routed=True)


def test_bool_mask_and_views():
    """A bool mask, and logits that start inside a buffer (4-byte alignment is enough)."""
    z, ids = _inputs(50, 33, 3, 11)
    mask = np.arange(50) % 4 != 1
    want = _run(z, ids, None, mask.astype(np.uint8), 1.0, False)
    buf = torch.empty(50 * 33 + 1, device="cuda")
    buf[1:] = dev(z).flatten()
    logits = buf[1:].view(50, 33)
    assert logits.data_ptr() % 16 == 4
    loss, counts, coef = moe.balance_loss_alloc(logits, dev(ids), token_mask=dev(mask))
    dl = torch.empty_like(logits)
    moe.moe_balance_loss_backward(logits, coef, torch.ones(1, device="cuda"), dl, token_mask=dev(mask))
    for a, b in zip((loss, counts, coef, dl), want):
        assert torch.equal(a.view(torch.int32), b.view(torch.int32))


def test_offsets_that_are_not_monotone_stay_in_range():
    """2^16 sequences that claim all tokens in turn: 2^31 chunks and more, past what 32 bits hold.  The
    values mean nothing, rows in front of and behind the tensors stay."""
    T, E, S = 1 << 19, 1, 1 << 16
    off = torch.zeros(S + 1, dtype=torch.int32, device="cuda")
    off[1::2] = T
    pad = 1 << 12
    buf = torch.full((T + 2 * pad,), 7.0, device="cuda")
    dl = buf[pad:pad + T].view(T, E)
    z = torch.zeros(T, E, device="cuda")
    loss, counts, coef = moe.balance_loss_alloc(z, torch.zeros(T, 1, dtype=torch.int32, device="cuda"), off)
    moe.moe_balance_loss_backward(z, coef, torch.ones(1, device="cuda"), dl, off)
    assert (buf[:pad] == 7).all() and (buf[pad + T:] == 7).all()
    # and the same call with good offsets afterwards
    good = torch.linspace(0, T, S + 1, device="cuda").round().int()
    loss, counts, coef = moe.balance_loss_alloc(z, torch.zeros(T, 1, dtype=torch.int32, device="cuda"), good)
    assert abs(loss.item() - 1) <= 64 * U32 and (counts.flatten() == good.diff()).all()

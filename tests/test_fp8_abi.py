"""The FP8 and balance-loss entry points on the CPU: every refusal returns its documented status
before any HIP call, the binding refuses tensors that the kernels could not read, the
argument structures agree with the header, and the 64-bit reference used by the GPU tests is
itself pinned to independent results."""
import ctypes as C
import os
import shutil
import subprocess

import numpy as np
import pytest
import torch

import block_scaled_fp4_02_amd as moe
from tests import fp8_ref as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = C.c_void_p(0x1000)   # never dereferenced: validation fails first
OK, NULL, SHAPE, UNSUPPORTED, WS = (moe.MOE_OK, moe.MOE_ERR_NULL, moe.MOE_ERR_SHAPE, moe.MOE_ERR_UNSUPPORTED,
                                    moe.MOE_ERR_WORKSPACE)


@pytest.mark.parametrize("kw, want", [
    (dict(rows=-1), SHAPE), (dict(C=8), SHAPE), (dict(C=24), SHAPE), (dict(C=0), SHAPE),
    (dict(dtype=2), UNSUPPORTED), (dict(C=(1 << 20) + 16), UNSUPPORTED), (dict(rows=1 << 40), UNSUPPORTED),
    (dict(rows=(1 << 63) - 1), UNSUPPORTED), (dict(x=None), NULL), (dict(q=None), NULL), (dict(sf=None), NULL)])
def test_quantize_rows_refusals(kw, want):
    a = dict(x=FAKE, dtype=0, rows=4, C=32, q=FAKE, sf=FAKE) | kw
    assert moe.lib().moe_quantize_fp8(a["x"], a["dtype"], a["rows"], a["C"], a["q"], a["sf"], None) == want


@pytest.mark.parametrize("kw, want", [
    (dict(E=0), SHAPE), (dict(E=1025), SHAPE), (dict(N=0), SHAPE), (dict(K=-16), SHAPE), (dict(N=20), UNSUPPORTED),
    (dict(K=24), UNSUPPORTED), (dict(dtype=7), UNSUPPORTED), (dict(N=1 << 21), UNSUPPORTED),
    (dict(E=1024, N=1 << 20, K=1 << 20), UNSUPPORTED), (dict(w=None), NULL), (dict(q=None), NULL), (dict(sf=None), NULL),
    (dict(qt=FAKE), NULL), (dict(sft=FAKE), NULL)])
def test_quantize_weights_refusals(kw, want):
    a = dict(w=FAKE, dtype=1, E=2, N=32, K=32, q=FAKE, sf=FAKE, qt=None, sft=None) | kw
    assert moe.lib().moe_quantize_fp8_weights(a["w"], a["dtype"], a["E"], a["N"], a["K"], a["q"], a["sf"], a["qt"], a["sft"],
                                              None) == want


@pytest.mark.parametrize("kw, want", [
    (dict(E=0), SHAPE), (dict(E=1025), SHAPE), (dict(R=-1), SHAPE), (dict(R=1 << 31), SHAPE), (dict(C=40), SHAPE),
    (dict(rows_x=-1), SHAPE), (dict(rows_x=0), SHAPE), (dict(rows=None, rows_x=7), SHAPE), (dict(dtype=-1), UNSUPPORTED),
    (dict(C=1 << 21), UNSUPPORTED), (dict(R=(1 << 31) - 1, C=1 << 20), UNSUPPORTED), (dict(x=None), NULL), (dict(off=None), NULL),
    (dict(q=None), NULL), (dict(sf=None), NULL)])
def test_quantize_tokens_refusals(kw, want):
    a = dict(x=FAKE, dtype=0, rows_x=8, rows=FAKE, off=FAKE, E=2, R=8, C=32, q=FAKE, sf=FAKE) | kw
    assert moe.lib().moe_quantize_fp8_tokens(a["x"], a["dtype"], a["rows_x"], a["rows"], a["off"], a["E"], a["R"], a["C"], a["q"],
                                             a["sf"], None) == want


def test_token_blocks():
    b = moe.moe_fp8_token_blocks
    assert [b(0, 4), b(1, 4), b(3, 4), b(4, 4), b(128, 1), b(129, 1), b(1000, 4)] == [0, 1, 3, 4, 2, 2, 11]
    assert b(-1, 4) == b(5, 0) == b(5, 1025) == b(1 << 31, 4) == 0
    rng = np.random.default_rng(3)
    for _ in range(200):   # never fewer than a partition of R rows into E groups can need
        E = int(rng.integers(1, 40))
        sizes = rng.integers(0, 300, E) * (rng.random(E) < 0.7)
        assert b(int(sizes.sum()), E) >= sum(-(-int(n) // 128) for n in sizes)


def gemm_args(**kw):
    a = moe.moe_gemm_fp8_args()
    v = dict(A=FAKE, A_sf=FAKE, A_rows=None, rows_A=256, B=FAKE, B_sf=FAKE, expert_offsets=FAKE, E=8, N=512, K=2064, epilogue=0, R=256,
             D=FAKE, D_sf=FAKE) | kw
    for f, x in v.items():
        setattr(a, f, x)
    return a


@pytest.mark.parametrize("kw, want", [
    ({}, OK), (dict(epilogue=3), OK), (dict(D_sf=None), OK), (dict(R=0, rows_A=0, A=None, A_sf=None, D=None), OK),
    (dict(E=0), SHAPE), (dict(E=1025), SHAPE), (dict(N=0), SHAPE), (dict(K=0), SHAPE), (dict(R=-1), SHAPE), (dict(R=1 << 31), SHAPE),
    (dict(rows_A=-1), SHAPE), (dict(rows_A=0, A_rows=FAKE), SHAPE), (dict(rows_A=255), SHAPE), (dict(N=520), UNSUPPORTED),
    (dict(K=24), UNSUPPORTED), (dict(N=1 << 21), UNSUPPORTED), (dict(N=1 << 16, K=1 << 15), UNSUPPORTED),
    (dict(epilogue=1), UNSUPPORTED), (dict(epilogue=2), UNSUPPORTED), (dict(epilogue=-1), UNSUPPORTED),
    (dict(epilogue=3, N=384), UNSUPPORTED), (dict(epilogue=3, N=528), UNSUPPORTED),
    (dict(A_rows=FAKE, rows_A=1 << 31), UNSUPPORTED), (dict(A_rows=FAKE, rows_A=(1 << 63) - 1), UNSUPPORTED),
    (dict(R=(1 << 31) - 1, rows_A=1 << 40, N=1 << 15), UNSUPPORTED),
    (dict(A=None), NULL), (dict(A_sf=None), NULL), (dict(B=None), NULL), (dict(B_sf=None), NULL), (dict(expert_offsets=None), NULL),
    (dict(D=None), NULL), (dict(epilogue=3, D_sf=None), NULL)])
def test_gemm_refusals(kw, want):
    L = moe.lib()
    a = gemm_args(**kw)
    assert L.moe_grouped_gemm_fp8_can_implement(C.byref(a)) == want
    if want != OK:
        assert L.moe_grouped_gemm_fp8(C.byref(a), None) == want
    assert L.moe_grouped_gemm_fp8_can_implement(None) == L.moe_grouped_gemm_fp8(None, None) == NULL


@pytest.mark.parametrize("kw, want", [
    ({}, OK), (dict(D_dtype=0), OK), (dict(R=0, Y=None, Y_sf=None, X=None, X_sf=None), OK), (dict(E=0), SHAPE), (dict(N=-16), SHAPE),
    (dict(R=-1), SHAPE), (dict(N=8), UNSUPPORTED), (dict(K=40), UNSUPPORTED), (dict(D_dtype=5), UNSUPPORTED),
    (dict(N=1 << 16, K=1 << 16), UNSUPPORTED), (dict(Y=None), NULL), (dict(Y_sf=None), NULL), (dict(X=None), NULL),
    (dict(X_sf=None), NULL), (dict(expert_offsets=None), NULL), (dict(D=None), NULL), (dict(R=0, D=None), NULL)])
def test_wgrad_refusals(kw, want):
    L = moe.lib()
    a = moe.moe_wgrad_fp8_args()
    for f, x in (dict(Y=FAKE, Y_sf=FAKE, X=FAKE, X_sf=FAKE, expert_offsets=FAKE, E=3, N=48, K=80, D_dtype=1, R=300, D=FAKE) | kw).items():
        setattr(a, f, x)
    assert L.moe_grouped_wgrad_fp8_can_implement(C.byref(a)) == want
    if want != OK:
        assert L.moe_grouped_wgrad_fp8(C.byref(a), None) == want
    assert L.moe_grouped_wgrad_fp8_can_implement(None) == NULL


@pytest.mark.parametrize("kw, want", [
    (dict(T=-1), SHAPE), (dict(E=0), SHAPE), (dict(E=1025), SHAPE), (dict(k=0), SHAPE), (dict(k=33, E=64), SHAPE), (dict(k=5), SHAPE),
    (dict(S=0), SHAPE), (dict(S=65537), SHAPE), (dict(T=(1 << 31) - 1, k=2), SHAPE), (dict(off=None, S=2), NULL), (dict(logits=None), NULL),
    (dict(ids=None), NULL), (dict(counts=None), NULL), (dict(coef=None), NULL), (dict(loss=None), NULL), (dict(ws=None), WS),
    (dict(ws_bytes=-1), WS)])
def test_balance_refusals(kw, want):
    L = moe.lib()
    a = dict(logits=FAKE, ids=FAKE, T=100, E=4, k=2, off=FAKE, S=3, counts=FAKE, coef=FAKE, loss=FAKE, ws=FAKE, ws_bytes=0) | kw
    need = L.moe_balance_loss_workspace(a["T"], a["E"], a["k"], a["S"])
    assert (need == 0) == (want == SHAPE)
    assert L.moe_balance_loss(a["logits"], a["ids"], a["T"], a["E"], a["k"], a["off"], a["S"], None, a["counts"], a["coef"],
                              a["loss"], a["ws"], need + a["ws_bytes"], None) == want


@pytest.mark.parametrize("kw, want", [
    (dict(T=-1), SHAPE), (dict(E=1025), SHAPE), (dict(S=0), SHAPE), (dict(dw=FAKE, k=0), SHAPE), (dict(dw=FAKE, k=5), SHAPE),
    (dict(off=None, S=2), NULL), (dict(logits=None), NULL), (dict(coef=None), NULL), (dict(grad=None), NULL), (dict(dlogits=None), NULL),
    (dict(dw=FAKE, ids=None), NULL), (dict(dw=FAKE, w=None), NULL)])
def test_balance_backward_refusals(kw, want):
    a = dict(logits=FAKE, T=100, E=4, off=FAKE, S=3, coef=FAKE, grad=FAKE, ids=FAKE, w=FAKE, dw=None, k=2, dlogits=FAKE) | kw
    assert moe.lib().moe_balance_loss_backward(a["logits"], a["T"], a["E"], a["off"], a["S"], None, a["coef"], a["grad"], a["ids"],
                                               a["w"], a["dw"], a["k"], a["dlogits"], None) == want


def test_most_rows():
    """Row numbers and the rows past a tile's end stay in 31 bits, and a launch has fewer than 2^32
    threads: more rows are refused before the launch."""
    L = moe.lib()
    for R, want in ((1 << 30, OK), ((1 << 30) + 1, UNSUPPORTED), ((1 << 31) - 1, UNSUPPORTED)):
        w = moe.moe_wgrad_fp8_args()
        for f, x in dict(Y=FAKE, Y_sf=FAKE, X=FAKE, X_sf=FAKE, expert_offsets=FAKE, E=3, N=48, K=80, D_dtype=1, R=R, D=FAKE).items():
            setattr(w, f, x)
        assert L.moe_grouped_wgrad_fp8_can_implement(C.byref(w)) == want
        # (a null pointer stands for a call that would be launched)
        assert L.moe_quantize_fp8_tokens(None, 0, R, None, FAKE, 2, R, 16, FAKE, FAKE, None) == (want or NULL)
    for R, N, want in (((1 << 30) - 2048, 16, OK), (1 << 30, 16, UNSUPPORTED), ((1 << 24) - 2048, 8192, OK), (1 << 24, 8192, UNSUPPORTED)):
        g = gemm_args(R=R, rows_A=1 << 31, N=N, K=16)
        assert L.moe_grouped_gemm_fp8_can_implement(C.byref(g)) == want
    for rows, C_, want in (((1 << 28) - 1, 16, NULL), (1 << 28, 16, UNSUPPORTED), (1 << 24, 2048, UNSUPPORTED)):
        assert L.moe_quantize_fp8(None, 0, rows, C_, FAKE, FAKE, None) == want
    for T, want in ((1 << 26, NULL), ((1 << 26) + 1, SHAPE)):
        assert (L.moe_balance_loss_workspace(T, 4, 1, 1) != 0) == (want == NULL)
        assert L.moe_balance_loss_backward(None, T, 4, None, 1, None, FAKE, FAKE, None, None, None, 1, FAKE, None) == want


def test_balance_workspace_alignment():
    """The workspace holds binary64 partial sums behind its first 16 bytes."""
    L = moe.lib()
    need = L.moe_balance_loss_workspace(100, 4, 2, 3)
    call = lambda ws: L.moe_balance_loss(FAKE, FAKE, 100, 4, 2, FAKE, 3, None, FAKE, FAKE, FAKE, C.c_void_p(ws), need, None)
    assert call(0x1004) == call(0x1008) == WS


def test_binding_refuses_what_kernels_cannot_read():
    """Wrong dtypes, strides, sizes, unaligned views and host tensors are refused before any launch."""
    bf, f32, u8, i32 = torch.bfloat16, torch.float32, torch.uint8, torch.int32
    z = lambda *s, dt=f32: torch.zeros(*s, dtype=dt)
    refused = lambda status, f, *a, **k: pytest.raises(moe.MoeError, f, *a, **k).value.status == status
    x, q, sf = z(4, 32, dt=bf), z(4, 32, dt=u8), z(4, 1)
    assert refused(UNSUPPORTED, moe.moe_quantize_fp8, x, q, sf)                      # not on the GPU
    assert refused(UNSUPPORTED, moe.moe_quantize_fp8, x.half(), q, sf)
    assert refused(UNSUPPORTED, moe.moe_quantize_fp8, z(32, 4, dt=bf).T, q, sf)       # strided
    assert refused(UNSUPPORTED, moe.moe_quantize_fp8, z(4 * 32 + 1, dt=bf)[1:].view(4, 32), q, sf)   # unaligned
    assert refused(SHAPE, moe.moe_quantize_fp8, x, q[:3], sf)
    assert refused(SHAPE, moe.moe_quantize_fp8, x, q, z(4, 2))
    w = z(2, 32, 48, dt=bf)
    assert refused(SHAPE, moe.moe_quantize_fp8_weights, w, z(2, 32, 48, dt=u8), z(2, 2, 1))
    assert refused(SHAPE, moe.moe_quantize_fp8_weights, w, z(2, 32, 48, dt=u8), z(2, 1, 1), z(2, 48, 16, dt=u8), z(2, 1, 1))
    off = z(3, dt=i32)
    assert refused(SHAPE, moe.moe_quantize_fp8_tokens, x, off, 4, z(1, 32, 128, dt=u8), z(2, 32))
    assert refused(UNSUPPORTED, moe.moe_quantize_fp8_tokens, x, off.long(), 4, z(2, 32, 128, dt=u8), z(2, 32))
    g = dict(A=q, A_sf=sf, B=z(2, 48, 32, dt=u8), B_sf=z(2, 1, 1), expert_offsets=off, R=4, epilogue=moe.MOE_EPI_NONE, D=z(4, 48, dt=bf))
    for bad in (dict(A=z(4, 48, dt=u8)), dict(A_sf=z(4, 2)), dict(B_sf=z(1, 1, 1)), dict(expert_offsets=z(4, dt=i32)), dict(D=z(3, 48, dt=bf)),
                dict(A_rows=z(3, dt=i32))):
        assert refused(SHAPE, moe.make_gemm_fp8_args, **(g | bad)), bad
    assert refused(UNSUPPORTED, moe.make_gemm_fp8_args, **(g | dict(D=z(4, 48))))
    assert refused(UNSUPPORTED, moe.make_gemm_fp8_args, **g)
    wg = dict(Y=z(2, 48, 128, dt=u8), Y_sf=z(2, 48), X=z(2, 32, 128, dt=u8), X_sf=z(2, 32), expert_offsets=off, R=4, D=z(2, 48, 32))
    for bad in (dict(Y=z(1, 48, 128, dt=u8)), dict(X_sf=z(1, 32)), dict(D=z(3, 48, 32))):
        assert refused(SHAPE, moe.make_wgrad_fp8_args, **(wg | bad)), bad
    b = dict(logits=z(6, 4), topk_ids=z(6, 2, dt=i32), counts=z(1, 4, dt=i32), coef=z(1, 4), loss=z(1))
    for bad in (dict(topk_ids=z(5, 2, dt=i32)), dict(counts=z(2, 4, dt=i32)), dict(seq_offsets=z(3, dt=i32)), dict(token_mask=z(5, dt=u8))):
        assert refused(SHAPE, moe.moe_balance_loss, **(b | bad)), bad
    assert refused(UNSUPPORTED, moe.moe_balance_loss, **(b | dict(logits=z(6, 4, dt=bf))))
    assert refused(UNSUPPORTED, moe.moe_balance_loss, **b)
    d = dict(logits=z(6, 4), coef=z(1, 4), grad_loss=z(1), dlogits=z(6, 4))
    for bad in (dict(dlogits=z(6, 5)), dict(d_topk_w=z(6, 2)), dict(d_topk_w=z(6, 2), topk_ids=z(6, 2, dt=i32), topk_w=z(6, 3))):
        assert refused(SHAPE, moe.moe_balance_loss_backward, **(d | bad)), bad


def test_structures_match_the_header(tmp_path):
    gcc = shutil.which("gcc")
    if gcc is None:
        pytest.skip("no gcc")
    src = ["#include <stdio.h>", "#include <stddef.h>", '#include "moe_nvfp4.h"', "int main(void) {",
           '  printf("epi %d\\n", (int)MOE_EPI_SWIGLU_FP8);']
    for t in ("moe_gemm_fp8_args", "moe_wgrad_fp8_args"):
        src.append(f'  printf("{t} size %zu\\n", sizeof({t}));')
        src += [f'  printf("{t} {f} %zu\\n", offsetof({t}, {f}));' for f, _ in getattr(moe, t)._fields_]
    (tmp_path / "s.c").write_text("\n".join(src + ["  return 0;", "}"]) + "\n")
    subprocess.run([gcc, "-std=c11", "-Wall", "-Wextra", "-Werror", "-D__HIP_PLATFORM_AMD__", "-I", os.path.join(ROOT, "include"),
                    "-I", "/opt/rocm/include", str(tmp_path / "s.c"), "-o", str(tmp_path / "s")], check=True)
    out = subprocess.run([str(tmp_path / "s")], check=True, capture_output=True, text=True).stdout.split("\n")
    got = dict(ln.rsplit(" ", 1) for ln in out if ln)
    assert int(got["epi"]) == moe.MOE_EPI_SWIGLU_FP8
    for t in ("moe_gemm_fp8_args", "moe_wgrad_fp8_args"):
        cls = getattr(moe, t)
        assert int(got[f"{t} size"]) == C.sizeof(cls)
        for f, _ in cls._fields_:
            assert int(got[f"{t} {f}"]) == getattr(cls, f).offset, (t, f)


# ---- the reference ----------------------------------------------------------------------------

def test_reference_e4m3_matches_torch():
    codes = np.arange(256, dtype=np.uint8)
    t = torch.from_numpy(codes.copy()).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(ref.values(codes), t, equal_nan=True)
    rng = np.random.default_rng(0)
    u = np.concatenate([rng.uniform(-448, 448, 20000), rng.standard_normal(20000) * 2.0 ** rng.integers(-12, 8, 20000),
                        (ref._POS[:-1] + ref._POS[1:]) / 2, -ref._POS, [0.0, -0.0, 448, -448]]).astype(np.float32)
    u = np.clip(u, -448, 448)
    assert np.array_equal(ref.e4m3_codes(u.astype(np.float64)), torch.from_numpy(u).to(torch.float8_e4m3fn).view(torch.uint8).numpy())


def test_reference_products_and_gradients():
    """The products on unquantised values against einsum, and the balance gradient against
    differences of the loss."""
    rng = np.random.default_rng(1)
    off = [0, 3, 3, 10]
    a, w = rng.standard_normal((10, 32)), rng.standard_normal((3, 16, 32))
    e = np.repeat(np.arange(3), np.diff(off))
    y, _ = ref.product(a, w, off)
    assert np.allclose(y, np.einsum("pk,pnk->pn", a, w[e]))
    T, E, k = 9, 7, 2
    z = rng.standard_normal((T, E))
    ids = np.argsort(-z, 1)[:, :k]
    mask = np.array([1, 1, 0, 1, 1, 1, 1, 0, 1])
    seq = [0, 4, 4, 9]
    loss, counts, coef, p = ref.balance(z, ids, seq, mask)
    assert counts.sum() == k * mask.sum()
    rw = lambda z: np.stack([np.exp(z[t, ids[t]]) / np.exp(z[t, ids[t]]).sum() for t in range(T)])
    w_, dw = rw(z), rng.standard_normal((T, k)) * mask[:, None]
    d, _ = ref.balance_grad(p, seq, coef, 1.7, mask, ids, w_, dw)
    h = 1e-6
    for t in range(T):
        for j in range(E):
            zp, zm = z.copy(), z.copy()
            zp[t, j] += h
            zm[t, j] -= h
            f = lambda v: 1.7 * (coef[[0] * 4 + [2] * 5] * mask[:, None] * ref.softmax(v)).sum() + (rw(v) * dw).sum()
            assert abs((f(zp) - f(zm)) / (2 * h) - d[t, j]) < 1e-7, (t, j)


def test_binding_refuses_another_device_and_wrong_layer_shapes():
    g = gemm_args()
    g.device = -1
    w = moe.moe_wgrad_fp8_args()
    w.device = -1
    for call, a in ((moe.moe_grouped_gemm_fp8, g), (moe.moe_grouped_wgrad_fp8, w)):
        with pytest.raises(moe.MoeError) as e:
            call(a)
        assert e.value.status == UNSUPPORTED
    E, H, I = 2, 256, 128
    z = lambda *s: moe.FP8Tensor(torch.zeros(*s, dtype=torch.uint8), torch.zeros(s[0], -(-s[1] // 128), -(-s[2] // 128)))
    for w1, w2 in ((z(E, I, H), z(E, H, I)), (z(E, 2 * I, H), z(E, I, I)), (z(E + 1, 2 * I, H), z(E, H, I))):
        with pytest.raises(moe.MoeError) as e:
            moe.MoEFP8LayerPlan(4, E, 1, H, I, w1, w2, device="cpu")
        assert e.value.status == SHAPE
    ws = torch.zeros(1 << 12)   # not bytes
    with pytest.raises(moe.MoeError) as e:
        moe.moe_balance_loss(torch.zeros(4, 8), torch.zeros(4, 2, dtype=torch.int32), torch.zeros(1, 8, dtype=torch.int32),
                             torch.zeros(1, 8), torch.zeros(1), ws=ws)
    assert e.value.status == UNSUPPORTED


def test_binding_takes_codes_in_their_own_type():
    """float8_e4m3fn beside uint8 (a wrong size is found behind the type); other 8-bit floats are refused."""
    bf, u8, f8, i32 = torch.bfloat16, torch.uint8, torch.float8_e4m3fn, torch.int32
    z = lambda *s, dt=torch.float32: torch.zeros(*s, dtype=torch.uint8 if dt.itemsize == 1 else dt).view(dt)
    refused = lambda status, f, *a, **k: pytest.raises(moe.MoeError, f, *a, **k).value.status == status
    x, w, off = z(4, 32, dt=bf), z(2, 32, 48, dt=bf), z(3, dt=i32)
    act = moe.MOE_EPI_SWIGLU_FP8
    calls = [lambda t: (moe.moe_quantize_fp8, x, z(3, 32, dt=t), z(4, 1)),
             lambda t: (moe.moe_quantize_fp8_weights, w, z(2, 32, 48, dt=t), z(2, 1, 1), z(2, 48, 16, dt=t), z(2, 1, 1)),
             lambda t: (moe.moe_quantize_fp8_tokens, x, off, 4, z(1, 32, 128, dt=t), z(2, 32)),
             lambda t: (moe.make_gemm_fp8_args, z(4, 48, dt=t), z(4, 1), z(2, 256, 32, dt=t), z(2, 2, 1), off, 4, act, z(4, 128, dt=t), z(4, 1)),
             lambda t: (moe.make_wgrad_fp8_args, z(1, 48, 128, dt=t), z(2, 48), z(2, 32, 128, dt=t), z(2, 32), off, 4, z(2, 48, 32))]
    for call in calls:
        assert refused(SHAPE, *call(u8)) and refused(SHAPE, *call(f8))
        assert refused(UNSUPPORTED, *call(torch.float8_e4m3fnuz)) and refused(UNSUPPORTED, *call(torch.float8_e5m2))


def test_binding_refuses_other_numbers_of_dimensions():
    """topk_ids [T, k, 2] and A [rows, K, 2] would be read as if their last axis were not there."""
    bf, u8, i32 = torch.bfloat16, torch.uint8, torch.int32
    z = lambda *s, dt=torch.float32: torch.zeros(*s, dtype=dt)
    off = z(3, dt=i32)
    g = dict(A=z(4, 32, dt=u8), A_sf=z(4, 1), B=z(2, 48, 32, dt=u8), B_sf=z(2, 1, 1), expert_offsets=off, R=4, epilogue=moe.MOE_EPI_NONE)
    b = dict(logits=z(6, 4), topk_ids=z(6, 2, dt=i32), counts=z(1, 4, dt=i32), coef=z(1, 4), loss=z(1))
    d = dict(logits=z(6, 4), coef=z(1, 4), grad_loss=z(1), dlogits=z(6, 4))
    wg = dict(Y=z(2, 48, 128, dt=u8), Y_sf=z(2, 48), X=z(2, 32, 128, dt=u8), X_sf=z(2, 32), expert_offsets=off, R=4, D=z(2, 48, 32))
    for f, kw in ((moe.make_gemm_fp8_args, g | dict(A=z(4, 32, 2, dt=u8))), (moe.make_gemm_fp8_args, g | dict(A=z(128, dt=u8))),
                  (moe.make_gemm_fp8_args, g | dict(B=z(96, 32, dt=u8))), (moe.make_wgrad_fp8_args, wg | dict(D=z(2, 48 * 32))),
                  (moe.moe_balance_loss, b | dict(topk_ids=z(6, 2, 2, dt=i32))), (moe.moe_balance_loss, b | dict(topk_ids=z(6, dt=i32))),
                  (moe.moe_balance_loss, b | dict(logits=z(2, 3, 4))), (moe.moe_balance_loss_backward, d | dict(logits=z(24))),
                  (moe.moe_balance_loss_backward, d | dict(d_topk_w=z(6))),
                  (moe.moe_quantize_fp8, dict(x=z(2, 2, 32, dt=bf), q=z(4, 32, dt=u8), sf=z(4, 1))),
                  (moe.moe_quantize_fp8_weights, dict(w=z(32, 48, dt=bf), q=z(32, 48, dt=u8), sf=z(1, 1))),
                  (moe.moe_quantize_fp8_tokens, dict(x=z(128, dt=bf), expert_offsets=off, R=4, q=z(2, 32, 128, dt=u8), sf=z(2, 32)))):
        with pytest.raises(moe.MoeError) as e:
            f(**kw)
        assert e.value.status == SHAPE, f.__name__


def test_whole_sums_are_asked_for_with_the_epilogue(tmp_path):
    L = moe.lib()
    whole = moe.MOE_SUMS_WHOLE
    for epi, want in ((whole, OK), (whole | moe.MOE_EPI_SWIGLU_FP8, OK), (whole | 1, UNSUPPORTED), (whole | 2, UNSUPPORTED),
                      (2 * whole, UNSUPPORTED), (whole >> 1, UNSUPPORTED), (-whole, UNSUPPORTED), (-1 - whole, UNSUPPORTED)):
        a = gemm_args(epilogue=epi)
        assert L.moe_grouped_gemm_fp8_can_implement(C.byref(a)) == want, epi
        if want != OK:
            assert L.moe_grouped_gemm_fp8(C.byref(a), None) == want
    assert L.moe_grouped_gemm_fp8_can_implement(C.byref(gemm_args(epilogue=whole | 3, D_sf=None))) == NULL
    assert L.moe_grouped_gemm_fp8_can_implement(C.byref(gemm_args(epilogue=whole | 3, N=384))) == UNSUPPORTED
    with open(os.path.join(ROOT, "include", "moe_nvfp4.h")) as f:
        assert f"MOE_SUMS_WHOLE = 0x{whole:x} " in f.read()


def test_layer_refuses_tensors_of_another_device_before_its_first_launch():
    """The routing call checks no device, so the plan has to before it."""
    plan = object.__new__(moe.MoEFP8LayerPlan)
    plan.T, plan.E, plan.k, plan.H, plan.I = 4, 2, 1, 256, 128
    plan.out = torch.zeros(4, 256, dtype=torch.bfloat16)
    with pytest.raises(moe.MoeError) as e:
        plan.forward(torch.zeros(4, 2), torch.zeros(4, 256, dtype=torch.bfloat16))
    assert e.value.status == UNSUPPORTED

"""The bf16 expert products, the gradient clipping and the single-token products on the CPU: every
refusal returns its documented status before any HIP call, the binding refuses tensors that the kernels
could not read, the argument structures agree with the header, and the 64-bit references that the GPU
tests use are held to differences and to independent results."""
import ctypes as C
import os
import shutil
import subprocess

import pytest
import torch

import block_scaled_fp4_02_amd as moe
from tests import experts_ref as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = C.c_void_p(0x1000)   # never dereferenced: validation fails first
OK, NULL, SHAPE, UNSUPPORTED, WS = (moe.MOE_OK, moe.MOE_ERR_NULL, moe.MOE_ERR_SHAPE, moe.MOE_ERR_UNSUPPORTED,
                                    moe.MOE_ERR_WORKSPACE)
BACK = dict(epilogue=moe.MOE_EPI_SWIGLU_BACKWARD, B_layout=moe.MOE_LAYOUT_TRANSPOSED)


def filled(cls, **kw):
    a = cls()
    for f, x in kw.items():
        setattr(a, f, x)
    return a


def gemm_args(**kw):
    return filled(moe.moe_gemm_bf16_args, **(dict(A=FAKE, A_rows=None, rows_A=256, B=FAKE, expert_offsets=FAKE, E=8, N=528, K=2056, epilogue=0,
                                                  B_layout=0, R=256, D=FAKE, Z=FAKE) | kw))


@pytest.mark.parametrize("kw, want", [
    ({}, OK), (dict(epilogue=1), OK), (dict(epilogue=1, Z=None), OK), (dict(B_layout=2), OK), (BACK, OK), (BACK | dict(N=8), OK),
    (dict(R=0, rows_A=0, A=None, D=None), OK), (BACK | dict(R=0, rows_A=0, A=None, D=None, Z=None), OK), (dict(N=1 << 15, K=1 << 14), OK),
    (dict(R=(1 << 24) - 8 * 32 - 256, N=128, rows_A=1 << 30), OK),
    (dict(E=0), SHAPE), (dict(E=1025), SHAPE), (dict(N=0), SHAPE), (dict(K=-8), SHAPE), (dict(R=-1), SHAPE), (dict(R=1 << 31), SHAPE),
    (dict(rows_A=-1), SHAPE), (dict(rows_A=0, A_rows=FAKE), SHAPE), (dict(rows_A=255), SHAPE), (dict(N=524), UNSUPPORTED), (dict(K=12), UNSUPPORTED),
    (dict(N=(1 << 20) + 8), UNSUPPORTED), (dict(N=1 << 15, K=1 << 15), UNSUPPORTED), (dict(epilogue=1, N=8), UNSUPPORTED),
    (dict(epilogue=1, B_layout=2), UNSUPPORTED), (BACK | dict(B_layout=0), UNSUPPORTED), (dict(epilogue=2), UNSUPPORTED), (dict(epilogue=3), UNSUPPORTED),
    (dict(epilogue=5), UNSUPPORTED), (dict(epilogue=-1), UNSUPPORTED), (dict(epilogue=0x100), UNSUPPORTED), (dict(B_layout=1), UNSUPPORTED),
    (dict(B_layout=3), UNSUPPORTED), (dict(A_rows=FAKE, rows_A=1 << 20), UNSUPPORTED), (dict(A_rows=FAKE, rows_A=(1 << 63) - 1), UNSUPPORTED),
    (dict(R=(1 << 30) + 1, rows_A=1 << 40), UNSUPPORTED), (dict(R=1 << 30, rows_A=1 << 40, N=1 << 13, K=8), UNSUPPORTED),
    (dict(A=None), NULL), (dict(B=None), NULL), (dict(expert_offsets=None), NULL), (dict(D=None), NULL), (BACK | dict(Z=None), NULL)])
def test_gemm_refusals(kw, want):
    L = moe.lib()
    a = gemm_args(**kw)
    assert L.moe_grouped_gemm_bf16_can_implement(C.byref(a)) == want
    if want != OK:
        assert L.moe_grouped_gemm_bf16(C.byref(a), None) == want
    assert L.moe_grouped_gemm_bf16_can_implement(None) == L.moe_grouped_gemm_bf16(None, None) == NULL


@pytest.mark.parametrize("kw, want", [
    ({}, OK), (dict(D_dtype=0), OK), (dict(X_rows=FAKE, rows_X=7), OK), (dict(R=0, rows_X=0, Y=None, X=None), OK), (dict(E=0), SHAPE),
    (dict(N=-8), SHAPE), (dict(R=-1), SHAPE), (dict(R=1 << 31), SHAPE), (dict(rows_X=-1), SHAPE), (dict(rows_X=299), SHAPE),
    (dict(rows_X=0, X_rows=FAKE), SHAPE), (dict(N=20), UNSUPPORTED), (dict(K=36), UNSUPPORTED), (dict(D_dtype=5), UNSUPPORTED),
    (dict(X_rows=FAKE, rows_X=1 << 27), UNSUPPORTED), (dict(E=1024, N=1 << 16, K=1 << 16), UNSUPPORTED), (dict(R=(1 << 30) + 1, rows_X=1 << 31), UNSUPPORTED),
    (dict(Y=None), NULL), (dict(X=None), NULL), (dict(expert_offsets=None), NULL), (dict(D=None), NULL), (dict(R=0, D=None), NULL)])
def test_wgrad_refusals(kw, want):
    L = moe.lib()
    a = filled(moe.moe_wgrad_bf16_args, **(dict(Y=FAKE, X=FAKE, X_rows=None, rows_X=300, expert_offsets=FAKE, E=3, N=48, K=88, D_dtype=1, R=300, D=FAKE) | kw))
    assert L.moe_grouped_wgrad_bf16_can_implement(C.byref(a)) == want
    if want != OK:
        assert L.moe_grouped_wgrad_bf16(C.byref(a), None) == want
    assert L.moe_grouped_wgrad_bf16_can_implement(None) == L.moe_grouped_wgrad_bf16(None, None) == NULL


@pytest.mark.parametrize("kw, want", [
    ({}, OK), (dict(ids=None, k=1, rows_x=3), OK), (dict(rows_x=12), OK), (dict(epilogue=1), OK), (dict(epilogue=5), OK), (dict(epilogue=5, topk_w=None), OK),
    (dict(B_layout=1, K=512, B_sf=None), OK), (dict(T=0, rows_x=0, x=None, B=None, B_gs=None, D=None), OK), (dict(T=4096, rows_x=4096), OK),
    (dict(T=-1), SHAPE), (dict(T=4097, rows_x=4097), SHAPE), (dict(k=0), SHAPE), (dict(k=33), SHAPE), (dict(E=0), SHAPE), (dict(E=65537), SHAPE),
    (dict(N=0), SHAPE), (dict(K=0), SHAPE), (dict(ids=None), SHAPE), (dict(rows_x=4), SHAPE), (dict(rows_x=0), SHAPE), (dict(rows_x=1 << 40), SHAPE),
    (dict(N=40), UNSUPPORTED), (dict(K=48), UNSUPPORTED), (dict(N=1 << 21), UNSUPPORTED), (dict(K=1 << 21), UNSUPPORTED), (dict(epilogue=1, N=48), UNSUPPORTED),
    (dict(epilogue=2), UNSUPPORTED), (dict(epilogue=3), UNSUPPORTED), (dict(epilogue=4), UNSUPPORTED), (dict(B_layout=2), UNSUPPORTED),
    (dict(B_layout=1, K=544), UNSUPPORTED), (dict(x=None), NULL), (dict(B=None), NULL), (dict(B_sf=None), NULL), (dict(B_gs=None), NULL), (dict(D=None), NULL)])
def test_gemv_refusals(kw, want):
    L = moe.lib()
    a = filled(moe.moe_gemv_args, **(dict(x=FAKE, rows_x=3, B=FAKE, B_sf=FAKE, B_gs=FAKE, ids=FAKE, topk_w=FAKE, T=3, k=4, E=9, N=96, K=544, epilogue=0,
                                          B_layout=0, D=FAKE) | kw))
    assert L.moe_gemv_nvfp4_can_implement(C.byref(a)) == want
    if want != OK:
        assert L.moe_gemv_nvfp4(C.byref(a), None) == want
    assert L.moe_gemv_nvfp4_can_implement(None) == L.moe_gemv_nvfp4(None, None) == NULL


def tensor_list(*items):
    t = (moe.moe_tensor * max(len(items), 1))()
    for i, it in enumerate(items):
        t[i] = it
    return t


GOOD = (0x1000, None, 100, 1)


@pytest.mark.parametrize("items, count, want", [
    ([GOOD], 1, OK), ([], 0, OK), ([(None, None, 0, 0)], 1, OK), ([GOOD, (0x1002, 0x2002, 7, 0)], 2, OK), ([GOOD], -1, SHAPE), ([GOOD], (1 << 20) + 1, SHAPE),
    ([(0x1000, None, -1, 1)], 1, SHAPE), ([(0x1000, None, (1 << 37) + 1, 1)], 1, SHAPE), ([(0x1000, None, 1 << 36, 1)] * 3, 3, SHAPE),
    ([(0x1000, None, 100, 2)], 1, UNSUPPORTED), ([(0x1002, None, 100, 1)], 1, UNSUPPORTED), ([(0x1001, None, 100, 0)], 1, UNSUPPORTED),
    ([(0x1000, 0x1002, 100, 1)], 1, UNSUPPORTED), ([(None, 0x1000, 100, 1)], 1, NULL)])
def test_grad_refusals(items, count, want):
    L, t = moe.lib(), tensor_list(*items)
    need = L.moe_grad_norm_workspace(t, count)
    assert (need > 0) == (want == OK)
    if want == OK:   # (all but the last check)
        assert L.moe_grad_norm(t, count, FAKE, FAKE, need - 1, None) == WS
        assert L.moe_grad_norm(t, count, FAKE, None, need, None) == WS
        assert L.moe_grad_norm(t, count, FAKE, C.c_void_p(0x1008), need, None) == WS
        assert L.moe_grad_norm(t, count, None, FAKE, need, None) == NULL
        assert L.moe_grad_clip(t, count, None, 1.0, None) == NULL
        for bad in (-1.0, float("nan"), -1e-30, float("-inf")):
            assert L.moe_grad_clip(t, count, FAKE, bad, None) == SHAPE
    else:
        assert L.moe_grad_norm(t, count, FAKE, FAKE, 1 << 30, None) == want
        assert L.moe_grad_clip(t, count, FAKE, 1.0, None) == want
    assert L.moe_grad_norm(None, 1, FAKE, FAKE, 1 << 20, None) == L.moe_grad_clip(None, 1, FAKE, 1.0, None) == NULL


def test_binding_refuses_what_kernels_cannot_read():
    """Wrong dtypes, strides, sizes, unaligned views, other numbers of dimensions and host tensors are
    refused before any launch."""
    bf, f32, u8, i32 = torch.bfloat16, torch.float32, torch.uint8, torch.int32
    z = lambda *s, dt=bf: torch.zeros(*s, dtype=dt)  # noqa: E731

    def refused(status, f, **kw):
        with pytest.raises(moe.MoeError) as e:
            f(**kw)
        assert e.value.status == status, (f.__name__, e.value)

    g = dict(A=z(4, 32), B=z(2, 48, 32), expert_offsets=z(3, dt=i32), R=4, epilogue=moe.MOE_EPI_NONE, D=z(4, 48))
    refused(UNSUPPORTED, moe.make_gemm_bf16_args, **g)                                # not on the GPU
    for kw in (dict(A=z(4, 32, dt=f32)), dict(A=z(32, 4).T), dict(A=z(4 * 32 + 1)[1:].view(4, 32)), dict(expert_offsets=z(3, dt=torch.int64)),
               dict(A_rows=z(4, dt=torch.int64)), dict(D=z(4, 48, dt=f32)), dict(Z=z(4, 48, dt=f32))):
        refused(UNSUPPORTED, moe.make_gemm_bf16_args, **(g | kw))
    gated, back = dict(epilogue=moe.MOE_EPI_SWIGLU, D=z(4, 24)), dict(epilogue=moe.MOE_EPI_SWIGLU_BACKWARD, B=z(2, 32, 48), B_layout=moe.MOE_LAYOUT_TRANSPOSED, D=z(4, 96))
    for kw in (dict(A=z(4, 40)), dict(A=z(4, 32, 1)), dict(A=z(128)), dict(B=z(96, 32)), dict(B_layout=moe.MOE_LAYOUT_TRANSPOSED), dict(R=5), dict(D=z(3, 48)),
               dict(expert_offsets=z(4, dt=i32)), dict(A_rows=z(3, dt=i32)), gated | dict(D=z(4, 23)), gated | dict(Z=z(3, 48)), back | dict(D=z(4, 48)),
               back | dict(Z=z(4, 48))):
        refused(SHAPE, moe.make_gemm_bf16_args, **(g | kw))
    w = dict(Y=z(4, 48), X=z(4, 32), expert_offsets=z(3, dt=i32), R=4, D=z(2, 48, 32, dt=f32))
    refused(UNSUPPORTED, moe.make_wgrad_bf16_args, **w)
    for kw in (dict(Y=z(4, 48, dt=f32)), dict(X=z(32, 4).T), dict(D=z(2, 48, 32, dt=torch.double)), dict(X_rows=z(4, dt=torch.int64))):
        refused(UNSUPPORTED, moe.make_wgrad_bf16_args, **(w | kw))
    for kw in (dict(Y=z(3, 48)), dict(Y=z(4, 40)), dict(X=z(4, 40)), dict(D=z(96, 32, dt=f32)), dict(X_rows=z(3, dt=i32)), dict(Y=z(192)), dict(R=5)):
        refused(SHAPE, moe.make_wgrad_bf16_args, **(w | kw))
    nv = lambda E, N, K: moe.NVFP4Tensor(z(E, N, K // 2, dt=u8), z(E, N, K // 16, dt=u8), z(E, dt=f32))  # noqa: E731
    v = dict(x=z(3, 64), B=nv(5, 32, 64), ids=z(3, 2, dt=i32), topk_w=z(3, 2, dt=f32), D=z(6, 32))
    refused(UNSUPPORTED, moe.make_gemv_args, **v)
    for kw in (dict(x=z(3, 64, dt=f32)), dict(x=z(64, 3).T), dict(ids=z(3, 2, dt=torch.int64)), dict(topk_w=z(3, 2)), dict(D=z(6, 32, dt=f32))):
        refused(UNSUPPORTED, moe.make_gemv_args, **(v | kw))
    packed = moe.PackedWeights(z(5, 32 * 256 * 9 // 16, dt=u8), z(5, dt=f32), 32, 256)
    for kw in (dict(x=z(4, 64)), dict(x=z(3, 32)), dict(x=z(192)), dict(ids=z(6, dt=i32)), dict(topk_w=z(3, 1, dt=f32)), dict(D=z(5, 32)),
               dict(D=z(3, 31), epilogue=moe.MOE_EPI_FINALIZE), dict(D=z(6, 15), epilogue=moe.MOE_EPI_SWIGLU), dict(B=packed),
               dict(B=moe.NVFP4Tensor(z(5, 32, 32, dt=u8), z(5, 32, 3, dt=u8), z(5, dt=f32))), dict(B=moe.NVFP4Tensor(z(5, 32, 32, dt=u8), z(5, 32, 4, dt=u8), z(4, dt=f32)))):
        refused(SHAPE, moe.make_gemv_args, **(v | kw))
    for bad in ([z(4, dt=torch.half)], [z(4, 4).T[:, :2]], [z(4), z(4, dt=i32)]):
        refused(UNSUPPORTED, moe.GradList, tensors=bad)
    refused(UNSUPPORTED, moe.GradList, tensors=[z(4)], out=[z(4, dt=f32)])
    refused(SHAPE, moe.GradList, tensors=[z(4)], out=[z(5)])
    refused(SHAPE, moe.GradList, tensors=[z(4)], out=[])
    refused(SHAPE, moe._grad_list, tensors=moe.GradList([z(4)]), out=[z(4)])
    refused(UNSUPPORTED, moe.moe_grad_norm, tensors=[z(4)], norm=z(1, dt=f32))          # not on the GPU
    refused(UNSUPPORTED, moe.moe_grad_clip, tensors=[z(4)], norm=z(1), max_norm=1.0)
    refused(UNSUPPORTED, moe.clip_grad_norm, tensors=[z(4)], max_norm=1.0)
    t, u = z(4), z(4)
    for kw in (dict(tensors=[t, u, t]), dict(tensors=[t, u], out=[z(8)[:4]] * 2), dict(tensors=moe.GradList([u, u]))):   # written twice
        refused(UNSUPPORTED, moe.moe_grad_clip, norm=z(1, dt=f32), max_norm=1.0, **kw)
    assert moe.GradList([t, u, t], [z(4), z(4), z(4)]).distinct and moe.GradList([z(0), t, z(0)]).distinct
    for f, cls in ((moe.moe_grouped_gemm_bf16, gemm_args), (moe.moe_grouped_wgrad_bf16, moe.moe_wgrad_bf16_args), (moe.moe_gemv_nvfp4, moe.moe_gemv_args)):
        a = cls()
        a.device = -1
        refused(UNSUPPORTED, f, args=a)


def test_structures_match_the_header(tmp_path):
    gcc = shutil.which("gcc")
    if gcc is None:
        pytest.skip("no gcc")
    names = ("MOE_EPI_SWIGLU_BACKWARD", "MOE_EPI_FINALIZE", "MOE_LAYOUT_TRANSPOSED")
    src = ["#include <stdio.h>", "#include <stddef.h>", '#include "moe_nvfp4.h"', "int main(void) {"] + [f'  printf("{n} %d\\n", (int){n});' for n in names]
    types = ("moe_gemm_bf16_args", "moe_wgrad_bf16_args", "moe_tensor", "moe_gemv_args")
    for t in types:
        src.append(f'  printf("{t} size %zu\\n", sizeof({t}));')
        src += [f'  printf("{t} {f} %zu\\n", offsetof({t}, {f}));' for f, _ in getattr(moe, t)._fields_]
    (tmp_path / "s.c").write_text("\n".join(src + ["  return 0;", "}"]) + "\n")
    subprocess.run([gcc, "-std=c11", "-Wall", "-Wextra", "-Werror", "-D__HIP_PLATFORM_AMD__", "-I", os.path.join(ROOT, "include"),
                    "-I", "/opt/rocm/include", str(tmp_path / "s.c"), "-o", str(tmp_path / "s")], check=True)
    out = subprocess.run([str(tmp_path / "s")], check=True, capture_output=True, text=True).stdout.split("\n")
    got = dict(ln.rsplit(" ", 1) for ln in out if ln)
    for n in names:
        assert int(got[n]) == getattr(moe, n)
    for t in types:
        cls = getattr(moe, t)
        assert int(got[f"{t} size"]) == C.sizeof(cls)
        for f, _ in cls._fields_:
            assert int(got[f"{t} {f}"]) == getattr(cls, f).offset, (t, f)


def test_reference_gradients_equal_differences():
    """The gradients of the gated block, by the formulas that the kernels use, against central
    differences of its output and against automatic differentiation."""
    g = torch.Generator().manual_seed(5)
    rnd = lambda *s: torch.randn(*s, generator=g, dtype=torch.double)  # noqa: E731
    off, T, K, I, H = [0, 3, 3, 8], 5, 12, 6, 10
    src = torch.randint(0, T, (8,), generator=g)
    x, w1, w2, dy = rnd(T, K), rnd(3, 2 * I, K), rnd(3, H, I), rnd(8, H)

    def block(x, w1, w2):
        z = torch.cat([x[src[lo:hi]] @ w1[e].T for e, lo, hi in ref.groups(off)])
        act = ref.swiglu(z)
        return z, act, torch.cat([act[lo:hi] @ w2[e].T for e, lo, hi in ref.groups(off)])

    z, act, y = block(x, w1, w2)
    dz, _ = ref.swiglu_backward(ref.product(dy, w2.transpose(1, 2), off)[0], z)
    rows = ref.product(dz, w1.transpose(1, 2), off)[0]
    dx = torch.zeros_like(x).index_add_(0, src, rows)
    grads = (dx, ref.wgrad(dz, x, off, src)[0], ref.wgrad(dy, act, off)[0])
    leaves = [t.clone().requires_grad_() for t in (x, w1, w2)]
    (block(*leaves)[2] * dy).sum().backward()
    for got, leaf in zip(grads, leaves):
        assert torch.allclose(got, leaf.grad, rtol=1e-10, atol=1e-12)
    h = 1e-5
    for i, got in enumerate(grads):
        v = rnd(*got.shape)
        moved = [[t + s * h * v if j == i else t for j, t in enumerate((x, w1, w2))] for s in (1, -1)]
        diff = ((block(*moved[0])[2] - block(*moved[1])[2]) * dy).sum() / (2 * h)
        assert abs(diff - (got * v).sum()) <= 1e-7 * (1 + abs(diff))   # h^2 and 2^-52 / h of values of order 10


def test_reference_roundings_and_decoding():
    g = torch.Generator().manual_seed(6)
    v = torch.randn(10000, generator=g, dtype=torch.double) * 2.0 ** torch.randint(-20, 20, (10000,), generator=g)
    ties = (1 + torch.arange(128).double() / 128 + 1 / 256)
    v = torch.cat([v.float().double(), ties, -ties])     # (from binary32 torch rounds to bf16 once)
    assert torch.equal(ref.bf16(v), v.float().bfloat16().double())
    q = torch.arange(256, dtype=torch.uint8).view(1, 2, 128)
    sf = torch.full((1, 2, 16), 0x38, dtype=torch.uint8)   # 1.0
    w = ref.nvfp4_values(q, sf, torch.tensor([2.0]))
    assert w[0, 0, :6].tolist() == [0.0, 0.0, 1.0, 0.0, 2.0, 0.0] and w[0, 1, -1] == -12.0 and w[0, 1, -2] == -12.0
    x = torch.randn(3, 256, generator=g)
    ids = torch.tensor([[0, -1], [0, 0], [1, 0]])
    y, _ = ref.gemv(x, w, ids)
    assert torch.allclose(y[2], w[0] @ x[1].double()) and not y[1].any() and not y[4].any()


def test_layer_plan_refuses_other_shapes():
    E, H, I = 2, 256, 128
    nv = lambda N, K, E=E: moe.NVFP4Tensor(torch.zeros(E, N, K // 2, dtype=torch.uint8), torch.zeros(E, N, K // 16, dtype=torch.uint8), torch.zeros(E))  # noqa: E731
    for w1, w2 in ((nv(2 * I, I), nv(H, I)), (nv(2 * I, H), nv(H, H))):
        with pytest.raises(moe.MoeError) as e:
            moe.MoETokenPlan(4, E, 1, H, I, w1, w2, device="cpu")
        assert e.value.status in (SHAPE, UNSUPPORTED)

"""Python binding of libmoe_nvfp4 (the MI355X NVFP4 MoE hot path).

Argument marshalling only: every function here passes device pointers of torch tensors
and torch's current HIP stream to the C ABI declared in ``include/moe_nvfp4.h`` and
raises :class:`MoeError` on a non-zero status.  Every step of the path runs in the
library's gfx950 kernels; there is no fallback.  If the library has not been built the
import of any entry point fails loudly.

Functions with the C names take caller-allocated tensors exactly like the C calls.  The
``*_alloc`` helpers allocate outputs and workspaces with torch; :func:`pack_weights` turns
an NVFP4 weight tensor into the packed layout once; :class:`MoELayerPlan` pre-allocates one
MoE layer's buffers and sequences its six calls.  The FP8 operators (:func:`moe_quantize_fp8` and its
kin, :func:`moe_grouped_gemm_fp8`, :func:`moe_grouped_wgrad_fp8`, :class:`MoEFP8LayerPlan`) and the
router's balance loss (:func:`moe_balance_loss`) check their tensors (dtype, strides, sizes,
device) before they pass the pointers on, and so do the gated experts in bf16 with their backward pass
(:func:`gated_ffn_alloc`, :func:`gated_ffn_backward_alloc`, :func:`moe_grouped_gemm_bf16`,
:func:`moe_grouped_wgrad_bf16`), the clipping of gradients (:func:`clip_grad_norm`) and the products of
single tokens with NVFP4 weights (:func:`moe_gemv_nvfp4`, :class:`MoETokenPlan`).
"""
from __future__ import annotations

import array
import contextlib
import ctypes as C
import os
from dataclasses import dataclass

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmoe_nvfp4.so")

MOE_OK, MOE_ERR_NULL, MOE_ERR_SHAPE, MOE_ERR_UNSUPPORTED, MOE_ERR_WORKSPACE, MOE_ERR_HIP = range(6)
MOE_DTYPE_BF16, MOE_DTYPE_F32 = 0, 1
MOE_GS_STATIC, MOE_GS_DYNAMIC = 0, 1
MOE_EPI_NONE, MOE_EPI_SWIGLU, MOE_EPI_SWIGLU_NVFP4, MOE_EPI_SWIGLU_FP8 = 0, 1, 2, 3
MOE_EPI_SWIGLU_BACKWARD, MOE_EPI_FINALIZE = 4, 5
MOE_SUMS_WHOLE = 0x100   # with an FP8 product's epilogue
MOE_LAYOUT_ROWMAJOR, MOE_LAYOUT_PACKED, MOE_LAYOUT_TRANSPOSED = 0, 1, 2

EXPORTED = [
    "moe_status_string", "moe_last_hip_error",
    "moe_route_permute_workspace", "moe_route_permute",
    "moe_quantize_nvfp4_workspace", "moe_quantize_nvfp4",
    "moe_grouped_gemm_nvfp4_workspace", "moe_grouped_gemm_nvfp4_amax_slots",
    "moe_grouped_gemm_nvfp4_can_implement", "moe_grouped_gemm_nvfp4", "moe_grouped_gemm_nvfp4_noalloc",
    "moe_pack_weights_nvfp4_bytes", "moe_pack_weights_nvfp4",
    "moe_finalize",
    "moe_quantize_fp8", "moe_quantize_fp8_weights", "moe_fp8_token_blocks", "moe_quantize_fp8_tokens",
    "moe_grouped_gemm_fp8_can_implement", "moe_grouped_gemm_fp8",
    "moe_grouped_wgrad_fp8_can_implement", "moe_grouped_wgrad_fp8",
    "moe_balance_loss_workspace", "moe_balance_loss", "moe_balance_loss_backward",
    "moe_grouped_gemm_bf16_can_implement", "moe_grouped_gemm_bf16",
    "moe_grouped_wgrad_bf16_can_implement", "moe_grouped_wgrad_bf16",
    "moe_grad_norm_workspace", "moe_grad_norm", "moe_grad_clip", "moe_grad_clip_can_implement",
    "moe_gemv_nvfp4_can_implement", "moe_gemv_nvfp4",
]


class MoeError(RuntimeError):
    def __init__(self, fn: str, status: int, msg: str, hip_error: int = 0):
        super().__init__(f"{fn}: status {status} ({msg})" + (f", hipError {hip_error}" if hip_error else ""))
        self.status = status


class moe_gemm_args(C.Structure):
    _fields_ = [
        ("A", C.c_void_p), ("A_sf", C.c_void_p), ("A_gs", C.c_void_p), ("A_rows", C.c_void_p),
        ("rows_A", C.c_int64),
        ("B", C.c_void_p), ("B_sf", C.c_void_p), ("B_gs", C.c_void_p),
        ("expert_offsets", C.c_void_p),
        ("E", C.c_int32), ("N", C.c_int32), ("K", C.c_int32),
        ("R", C.c_int64),
        ("epilogue", C.c_int32),
        ("D", C.c_void_p), ("amax_out", C.c_void_p),
        ("B_layout", C.c_int32),
        ("D_sf", C.c_void_p), ("D_gs", C.c_void_p),
    ]


class moe_gemm_fp8_args(C.Structure):
    _fields_ = [
        ("A", C.c_void_p), ("A_sf", C.c_void_p), ("A_rows", C.c_void_p), ("rows_A", C.c_int64),
        ("B", C.c_void_p), ("B_sf", C.c_void_p), ("expert_offsets", C.c_void_p),
        ("E", C.c_int32), ("N", C.c_int32), ("K", C.c_int32), ("epilogue", C.c_int32),
        ("R", C.c_int64), ("D", C.c_void_p), ("D_sf", C.c_void_p),
    ]


class moe_wgrad_fp8_args(C.Structure):
    _fields_ = [
        ("Y", C.c_void_p), ("Y_sf", C.c_void_p), ("X", C.c_void_p), ("X_sf", C.c_void_p),
        ("expert_offsets", C.c_void_p), ("E", C.c_int32), ("N", C.c_int32), ("K", C.c_int32),
        ("D_dtype", C.c_int32), ("R", C.c_int64), ("D", C.c_void_p),
    ]


class moe_gemm_bf16_args(C.Structure):
    _fields_ = [
        ("A", C.c_void_p), ("A_rows", C.c_void_p), ("rows_A", C.c_int64),
        ("B", C.c_void_p), ("expert_offsets", C.c_void_p),
        ("E", C.c_int32), ("N", C.c_int32), ("K", C.c_int32), ("epilogue", C.c_int32), ("B_layout", C.c_int32),
        ("R", C.c_int64), ("D", C.c_void_p), ("Z", C.c_void_p),
    ]


class moe_wgrad_bf16_args(C.Structure):
    _fields_ = [
        ("Y", C.c_void_p), ("X", C.c_void_p), ("X_rows", C.c_void_p), ("rows_X", C.c_int64),
        ("expert_offsets", C.c_void_p), ("E", C.c_int32), ("N", C.c_int32), ("K", C.c_int32),
        ("D_dtype", C.c_int32), ("R", C.c_int64), ("D", C.c_void_p),
    ]


class moe_tensor(C.Structure):
    _fields_ = [("src", C.c_void_p), ("dst", C.c_void_p), ("n", C.c_int64), ("dtype", C.c_int32)]


class moe_gemv_args(C.Structure):
    _fields_ = [
        ("x", C.c_void_p), ("rows_x", C.c_int64), ("B", C.c_void_p), ("B_sf", C.c_void_p), ("B_gs", C.c_void_p),
        ("ids", C.c_void_p), ("topk_w", C.c_void_p),
        ("T", C.c_int32), ("k", C.c_int32), ("E", C.c_int32), ("N", C.c_int32), ("K", C.c_int32),
        ("epilogue", C.c_int32), ("B_layout", C.c_int32), ("D", C.c_void_p),
    ]


_lib = None


def lib():
    """The loaded C library; raises if it was not built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with __graft_entry__.build() "
                               "(hipcc, gfx950); there is no fallback path")
        L = C.CDLL(LIB_PATH)
        P, i32, i64, sz = C.c_void_p, C.c_int, C.c_int64, C.c_size_t
        args_p = C.POINTER(moe_gemm_args)
        fp8_p, wgrad_p = C.POINTER(moe_gemm_fp8_args), C.POINTER(moe_wgrad_fp8_args)
        bf16_p, bf16_wgrad_p = C.POINTER(moe_gemm_bf16_args), C.POINTER(moe_wgrad_bf16_args)
        gemv_p = C.POINTER(moe_gemv_args)
        sig = {
            "moe_status_string": (C.c_char_p, [i32]),
            "moe_last_hip_error": (i32, []),
            "moe_route_permute_workspace": (sz, [i32, i32, i32]),
            "moe_route_permute": (i32, [P, i32, i32, i32, P, P, P, P, P, P, sz, P]),
            "moe_quantize_nvfp4_workspace": (sz, [i64, i64]),
            "moe_quantize_nvfp4": (i32, [P, i32, i64, i64, P, P, P, i32, P, i64, P, sz, P]),
            "moe_grouped_gemm_nvfp4_workspace": (sz, [args_p]),
            "moe_grouped_gemm_nvfp4_amax_slots": (i64, [args_p]),
            "moe_grouped_gemm_nvfp4_can_implement": (i32, [args_p]),
            "moe_grouped_gemm_nvfp4": (i32, [args_p, P, sz, P]),
            "moe_grouped_gemm_nvfp4_noalloc": (i32, [args_p, P]),
            "moe_pack_weights_nvfp4_bytes": (sz, [i64, i32]),
            "moe_pack_weights_nvfp4": (i32, [P, P, i64, i32, P, P]),
            "moe_finalize": (i32, [P, i64, P, P, i32, i32, i32, P, P]),
            "moe_quantize_fp8": (i32, [P, i32, i64, i64, P, P, P]),
            "moe_quantize_fp8_weights": (i32, [P, i32, i32, i32, i32, P, P, P, P, P]),
            "moe_fp8_token_blocks": (i64, [i64, i32]),
            "moe_quantize_fp8_tokens": (i32, [P, i32, i64, P, P, i32, i64, i64, P, P, P]),
            "moe_grouped_gemm_fp8_can_implement": (i32, [fp8_p]),
            "moe_grouped_gemm_fp8": (i32, [fp8_p, P]),
            "moe_grouped_wgrad_fp8_can_implement": (i32, [wgrad_p]),
            "moe_grouped_wgrad_fp8": (i32, [wgrad_p, P]),
            "moe_balance_loss_workspace": (sz, [i32, i32, i32, i32]),
            "moe_balance_loss": (i32, [P, P, i32, i32, i32, P, i32, P, P, P, P, P, sz, P]),
            "moe_balance_loss_backward": (i32, [P, i32, i32, P, i32, P, P, P, P, P, P, i32, P, P]),
            "moe_grouped_gemm_bf16_can_implement": (i32, [bf16_p]),
            "moe_grouped_gemm_bf16": (i32, [bf16_p, P]),
            "moe_grouped_wgrad_bf16_can_implement": (i32, [bf16_wgrad_p]),
            "moe_grouped_wgrad_bf16": (i32, [bf16_wgrad_p, P]),
            "moe_grad_norm_workspace": (sz, [P, i32]),
            "moe_grad_norm": (i32, [P, i32, P, P, sz, P]),
            "moe_grad_clip": (i32, [P, i32, P, C.c_float, P]),
            "moe_grad_clip_can_implement": (i32, [P, i32, P]),
            "moe_gemv_nvfp4_can_implement": (i32, [gemv_p]),
            "moe_gemv_nvfp4": (i32, [gemv_p, P]),
        }
        for name, (res, argt) in sig.items():
            fn = getattr(L, name)
            fn.restype, fn.argtypes = res, argt
        _lib = L
    return _lib


def _check(fn: str, st: int):
    if st != MOE_OK:
        L = lib()
        raise MoeError(fn, st, L.moe_status_string(st).decode(),
                       L.moe_last_hip_error() if st == MOE_ERR_HIP else 0)


def _p(t):
    return None if t is None else C.c_void_p(t.data_ptr())


def _at(t):
    return None if t is None else t.data_ptr()


def _stream(stream):
    if stream is None:
        # the handle of torch.cuda.current_stream() without the Python object around it (0.3 us
        # instead of 3 us, a third of a small call)
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())
    return stream.cuda_stream


_NO_STREAM = contextlib.nullcontext()


def _allocating(stream):
    """Allocations inside belong to `stream`, the one whose kernels use them (None: the current one)."""
    return _NO_STREAM if stream is None else torch.cuda.stream(stream)


def _ws(nbytes: int, device) -> torch.Tensor:
    return torch.empty(max(int(nbytes), 16), dtype=torch.uint8, device=device)


# ---- the C entry points ------------------------------------------------------------

def moe_route_permute(logits, k, topk_ids, topk_w, expert_offsets, row_src, token_slot_row,
                      ws, stream=None):
    T, E = logits.shape
    _check("moe_route_permute", lib().moe_route_permute(
        _p(logits), T, E, k, _p(topk_ids), _p(topk_w), _p(expert_offsets), _p(row_src),
        _p(token_slot_row), _p(ws), ws.numel(), _stream(stream)))


def moe_quantize_nvfp4(x, q, sf, gs, gs_mode=MOE_GS_DYNAMIC, amax_in=None, ws=None, stream=None):
    rows, cols = x.shape
    dt = {torch.bfloat16: MOE_DTYPE_BF16, torch.float32: MOE_DTYPE_F32}[x.dtype]
    if ws is None:
        ws = _ws(lib().moe_quantize_nvfp4_workspace(rows, cols), x.device)
    _check("moe_quantize_nvfp4", lib().moe_quantize_nvfp4(
        _p(x), dt, rows, cols, _p(q), _p(sf), _p(gs), gs_mode, _p(amax_in),
        0 if amax_in is None else amax_in.numel(), _p(ws), ws.numel(), _stream(stream)))


def make_gemm_args(A, A_sf, A_gs, B, B_sf, B_gs, expert_offsets, R, epilogue, D=None,
                   amax_out=None, A_rows=None, N=None, K=None, D_sf=None, D_gs=None) -> moe_gemm_args:
    """B / B_sf are row-major NVFP4 [E, N, K/2] / [E, N, K/16]; pass B_sf=None and B as the
    packed buffer [E, N*K*9/16 bytes] (moe_pack_weights_nvfp4) with N and K for the packed
    layout.  D_sf / D_gs: scales and static global scale of D (SWIGLU_NVFP4 only)."""
    packed = B_sf is None
    if packed:
        E = B.shape[0]
    else:
        E, N, half_k = B.shape
        K = 2 * half_k
    a = moe_gemm_args()
    a.A, a.A_sf, a.A_gs, a.A_rows = _p(A), _p(A_sf), _p(A_gs), _p(A_rows)
    a.rows_A = A.shape[0]
    a.B, a.B_sf, a.B_gs, a.expert_offsets = _p(B), _p(B_sf), _p(B_gs), _p(expert_offsets)
    a.E, a.N, a.K, a.R, a.epilogue = E, N, K, int(R), epilogue
    a.D, a.amax_out = _p(D), _p(amax_out)
    a.B_layout = MOE_LAYOUT_PACKED if packed else MOE_LAYOUT_ROWMAJOR
    a.D_sf, a.D_gs = _p(D_sf), _p(D_gs)
    return a


def moe_grouped_gemm_nvfp4_workspace(args: moe_gemm_args) -> int:
    return lib().moe_grouped_gemm_nvfp4_workspace(C.byref(args))


def moe_grouped_gemm_nvfp4_amax_slots(args: moe_gemm_args) -> int:
    return lib().moe_grouped_gemm_nvfp4_amax_slots(C.byref(args))


def moe_grouped_gemm_nvfp4_can_implement(args: moe_gemm_args) -> int:
    return lib().moe_grouped_gemm_nvfp4_can_implement(C.byref(args))


def moe_grouped_gemm_nvfp4(args: moe_gemm_args, ws, stream=None):
    _check("moe_grouped_gemm_nvfp4",
           lib().moe_grouped_gemm_nvfp4(C.byref(args), _p(ws), ws.numel(), _stream(stream)))


MOE_NOALLOC_SCRATCH_BYTES = 1 << 20


def moe_grouped_gemm_nvfp4_noalloc(args: moe_gemm_args, stream=None):
    """The grouped GEMM with the library's static device scratch in place of a workspace
    (nothing is allocated; calls that overlap on one GPU race)."""
    _check("moe_grouped_gemm_nvfp4_noalloc",
           lib().moe_grouped_gemm_nvfp4_noalloc(C.byref(args), _stream(stream)))


def moe_pack_weights_nvfp4(B, B_sf, packed, stream=None):
    """B [..., K/2] codes and B_sf [..., K/16] scales of rows*K elements -> packed bytes."""
    K = B.shape[-1] * 2
    rows = B.numel() // (K // 2)
    _check("moe_pack_weights_nvfp4", lib().moe_pack_weights_nvfp4(
        _p(B), _p(B_sf), rows, K, _p(packed), _stream(stream)))


def moe_finalize(Y, topk_w, token_slot_row, out, stream=None):
    T, k = topk_w.shape
    H = out.shape[1]
    _check("moe_finalize", lib().moe_finalize(
        _p(Y), Y.shape[0], _p(topk_w), _p(token_slot_row), T, k, H, _p(out), _stream(stream)))


_DTYPES = {torch.bfloat16: MOE_DTYPE_BF16, torch.float32: MOE_DTYPE_F32}


def _fp8_blocks(n: int) -> int:
    return -(-n // 128)


def _dense(fn: str, *tensors):
    """The library reads raw pointers: every (name, tensor, dtypes) given, None apart, has to be dense, of
    one of the dtypes and on one device, and what is read 16 bytes at a time (codes and bf16 or f32
    data) aligned to that."""
    device = None
    for name, t, dtypes in tensors:
        if t is None:
            continue
        at = t.get_device()
        if device is None:
            device = at
        if t.dtype not in dtypes or at != device or not t.is_contiguous() or (dtypes in _WIDE and t.data_ptr() % 16):
            raise MoeError(fn, MOE_ERR_UNSUPPORTED, f"{name}: a dense, aligned tensor of {dtypes} on one device is needed, got "
                           f"{t.dtype} {tuple(t.shape)} strides {t.stride()} on {t.device}")


def _current(fn: str, at: int, stream=None):
    """Kernels are launched on the current device: its tensors (device index `at`) and streams only."""
    if at < 0 or at != torch.cuda.current_device() or (stream is not None and stream.device_index != at):
        raise MoeError(fn, MOE_ERR_UNSUPPORTED, f"tensors and a stream of the current device are needed, got tensors of device {at}")


_U8, _MASK, _I32, _F32 = (torch.uint8,), (torch.uint8, torch.bool), (torch.int32,), (torch.float32,)
_BF16, _REAL = (torch.bfloat16,), (torch.bfloat16, torch.float32)
_CODES = (torch.uint8, torch.float8_e4m3fn)   # E4M3 codes as bytes, or as the type that checkpoints hold them in
_WIDE = (_U8, _BF16, _REAL, _CODES)


def _sized(fn: str, ok: bool, what: str):
    if not ok:
        raise MoeError(fn, MOE_ERR_SHAPE, what)


def moe_quantize_fp8(x, q, sf, stream=None):
    """x [rows, C] bf16 or f32 -> q [rows, C] E4M3 codes, sf [rows, ceil(C/128)] f32 scales.  Codes are u8
    or float8_e4m3fn, here and in the functions below."""
    _dense("moe_quantize_fp8", ("x", x, _REAL), ("q", q, _CODES), ("sf", sf, _F32))
    _sized("moe_quantize_fp8", x.dim() == 2, "x [rows, C] is needed")
    rows, cols = x.shape
    _sized("moe_quantize_fp8", q.numel() == rows * cols and sf.numel() == rows * _fp8_blocks(cols), "q or sf size")
    _current("moe_quantize_fp8", x.get_device(), stream)
    _check("moe_quantize_fp8", lib().moe_quantize_fp8(_at(x), _DTYPES[x.dtype], rows, cols, _at(q), _at(sf), _stream(stream)))


def moe_quantize_fp8_weights(w, q, sf, qt=None, sft=None, stream=None):
    """w [E, N, K] bf16 or f32 -> q, sf with one scale per 128 x 128 tile; qt [E, K, N] and sft
    receive the transposed copy."""
    _dense("moe_quantize_fp8_weights", ("w", w, _REAL), ("q", q, _CODES), ("sf", sf, _F32), ("qt", qt, _CODES), ("sft", sft, _F32))
    _sized("moe_quantize_fp8_weights", w.dim() == 3, "w [E, N, K] is needed")
    E, N, K = w.shape
    tiles = E * _fp8_blocks(N) * _fp8_blocks(K)
    _sized("moe_quantize_fp8_weights", all(t is None or t.numel() == n for t, n in (
        (q, w.numel()), (sf, tiles), (qt, w.numel()), (sft, tiles))), "an output's size")
    _current("moe_quantize_fp8_weights", w.get_device(), stream)
    _check("moe_quantize_fp8_weights", lib().moe_quantize_fp8_weights(
        _at(w), _DTYPES[w.dtype], E, N, K, _at(q), _at(sf), _at(qt), _at(sft), _stream(stream)))


def moe_fp8_token_blocks(R: int, E: int) -> int:
    return lib().moe_fp8_token_blocks(int(R), E)


def moe_quantize_fp8_tokens(x, expert_offsets, R, q, sf, rows=None, stream=None):
    """x [rows_x, C] -> q [blocks, C, 128], sf [blocks, C]: blocks of 128 permuted rows of a group,
    one scale per column (blocks = moe_fp8_token_blocks(R, E))."""
    _dense("moe_quantize_fp8_tokens", ("x", x, _REAL), ("expert_offsets", expert_offsets, _I32), ("q", q, _CODES), ("sf", sf, _F32), ("rows", rows, _I32))
    _sized("moe_quantize_fp8_tokens", x.dim() == 2, "x [rows_x, C] is needed")
    rows_x, cols = x.shape
    E = expert_offsets.numel() - 1
    blocks = moe_fp8_token_blocks(R, E)
    _sized("moe_quantize_fp8_tokens", q.numel() >= blocks * cols * 128 and sf.numel() >= blocks * cols
           and (rows is None or rows.numel() >= R), "q, sf or rows size")
    _current("moe_quantize_fp8_tokens", x.get_device(), stream)
    _check("moe_quantize_fp8_tokens", lib().moe_quantize_fp8_tokens(
        _at(x), _DTYPES[x.dtype], rows_x, _at(rows), _at(expert_offsets), E, int(R), cols, _at(q), _at(sf), _stream(stream)))


def make_gemm_fp8_args(A, A_sf, B, B_sf, expert_offsets, R, epilogue, D=None, D_sf=None, A_rows=None) -> moe_gemm_fp8_args:
    """A [rows_A, K] / A_sf from moe_quantize_fp8, B [E, N, K] / B_sf from moe_quantize_fp8_weights;
    D bf16 [R, N] (NONE), or codes [R, N/2] with D_sf f32 [R, N/256] (SWIGLU_FP8).  The tensors must
    outlive the arguments' use.  epilogue | MOE_SUMS_WHOLE: whole products and binary32 sums."""
    fp8_act = epilogue & ~MOE_SUMS_WHOLE == MOE_EPI_SWIGLU_FP8
    _dense("make_gemm_fp8_args", ("A", A, _CODES), ("A_sf", A_sf, _F32), ("B", B, _CODES), ("B_sf", B_sf, _F32), ("expert_offsets", expert_offsets, _I32),
           ("D", D, _CODES if fp8_act else _BF16), ("D_sf", D_sf, _F32), ("A_rows", A_rows, _I32))
    _sized("make_gemm_fp8_args", A.dim() == 2 and B.dim() == 3, "A [rows_A, K] and B [E, N, K] are needed")
    E, N, K = B.shape
    rows_A, R, kb = A.shape[0], int(R), _fp8_blocks(K)
    _sized("make_gemm_fp8_args", A.shape[1] == K and A_sf.numel() == rows_A * kb and B_sf.numel() == E * _fp8_blocks(N) * kb
           and expert_offsets.numel() == E + 1 and (A_rows is None or A_rows.numel() >= R)
           and (D is None or D.numel() >= R * (N // 2 if fp8_act else N))
           and (D_sf is None or D_sf.numel() >= R * (N // 256)), "operand sizes do not agree")
    _current("make_gemm_fp8_args", A.get_device())
    args = moe_gemm_fp8_args(A.data_ptr(), A_sf.data_ptr(), A_rows.data_ptr() if A_rows is not None else None, rows_A,
                             B.data_ptr(), B_sf.data_ptr(), expert_offsets.data_ptr(), E, N, K, epilogue, R,
                             D.data_ptr() if D is not None else None, D_sf.data_ptr() if D_sf is not None else None)
    args.device = A.get_device()
    return args


def moe_grouped_gemm_fp8_can_implement(args: moe_gemm_fp8_args) -> int:
    return lib().moe_grouped_gemm_fp8_can_implement(C.byref(args))


def moe_grouped_gemm_fp8(args: moe_gemm_fp8_args, stream=None):
    if (at := getattr(args, "device", None)) is not None:   # (a caller may fill the structure without make_gemm_fp8_args)
        _current("moe_grouped_gemm_fp8", at, stream)
    _check("moe_grouped_gemm_fp8", lib().moe_grouped_gemm_fp8(C.byref(args), _stream(stream)))


def make_wgrad_fp8_args(Y, Y_sf, X, X_sf, expert_offsets, R, D) -> moe_wgrad_fp8_args:
    """Y [blocks, N, 128] / Y_sf and X [blocks, K, 128] / X_sf from moe_quantize_fp8_tokens over the
    same expert_offsets and R; D [E, N, K] f32 or bf16."""
    _dense("make_wgrad_fp8_args", ("Y", Y, _CODES), ("Y_sf", Y_sf, _F32), ("X", X, _CODES), ("X_sf", X_sf, _F32), ("expert_offsets", expert_offsets, _I32), ("D", D, _REAL))
    _sized("make_wgrad_fp8_args", D.dim() == 3, "D [E, N, K] is needed")
    E, N, K = D.shape
    blocks = moe_fp8_token_blocks(R, E)
    _sized("make_wgrad_fp8_args", expert_offsets.numel() == E + 1 and Y.numel() >= blocks * N * 128
           and Y_sf.numel() >= blocks * N and X.numel() >= blocks * K * 128 and X_sf.numel() >= blocks * K,
           "operand sizes do not agree")
    _current("make_wgrad_fp8_args", D.get_device())
    args = moe_wgrad_fp8_args(Y.data_ptr(), Y_sf.data_ptr(), X.data_ptr(), X_sf.data_ptr(), expert_offsets.data_ptr(),
                              E, N, K, _DTYPES[D.dtype], int(R), D.data_ptr())
    args.device = D.get_device()
    return args


def moe_grouped_wgrad_fp8_can_implement(args: moe_wgrad_fp8_args) -> int:
    return lib().moe_grouped_wgrad_fp8_can_implement(C.byref(args))


def moe_grouped_wgrad_fp8(args: moe_wgrad_fp8_args, stream=None):
    if (at := getattr(args, "device", None)) is not None:   # (a caller may fill the structure without make_wgrad_fp8_args)
        _current("moe_grouped_wgrad_fp8", at, stream)
    _check("moe_grouped_wgrad_fp8", lib().moe_grouped_wgrad_fp8(C.byref(args), _stream(stream)))


def moe_balance_loss_workspace(T: int, E: int, k: int, S: int) -> int:
    return lib().moe_balance_loss_workspace(T, E, k, S)


def moe_balance_loss(logits, topk_ids, counts, coef, loss, seq_offsets=None, token_mask=None, ws=None, stream=None):
    """logits [T, E] f32, topk_ids [T, k] i32, seq_offsets [S+1] i32 or None (S = 1), token_mask [T] u8
    or None -> counts [S, E] i32, coef [S, E] f32 (for the backward pass), loss [1] f32."""
    _dense("moe_balance_loss", ("logits", logits, _F32), ("topk_ids", topk_ids, _I32), ("counts", counts, _I32), ("coef", coef, _F32), ("loss", loss, _F32),
           ("seq_offsets", seq_offsets, _I32), ("token_mask", token_mask, _MASK), ("ws", ws, _U8))
    _sized("moe_balance_loss", logits.dim() == 2 and topk_ids.dim() == 2, "logits [T, E] and topk_ids [T, k] are needed")
    (T, E), k = logits.shape, topk_ids.shape[1]
    S = 1 if seq_offsets is None else seq_offsets.numel() - 1
    _sized("moe_balance_loss", topk_ids.shape[0] == T and counts.numel() == S * E and coef.numel() == S * E
           and loss.numel() >= 1 and (token_mask is None or token_mask.numel() == T), "operand sizes do not agree")
    _current("moe_balance_loss", logits.get_device(), stream)
    if ws is None:
        with _allocating(stream):
            ws = _ws(moe_balance_loss_workspace(T, E, k, S), logits.device)
    _check("moe_balance_loss", lib().moe_balance_loss(
        _at(logits), _at(topk_ids), T, E, k, _at(seq_offsets), S, _at(token_mask), _at(counts), _at(coef), _at(loss),
        _at(ws), ws.numel(), _stream(stream)))


def moe_balance_loss_backward(logits, coef, grad_loss, dlogits, seq_offsets=None, token_mask=None,
                              topk_ids=None, topk_w=None, d_topk_w=None, stream=None):
    """dlogits [T, E] from grad_loss [1] and coef (moe_balance_loss); with topk_ids, topk_w and
    d_topk_w [T, k] the gradient of the routing weights is added in the same pass."""
    _dense("moe_balance_loss_backward", ("logits", logits, _F32), ("coef", coef, _F32), ("grad_loss", grad_loss, _F32), ("dlogits", dlogits, _F32),
           ("seq_offsets", seq_offsets, _I32), ("token_mask", token_mask, _MASK), ("topk_ids", topk_ids, _I32), ("topk_w", topk_w, _F32),
           ("d_topk_w", d_topk_w, _F32))
    _sized("moe_balance_loss_backward", logits.dim() == 2 and (d_topk_w is None or d_topk_w.dim() == 2), "logits [T, E] and d_topk_w [T, k] are needed")
    T, E = logits.shape
    S = 1 if seq_offsets is None else seq_offsets.numel() - 1
    k = 1 if d_topk_w is None else d_topk_w.shape[1]
    _sized("moe_balance_loss_backward", coef.numel() == S * E and grad_loss.numel() >= 1 and dlogits.shape == logits.shape
           and (token_mask is None or token_mask.numel() == T)
           and (d_topk_w is None or all(t is not None and t.shape == (T, k) for t in (topk_ids, topk_w, d_topk_w))),
           "operand sizes do not agree")
    _current("moe_balance_loss_backward", logits.get_device(), stream)
    _check("moe_balance_loss_backward", lib().moe_balance_loss_backward(
        _at(logits), T, E, _at(seq_offsets), S, _at(token_mask), _at(coef), _at(grad_loss), _at(topk_ids), _at(topk_w),
        _at(d_topk_w), k, _at(dlogits), _stream(stream)))


def make_gemm_bf16_args(A, B, expert_offsets, R, epilogue, D=None, Z=None, A_rows=None, B_layout=MOE_LAYOUT_ROWMAJOR) -> moe_gemm_bf16_args:
    """A [rows_A, K] and B [E, N, K] (MOE_LAYOUT_TRANSPOSED: [E, K, N]) bf16; D [R, N] (NONE), [R, N/2] with
    the pre-activations Z [R, N] or None (SWIGLU), [R, 2N] of Z [R, 2N] (SWIGLU_BACKWARD), all bf16.  The
    tensors must outlive the arguments' use."""
    fn = "make_gemm_bf16_args"
    _dense(fn, ("A", A, _BF16), ("B", B, _BF16), ("expert_offsets", expert_offsets, _I32), ("D", D, _BF16), ("Z", Z, _BF16), ("A_rows", A_rows, _I32))
    _sized(fn, A.dim() == 2 and B.dim() == 3, "A [rows_A, K] and B [E, N, K] or [E, K, N] are needed")
    E, N, K = B.shape
    if B_layout == MOE_LAYOUT_TRANSPOSED:
        N, K = K, N
    rows_A, R = A.shape[0], int(R)
    cols_D, cols_Z = {MOE_EPI_SWIGLU: (N // 2, N), MOE_EPI_SWIGLU_BACKWARD: (2 * N, 2 * N)}.get(epilogue, (N, 0))
    _sized(fn, A.shape[1] == K and expert_offsets.numel() == E + 1 and (A_rows is None or A_rows.numel() >= R)
           and (D is None or D.numel() >= R * cols_D) and (Z is None or Z.numel() >= R * cols_Z), "operand sizes do not agree")
    _current(fn, A.get_device())
    args = moe_gemm_bf16_args(A.data_ptr(), _at(A_rows), rows_A, B.data_ptr(), expert_offsets.data_ptr(), E, N, K, epilogue, B_layout, R, _at(D), _at(Z))
    args.device = A.get_device()
    return args


def moe_grouped_gemm_bf16_can_implement(args: moe_gemm_bf16_args) -> int:
    return lib().moe_grouped_gemm_bf16_can_implement(C.byref(args))


def moe_grouped_gemm_bf16(args: moe_gemm_bf16_args, stream=None):
    if (at := getattr(args, "device", None)) is not None:   # (a caller may fill the structure without make_gemm_bf16_args)
        _current("moe_grouped_gemm_bf16", at, stream)
    _check("moe_grouped_gemm_bf16", lib().moe_grouped_gemm_bf16(C.byref(args), _stream(stream)))


def make_wgrad_bf16_args(Y, X, expert_offsets, R, D, X_rows=None) -> moe_wgrad_bf16_args:
    """Y [R, N] (permuted rows) and X [rows_X, K] bf16, D [E, N, K] f32 or bf16."""
    fn = "make_wgrad_bf16_args"
    _dense(fn, ("Y", Y, _BF16), ("X", X, _BF16), ("expert_offsets", expert_offsets, _I32), ("D", D, _REAL), ("X_rows", X_rows, _I32))
    _sized(fn, D.dim() == 3 and Y.dim() == 2 and X.dim() == 2, "Y [R, N], X [rows_X, K] and D [E, N, K] are needed")
    (E, N, K), R = D.shape, int(R)
    _sized(fn, expert_offsets.numel() == E + 1 and Y.shape[0] >= R and Y.shape[1] == N and X.shape[1] == K
           and (X_rows is None or X_rows.numel() >= R), "operand sizes do not agree")
    _current(fn, D.get_device())
    args = moe_wgrad_bf16_args(Y.data_ptr(), X.data_ptr(), _at(X_rows), X.shape[0], expert_offsets.data_ptr(), E, N, K, _DTYPES[D.dtype], R, D.data_ptr())
    args.device = D.get_device()
    return args


def moe_grouped_wgrad_bf16_can_implement(args: moe_wgrad_bf16_args) -> int:
    return lib().moe_grouped_wgrad_bf16_can_implement(C.byref(args))


def moe_grouped_wgrad_bf16(args: moe_wgrad_bf16_args, stream=None):
    if (at := getattr(args, "device", None)) is not None:   # (a caller may fill the structure without make_wgrad_bf16_args)
        _current("moe_grouped_wgrad_bf16", at, stream)
    _check("moe_grouped_wgrad_bf16", lib().moe_grouped_wgrad_bf16(C.byref(args), _stream(stream)))


class GradList:
    """The tensors of a gradient norm and its clipping, checked and laid out for the library once: `tensors`
    f32 or bf16, dense, on one device; `out` (of the same sizes and types) receives the clipped values, None:
    `tensors` themselves.  It may serve any number of calls, as long as the tensors keep their memory (a
    tensor given other memory through `.data` or `.grad = ` needs a new GradList).  Clipping refuses (the norm
    does not) what it would write, outputs or `tensors` themselves, where that overlaps anything else of the list: of each
    tensor, its output may be the tensor itself, or lie apart from all."""

    def __init__(self, tensors, out=None):
        fn = "GradList"
        self.tensors, self.out = list(tensors), None if out is None else list(out)
        ts, outs = self.tensors, self.out
        self.count = len(ts)
        _sized(fn, outs is None or len(outs) == self.count, "as many outputs as tensors are needed")
        self.device = ts[0].get_device() if ts else None
        # (each question is put to all tensors at once: a model has hundreds, and this runs every step)
        T = torch.Tensor
        types, sizes = [t.dtype for t in ts], list(map(T.numel, ts))
        every = ts if outs is None else ts + outs
        if not (set(types) <= _DTYPES.keys() and (outs is None or [o.dtype for o in outs] == types)
                and all(map(T.is_contiguous, every)) and set(map(T.get_device, every)) <= {self.device}):
            raise MoeError(fn, MOE_ERR_UNSUPPORTED, "dense f32 or bf16 tensors on one device are needed, each output of its tensor's type, got "
                           + ", ".join(f"{t.dtype} {tuple(t.shape)} strides {t.stride()} on {t.device}" for t in every[:8]))
        if outs is not None and list(map(T.numel, outs)) != sizes:
            raise MoeError(fn, MOE_ERR_SHAPE, "each output needs its tensor's number of elements")
        words = [0] * (4 * max(self.count, 1))   # of each moe_tensor: src, dst, n, dtype
        n = 4 * self.count
        words[0:n:4] = map(T.data_ptr, ts)
        if outs is not None:
            words[1:n:4] = map(T.data_ptr, outs)
        words[2:n:4] = sizes
        words[3:n:4] = [_DTYPES[d] for d in types]
        self._words = array.array("q", words)
        self.items = self._words.buffer_info()[0]
        scratch = self._words[:]
        self.distinct = moe_grad_clip_can_implement(self, scratch) != MOE_ERR_UNSUPPORTED


def _grad_list(tensors, out=None) -> GradList:
    if isinstance(tensors, GradList):
        _sized("GradList", out is None, "a GradList has its outputs")
        return tensors
    return GradList(tensors, out)


def moe_grad_clip_can_implement(tensors: GradList, scratch: array.array) -> int:
    return lib().moe_grad_clip_can_implement(tensors.items, tensors.count, scratch.buffer_info()[0])


def _clippable(fn: str, g: GradList):
    if not g.distinct:
        raise MoeError(fn, MOE_ERR_UNSUPPORTED, "what is written may overlap nothing else of the list, and be in it once only")


def moe_grad_norm_workspace(tensors) -> int:
    g = _grad_list(tensors)
    return lib().moe_grad_norm_workspace(g.items, g.count)


def moe_grad_norm(tensors, norm, ws=None, stream=None):
    """norm [1] f32 = the 2-norm of all elements of `tensors` (a list, or a GradList)."""
    g = _grad_list(tensors)
    _dense("moe_grad_norm", ("norm", norm, _F32), ("ws", ws, _U8))
    _sized("moe_grad_norm", norm.numel() >= 1 and g.device in (None, norm.get_device()), "norm [1] on the tensors' device is needed")
    _current("moe_grad_norm", norm.get_device(), stream)
    if ws is None:
        with _allocating(stream):
            ws = _ws(lib().moe_grad_norm_workspace(g.items, g.count), norm.device)
    _check("moe_grad_norm", lib().moe_grad_norm(g.items, g.count, _at(norm), _at(ws), ws.numel(), _stream(stream)))


def moe_grad_clip(tensors, norm, max_norm, out=None, stream=None):
    """out (None: `tensors`, or what the GradList has) = tensors * min(1, max_norm / (norm + 1e-6))."""
    g = _grad_list(tensors, out)
    _clippable("moe_grad_clip", g)
    _dense("moe_grad_clip", ("norm", norm, _F32))
    _sized("moe_grad_clip", norm.numel() >= 1 and g.device in (None, norm.get_device()), "norm [1] on the tensors' device is needed")
    _current("moe_grad_clip", norm.get_device(), stream)
    _check("moe_grad_clip", lib().moe_grad_clip(g.items, g.count, _at(norm), float(max_norm), _stream(stream)))


def make_gemv_args(x, B, ids=None, topk_w=None, epilogue=MOE_EPI_NONE, D=None) -> moe_gemv_args:
    """x [T, K] bf16 (or [T*k, K], a row for each slot), B an NVFP4Tensor [E, N, K] or PackedWeights, ids
    [T, k] i32 or None (one expert), topk_w [T, k] f32 (FINALIZE); D bf16 [T*k, N] (NONE), [T*k, N/2]
    (SWIGLU), [T, N] (FINALIZE).  The tensors must outlive the arguments' use."""
    fn = "make_gemv_args"
    packed = isinstance(B, PackedWeights)
    codes, sf = (B.data, None) if packed else (B.q, B.sf)
    _dense(fn, ("x", x, _BF16), ("B", codes, _U8), ("B_sf", sf, _U8), ("B_gs", B.gs, _F32), ("ids", ids, _I32), ("topk_w", topk_w, _F32), ("D", D, _BF16))
    _sized(fn, x.dim() == 2 and codes.dim() == (2 if packed else 3) and (ids is None or ids.dim() == 2), "x [rows, K], B [E, N, K] and ids [T, k] are needed")
    E, (N, K) = codes.shape[0], (B.N, B.K) if packed else (codes.shape[1], 2 * codes.shape[2])
    T, k = (x.shape[0], 1) if ids is None else ids.shape
    cols, rows = (N // 2, T * k) if epilogue == MOE_EPI_SWIGLU else (N, T if epilogue == MOE_EPI_FINALIZE else T * k)
    _sized(fn, x.shape[1] == K and x.shape[0] in (T, T * k) and B.gs.numel() == E
           and (codes.numel() == E * N * K * 9 // 16 if packed else sf.numel() == E * N * K // 16)
           and (topk_w is None or topk_w.numel() == T * k) and (D is None or D.numel() >= rows * cols), "operand sizes do not agree")
    _current(fn, x.get_device())
    args = moe_gemv_args(x.data_ptr(), x.shape[0], codes.data_ptr(), _at(sf), B.gs.data_ptr(), _at(ids), _at(topk_w), T, k, E, N, K, epilogue,
                         MOE_LAYOUT_PACKED if packed else MOE_LAYOUT_ROWMAJOR, _at(D))
    args.device = x.get_device()
    return args


def moe_gemv_nvfp4_can_implement(args: moe_gemv_args) -> int:
    return lib().moe_gemv_nvfp4_can_implement(C.byref(args))


def moe_gemv_nvfp4(args: moe_gemv_args, stream=None):
    if (at := getattr(args, "device", None)) is not None:   # (a caller may fill the structure without make_gemv_args)
        _current("moe_gemv_nvfp4", at, stream)
    _check("moe_gemv_nvfp4", lib().moe_gemv_nvfp4(C.byref(args), _stream(stream)))


# ---- allocating helpers ------------------------------------------------------------

@dataclass
class NVFP4Tensor:
    """Device NVFP4 tensor: codes [..., C/2] u8, scales [..., C/16] u8, global scale(s) f32."""
    q: torch.Tensor
    sf: torch.Tensor
    gs: torch.Tensor


@dataclass
class PackedWeights:
    """Expert weights [E, N, K] in the packed layout: data [E, N*K*9/16] u8, gs [E] f32."""
    data: torch.Tensor
    gs: torch.Tensor
    N: int
    K: int


def pack_weights(W: NVFP4Tensor, stream=None) -> PackedWeights:
    E, N, half_k = W.q.shape
    K = 2 * half_k
    nbytes = lib().moe_pack_weights_nvfp4_bytes(E * N, K)
    if nbytes == 0:
        raise MoeError("moe_pack_weights_nvfp4_bytes", MOE_ERR_UNSUPPORTED, "rows % 32 or K % 256")
    data = torch.empty(E, nbytes // E, dtype=torch.uint8, device=W.q.device)
    moe_pack_weights_nvfp4(W.q, W.sf, data, stream)
    return PackedWeights(data, W.gs, N, K)


def quantize_alloc(x: torch.Tensor, gs=None, amax_in=None, stream=None) -> NVFP4Tensor:
    rows, cols = x.shape
    q = torch.empty(rows, cols // 2, dtype=torch.uint8, device=x.device)
    sf = torch.empty(rows, cols // 16, dtype=torch.uint8, device=x.device)
    mode = MOE_GS_STATIC if gs is not None else MOE_GS_DYNAMIC
    g = gs if gs is not None else torch.empty(1, dtype=torch.float32, device=x.device)
    moe_quantize_nvfp4(x, q, sf, g, mode, amax_in, stream=stream)
    return NVFP4Tensor(q, sf, g)


def route_permute_alloc(logits: torch.Tensor, k: int, stream=None):
    T, E = logits.shape
    dev = logits.device
    ids = torch.empty(T, k, dtype=torch.int32, device=dev)
    w = torch.empty(T, k, dtype=torch.float32, device=dev)
    off = torch.empty(E + 1, dtype=torch.int32, device=dev)
    row_src = torch.empty(T * k, dtype=torch.int32, device=dev)
    tsr = torch.empty(T * k, dtype=torch.int32, device=dev)
    ws = _ws(lib().moe_route_permute_workspace(T, E, k), dev)
    moe_route_permute(logits, k, ids, w, off, row_src, tsr, ws, stream)
    return ids, w, off, row_src, tsr


def _gemm_args_for(A: NVFP4Tensor, B, expert_offsets, R, epilogue, D, A_rows):
    if isinstance(B, PackedWeights):
        return make_gemm_args(A.q, A.sf, A.gs, B.data, None, B.gs, expert_offsets, R, epilogue, D,
                              None, A_rows, N=B.N, K=B.K)
    return make_gemm_args(A.q, A.sf, A.gs, B.q, B.sf, B.gs, expert_offsets, R, epilogue, D, None, A_rows)


def grouped_gemm_alloc(A: NVFP4Tensor, B, expert_offsets, R, epilogue=MOE_EPI_NONE,
                       A_rows=None, stream=None, D_gs=None):
    """B: NVFP4Tensor (row-major) or PackedWeights.  Returns D (and the partial-maxima tensor
    for SWIGLU; an NVFP4Tensor with global scale D_gs for SWIGLU_NVFP4)."""
    N = B.N if isinstance(B, PackedWeights) else B.q.shape[1]
    dev = A.q.device
    if epilogue == MOE_EPI_SWIGLU_NVFP4:
        I = N // 2
        Dq = NVFP4Tensor(torch.empty(int(R), I // 2, dtype=torch.uint8, device=dev),
                         torch.empty(int(R), I // 16, dtype=torch.uint8, device=dev), D_gs)
        a = _gemm_args_for(A, B, expert_offsets, R, epilogue, Dq.q, A_rows)
        a.D_sf, a.D_gs = _p(Dq.sf), _p(D_gs)
        _check("moe_grouped_gemm_nvfp4_can_implement", moe_grouped_gemm_nvfp4_can_implement(a))
        moe_grouped_gemm_nvfp4(a, _ws(moe_grouped_gemm_nvfp4_workspace(a), dev), stream)
        return Dq
    cols = N if epilogue == MOE_EPI_NONE else N // 2
    D = torch.empty(int(R), cols, dtype=torch.bfloat16, device=dev)
    a = _gemm_args_for(A, B, expert_offsets, R, epilogue, D, A_rows)
    amax = None
    if epilogue == MOE_EPI_SWIGLU:
        amax = torch.empty(max(moe_grouped_gemm_nvfp4_amax_slots(a), 1), dtype=torch.float32, device=dev)
        a.amax_out = _p(amax)
    _check("moe_grouped_gemm_nvfp4_can_implement", moe_grouped_gemm_nvfp4_can_implement(a))
    ws = _ws(moe_grouped_gemm_nvfp4_workspace(a), dev)
    moe_grouped_gemm_nvfp4(a, ws, stream)
    return (D, amax) if epilogue == MOE_EPI_SWIGLU else D


class MoELayerPlan:
    """Pre-allocated buffers and argument blocks for repeated forward passes of one layer
    shape (what a serving loop or a benchmark reuses): no allocation per call."""

    def __init__(self, T: int, E: int, k: int, H: int, I: int, W1, W2, device="cuda", static_g2=None):
        """W1 / W2: NVFP4Tensor (row-major) or PackedWeights (the fast decode layout).
        static_g2: a caller-calibrated global scale (one-element f32 device tensor) for the
        SwiGLU output; with it the gate/up GEMM requantises in its epilogue
        (MOE_EPI_SWIGLU_NVFP4) and requantize() does nothing."""
        self.T, self.E, self.k, self.H, self.I = T, E, k, H, I
        R = T * k
        self.R = R
        dev = torch.device(device)
        z = lambda *s, dt: torch.empty(*s, dtype=dt, device=dev)
        self.ids, self.w = z(T, k, dt=torch.int32), z(T, k, dt=torch.float32)
        self.off, self.row_src, self.tsr = z(E + 1, dt=torch.int32), z(R, dt=torch.int32), z(R, dt=torch.int32)
        self.xq = NVFP4Tensor(z(T, H // 2, dt=torch.uint8), z(T, H // 16, dt=torch.uint8), z(1, dt=torch.float32))
        self.act = z(R, I, dt=torch.bfloat16)
        self.actq = NVFP4Tensor(z(R, I // 2, dt=torch.uint8), z(R, I // 16, dt=torch.uint8), z(1, dt=torch.float32))
        self.Y = z(R, H, dt=torch.bfloat16)
        self.out = z(T, H, dt=torch.bfloat16)
        self.W1, self.W2 = W1, W2
        self.fused = static_g2 is not None
        if self.fused:
            self.actq.gs.copy_(static_g2.reshape(1))
            self.args1 = _gemm_args_for(self.xq, W1, self.off, R, MOE_EPI_SWIGLU_NVFP4, self.actq.q, self.row_src)
            self.args1.D_sf, self.args1.D_gs = _p(self.actq.sf), _p(self.actq.gs)
        else:
            self.args1 = _gemm_args_for(self.xq, W1, self.off, R, MOE_EPI_SWIGLU, self.act, self.row_src)
            self.amax = z(max(moe_grouped_gemm_nvfp4_amax_slots(self.args1), 1), dt=torch.float32)
            self.args1.amax_out = _p(self.amax)
        self.args2 = _gemm_args_for(self.actq, W2, self.off, R, MOE_EPI_NONE, self.Y, None)
        for a in (self.args1, self.args2):
            _check("moe_grouped_gemm_nvfp4_can_implement", moe_grouped_gemm_nvfp4_can_implement(a))
        L = lib()
        self.ws_route = _ws(L.moe_route_permute_workspace(T, E, k), dev)
        self.ws_q1 = _ws(L.moe_quantize_nvfp4_workspace(T, H), dev)
        self.ws_q2 = _ws(L.moe_quantize_nvfp4_workspace(R, I), dev)
        self.ws_g1 = _ws(moe_grouped_gemm_nvfp4_workspace(self.args1), dev)
        self.ws_g2 = _ws(moe_grouped_gemm_nvfp4_workspace(self.args2), dev)

    # the six calls of the layer, individually (the benchmark times them one by one)
    def route(self, logits, stream=None):
        moe_route_permute(logits, self.k, self.ids, self.w, self.off, self.row_src, self.tsr,
                          self.ws_route, stream)

    def quantize_input(self, x, stream=None):
        moe_quantize_nvfp4(x, self.xq.q, self.xq.sf, self.xq.gs, MOE_GS_DYNAMIC, None, self.ws_q1, stream)

    def gemm1(self, stream=None):
        moe_grouped_gemm_nvfp4(self.args1, self.ws_g1, stream)

    def requantize(self, stream=None):
        if self.fused:   # done in the gate/up GEMM's epilogue
            return
        moe_quantize_nvfp4(self.act, self.actq.q, self.actq.sf, self.actq.gs, MOE_GS_DYNAMIC, self.amax,
                           self.ws_q2, stream)

    def gemm2(self, stream=None):
        moe_grouped_gemm_nvfp4(self.args2, self.ws_g2, stream)

    def finalize(self, stream=None):
        moe_finalize(self.Y, self.w, self.tsr, self.out, stream)

    def forward(self, logits, x, stream=None):
        # One stream.  Routing (logits) and token quantisation (x) are independent, but running
        # the quantiser on a second stream beside the routing kernels made the layer slower:
        # the two cross-stream waits cost more than the ~15 us the overlap saves.
        main = stream if stream is not None else torch.cuda.current_stream()
        self.route(logits, main)
        self.quantize_input(x, main)
        self.gemm1(main)
        self.requantize(main)
        self.gemm2(main)
        self.finalize(main)
        return self.out

    def graph(self, logits, x) -> "torch.cuda.CUDAGraph":
        """Capture one forward pass over the input buffers `logits` and `x` into a HIP graph.
        replay() reruns the whole layer on whatever those buffers hold at the time, writing
        the same output buffers; a serving loop copies each batch into them first.  The pass
        allocates nothing and records no memory-set node: every buffer is cleared or written
        by the library's own kernels."""
        self.forward(logits, x)              # one eager pass first (lazy initialisation)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            self.forward(logits, x)
        torch.cuda.synchronize()
        return g


@dataclass
class FP8Tensor:
    """Device FP8 tensor: E4M3 codes (u8 or float8_e4m3fn) and f32 scales, one per 128 elements of the contraction (rows
    [rows, C] / [rows, ceil(C/128)], weights [E, N, K] / one per 128 x 128 tile, or token blocks
    [blocks, C, 128] / [blocks, C])."""
    q: torch.Tensor
    sf: torch.Tensor


def quantize_fp8_alloc(x: torch.Tensor, stream=None) -> FP8Tensor:
    rows, cols = x.shape
    with _allocating(stream):
        out = FP8Tensor(torch.empty(rows, cols, dtype=torch.uint8, device=x.device),
                        torch.empty(rows, _fp8_blocks(cols), dtype=torch.float32, device=x.device))
    moe_quantize_fp8(x, out.q, out.sf, stream)
    return out


def quantize_fp8_weights_alloc(w: torch.Tensor, transposed=False, stream=None):
    """FP8Tensor of w [E, N, K]; with `transposed` the pair (W, W^T) from one pass over w."""
    E, N, K = w.shape
    z = lambda a, b: FP8Tensor(torch.empty(E, a, b, dtype=torch.uint8, device=w.device),
                               torch.empty(E, _fp8_blocks(a), _fp8_blocks(b), dtype=torch.float32, device=w.device))
    with _allocating(stream):
        out, t = z(N, K), z(K, N) if transposed else None
    if not transposed:
        moe_quantize_fp8_weights(w, out.q, out.sf, stream=stream)
        return out
    moe_quantize_fp8_weights(w, out.q, out.sf, t.q, t.sf, stream)
    return out, t


def quantize_fp8_tokens_alloc(x: torch.Tensor, expert_offsets, R, rows=None, stream=None) -> FP8Tensor:
    blocks = moe_fp8_token_blocks(R, expert_offsets.numel() - 1)
    with _allocating(stream):
        out = FP8Tensor(torch.empty(blocks, x.shape[1], 128, dtype=torch.uint8, device=x.device),
                        torch.empty(blocks, x.shape[1], dtype=torch.float32, device=x.device))
    moe_quantize_fp8_tokens(x, expert_offsets, R, out.q, out.sf, rows, stream)
    return out


def grouped_gemm_fp8_alloc(A: FP8Tensor, B: FP8Tensor, expert_offsets, R, epilogue=MOE_EPI_NONE, A_rows=None, stream=None):
    """D bf16 [R, N] (NONE) or the FP8Tensor act [R, N/2] (SWIGLU_FP8); epilogue | MOE_SUMS_WHOLE as in
    make_gemm_fp8_args."""
    N, R, dev = B.q.shape[1], int(R), A.q.device
    with _allocating(stream):
        if epilogue & ~MOE_SUMS_WHOLE == MOE_EPI_SWIGLU_FP8:
            out = FP8Tensor(torch.empty(R, N // 2, dtype=torch.uint8, device=dev),
                            torch.empty(R, N // 256, dtype=torch.float32, device=dev))
            D, D_sf = out.q, out.sf
        else:
            out = D = torch.empty(R, N, dtype=torch.bfloat16, device=dev)
            D_sf = None
    moe_grouped_gemm_fp8(make_gemm_fp8_args(A.q, A.sf, B.q, B.sf, expert_offsets, R, epilogue, D, D_sf, A_rows), stream)
    return out


def grouped_wgrad_fp8_alloc(dY: FP8Tensor, X: FP8Tensor, expert_offsets, R, dtype=torch.float32, stream=None):
    """dW [E, N, K] from quantize_fp8_tokens_alloc of the output gradients and of the rows."""
    E, N, K = expert_offsets.numel() - 1, dY.q.shape[1], X.q.shape[1]
    with _allocating(stream):
        D = torch.empty(E, N, K, dtype=dtype, device=dY.q.device)
    moe_grouped_wgrad_fp8(make_wgrad_fp8_args(dY.q, dY.sf, X.q, X.sf, expert_offsets, R, D), stream)
    return D


def balance_loss_alloc(logits: torch.Tensor, topk_ids: torch.Tensor, seq_offsets=None, token_mask=None, stream=None):
    """(loss [1], counts [S, E], coef [S, E]); coef goes to moe_balance_loss_backward."""
    S, E = 1 if seq_offsets is None else seq_offsets.numel() - 1, logits.shape[1]
    with _allocating(stream):
        counts = torch.empty(S, E, dtype=torch.int32, device=logits.device)
        coef = torch.empty(S, E, dtype=torch.float32, device=logits.device)
        loss = torch.empty(1, dtype=torch.float32, device=logits.device)
    moe_balance_loss(logits, topk_ids, counts, coef, loss, seq_offsets, token_mask, stream=stream)
    return loss, counts, coef


class MoEFP8LayerPlan:
    """The layer of MoELayerPlan with FP8 experts: W1 [E, 2I, H] and W2 [E, H, I] as FP8Tensor of
    quantize_fp8_weights_alloc (I % 128 == 0).  Buffers and argument blocks are allocated once; the
    gate/up product quantises its SwiGLU output itself.  whole_sums: both products with MOE_SUMS_WHOLE,
    so a token's output does not depend on the tokens beside it."""

    def __init__(self, T: int, E: int, k: int, H: int, I: int, W1: FP8Tensor, W2: FP8Tensor, device="cuda", whole_sums=False):
        self.T, self.E, self.k, self.H, self.I = T, E, k, H, I
        R = self.R = T * k
        dev = torch.device(device)
        z = lambda *s, dt: torch.empty(*s, dtype=dt, device=dev)
        self.ids, self.w = z(T, k, dt=torch.int32), z(T, k, dt=torch.float32)
        self.off, self.row_src, self.tsr = z(E + 1, dt=torch.int32), z(R, dt=torch.int32), z(R, dt=torch.int32)
        self.xq = FP8Tensor(z(T, H, dt=torch.uint8), z(T, _fp8_blocks(H), dt=torch.float32))
        self.actq = FP8Tensor(z(R, I, dt=torch.uint8), z(R, _fp8_blocks(I), dt=torch.float32))
        self.Y, self.out = z(R, H, dt=torch.bfloat16), z(T, H, dt=torch.bfloat16)
        _sized("MoEFP8LayerPlan", W1.q.shape == (E, 2 * I, H) and W2.q.shape == (E, H, I), "W1 [E, 2I, H] and W2 [E, H, I] are needed")
        self.W1, self.W2 = W1, W2
        whole = MOE_SUMS_WHOLE if whole_sums else 0
        self.args1 = make_gemm_fp8_args(self.xq.q, self.xq.sf, W1.q, W1.sf, self.off, R, MOE_EPI_SWIGLU_FP8 | whole,
                                        self.actq.q, self.actq.sf, self.row_src)
        self.args2 = make_gemm_fp8_args(self.actq.q, self.actq.sf, W2.q, W2.sf, self.off, R, MOE_EPI_NONE | whole, self.Y)
        for a in (self.args1, self.args2):
            _check("moe_grouped_gemm_fp8_can_implement", moe_grouped_gemm_fp8_can_implement(a))
        self.ws_route = _ws(lib().moe_route_permute_workspace(T, E, k), dev)

    def forward(self, logits, x, stream=None):
        _dense("MoEFP8LayerPlan.forward", ("logits", logits, _F32), ("x", x, _REAL), ("out", self.out, _BF16))
        _sized("MoEFP8LayerPlan.forward", logits.shape == (self.T, self.E) and x.shape == (self.T, self.H), "logits [T, E] and x [T, H] are needed")
        _current("MoEFP8LayerPlan.forward", self.out.get_device(), stream)
        main = stream if stream is not None else torch.cuda.current_stream()
        moe_route_permute(logits, self.k, self.ids, self.w, self.off, self.row_src, self.tsr, self.ws_route, main)
        moe_quantize_fp8(x, self.xq.q, self.xq.sf, main)
        moe_grouped_gemm_fp8(self.args1, main)
        moe_grouped_gemm_fp8(self.args2, main)
        moe_finalize(self.Y, self.w, self.tsr, self.out, main)
        return self.out

    def graph(self, logits, x) -> "torch.cuda.CUDAGraph":
        """As MoELayerPlan.graph: one forward pass over these input buffers, captured."""
        self.forward(logits, x)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            self.forward(logits, x)
        torch.cuda.synchronize()
        return g


def grouped_gemm_bf16_alloc(A: torch.Tensor, B: torch.Tensor, expert_offsets, R, A_rows=None, transposed=False, stream=None) -> torch.Tensor:
    """D bf16 [R, N] of A [rows_A, K] and B [E, N, K]; `transposed`: B [E, K, N]."""
    with _allocating(stream):
        D = torch.empty(int(R), B.shape[2 if transposed else 1], dtype=torch.bfloat16, device=A.device)
    moe_grouped_gemm_bf16(make_gemm_bf16_args(A, B, expert_offsets, R, MOE_EPI_NONE, D, A_rows=A_rows,
                                              B_layout=MOE_LAYOUT_TRANSPOSED if transposed else MOE_LAYOUT_ROWMAJOR), stream)
    return D


def gated_ffn_alloc(x: torch.Tensor, W1: torch.Tensor, expert_offsets, R, A_rows=None, save=True, stream=None):
    """(act [R, I], Z [R, 2I]) of x [rows, K] and W1 [E, 2I, K] (gate rows, then up rows): act = silu(gate) up,
    and with `save` the pre-activations that gated_ffn_backward_alloc reads (else None)."""
    N, R = W1.shape[1], int(R)
    with _allocating(stream):
        act = torch.empty(R, N // 2, dtype=torch.bfloat16, device=x.device)
        Z = torch.empty(R, N, dtype=torch.bfloat16, device=x.device) if save else None
    moe_grouped_gemm_bf16(make_gemm_bf16_args(x, W1, expert_offsets, R, MOE_EPI_SWIGLU, act, Z, A_rows), stream)
    return act, Z


def gated_ffn_backward_alloc(dY: torch.Tensor, W2: torch.Tensor, Z: torch.Tensor, expert_offsets, R, stream=None) -> torch.Tensor:
    """dZ [R, 2I]: the gradient of the pre-activations Z, from that of the down projection's output dY [R, H]
    and its weights W2 [E, H, I], in one product.  The rows' gradient is grouped_gemm_bf16_alloc(dZ, W1, ...,
    transposed=True), the weights' grouped_wgrad_bf16_alloc(dZ, x, ...)."""
    with _allocating(stream):
        dZ = torch.empty(int(R), 2 * W2.shape[2], dtype=torch.bfloat16, device=dY.device)
    moe_grouped_gemm_bf16(make_gemm_bf16_args(dY, W2, expert_offsets, R, MOE_EPI_SWIGLU_BACKWARD, dZ, Z, B_layout=MOE_LAYOUT_TRANSPOSED), stream)
    return dZ


def grouped_wgrad_bf16_alloc(dY: torch.Tensor, X: torch.Tensor, expert_offsets, R, X_rows=None, dtype=torch.float32, stream=None) -> torch.Tensor:
    """dW [E, N, K] of the permuted rows dY [R, N] and X [rows, K]."""
    with _allocating(stream):
        D = torch.empty(expert_offsets.numel() - 1, dY.shape[1], X.shape[1], dtype=dtype, device=dY.device)
    moe_grouped_wgrad_bf16(make_wgrad_bf16_args(dY, X, expert_offsets, R, D, X_rows), stream)
    return D


def clip_grad_norm(tensors, max_norm, out=None, stream=None) -> torch.Tensor:
    """Clips `tensors` (a list, or a GradList) by their global norm, in place or into `out`, and returns the
    norm before it, [1] f32 on the device."""
    g = _grad_list(tensors, out)
    if g.count:
        _current("clip_grad_norm", g.device, stream)
        _clippable("clip_grad_norm", g)
    device = torch.device("cuda", g.device if g.count else torch.cuda.current_device())
    with _allocating(stream):
        norm = torch.empty(1, dtype=torch.float32, device=device)
    moe_grad_norm(g, norm, stream=stream)
    moe_grad_clip(g, norm, max_norm, stream=stream)
    return norm


def gemv_nvfp4_alloc(x: torch.Tensor, B, ids=None, topk_w=None, epilogue=MOE_EPI_NONE, stream=None) -> torch.Tensor:
    """D of make_gemv_args, allocated."""
    N = B.N if isinstance(B, PackedWeights) else B.q.shape[1]
    T, k = (x.shape[0], 1) if ids is None else ids.shape
    with _allocating(stream):
        D = torch.empty(T if epilogue == MOE_EPI_FINALIZE else T * k, N // 2 if epilogue == MOE_EPI_SWIGLU else N, dtype=torch.bfloat16, device=x.device)
    moe_gemv_nvfp4(make_gemv_args(x, B, ids, topk_w, epilogue, D), stream)
    return D


class MoETokenPlan:
    """The layer of MoELayerPlan for one or a few tokens: the same weights (NVFP4Tensor or PackedWeights), the
    tokens and activations left in bf16, and three calls: routing, gate/up products with SwiGLU, down products
    with the weighted sum.  Buffers are allocated once.  From about five tokens on MoELayerPlan is faster."""

    def __init__(self, T: int, E: int, k: int, H: int, I: int, W1, W2, device="cuda"):
        self.T, self.E, self.k, self.H, self.I = T, E, k, H, I
        dev = torch.device(device)
        z = lambda *s, dt: torch.empty(*s, dtype=dt, device=dev)
        self.ids, self.w = z(T, k, dt=torch.int32), z(T, k, dt=torch.float32)
        self.off, self.row_src, self.tsr = z(E + 1, dt=torch.int32), z(T * k, dt=torch.int32), z(T * k, dt=torch.int32)
        self.x, self.act, self.out = z(T, H, dt=torch.bfloat16), z(T * k, I, dt=torch.bfloat16), z(T, H, dt=torch.bfloat16)
        self.W1, self.W2 = W1, W2
        self.args1 = make_gemv_args(self.x, W1, self.ids, None, MOE_EPI_SWIGLU, self.act)
        self.args2 = make_gemv_args(self.act, W2, self.ids, self.w, MOE_EPI_FINALIZE, self.out)
        _sized("MoETokenPlan", (self.args1.E, self.args1.N, self.args1.K) == (E, 2 * I, H)
               and (self.args2.E, self.args2.N, self.args2.K) == (E, H, I), "W1 [E, 2I, H] and W2 [E, H, I] are needed")
        for a in (self.args1, self.args2):
            _check("moe_gemv_nvfp4_can_implement", moe_gemv_nvfp4_can_implement(a))
        self.ws_route = _ws(lib().moe_route_permute_workspace(T, E, k), dev)

    def forward(self, logits, x, stream=None):
        fn = "MoETokenPlan.forward"
        _dense(fn, ("logits", logits, _F32), ("x", x, _BF16), ("out", self.out, _BF16))
        _sized(fn, logits.shape == (self.T, self.E) and x.shape == (self.T, self.H), "logits [T, E] and x [T, H] are needed")
        _current(fn, self.out.get_device(), stream)
        main = stream if stream is not None else torch.cuda.current_stream()
        moe_route_permute(logits, self.k, self.ids, self.w, self.off, self.row_src, self.tsr, self.ws_route, main)
        self.args1.x = x.data_ptr()
        moe_gemv_nvfp4(self.args1, main)
        moe_gemv_nvfp4(self.args2, main)
        return self.out

    def graph(self, logits, x) -> "torch.cuda.CUDAGraph":
        """As MoELayerPlan.graph: one forward pass over these input buffers, captured."""
        self.forward(logits, x)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            self.forward(logits, x)
        torch.cuda.synchronize()
        return g


def quantize_experts(W: torch.Tensor, stream=None) -> NVFP4Tensor:
    """NVFP4-quantise stacked expert weights W [E, rows, cols] (f32 or bf16), one dynamic
    global scale per expert, into one contiguous [E, rows, cols/2] tensor."""
    E, rows, cols = W.shape
    dev = W.device
    q = torch.empty(E, rows, cols // 2, dtype=torch.uint8, device=dev)
    sf = torch.empty(E, rows, cols // 16, dtype=torch.uint8, device=dev)
    gs = torch.empty(E, dtype=torch.float32, device=dev)
    ws = _ws(lib().moe_quantize_nvfp4_workspace(rows, cols), dev)
    for e in range(E):
        moe_quantize_nvfp4(W[e], q[e], sf[e], gs[e:e + 1], MOE_GS_DYNAMIC, None, ws, stream)
    return NVFP4Tensor(q, sf, gs)

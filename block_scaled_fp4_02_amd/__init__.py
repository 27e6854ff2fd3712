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
device) before they pass the pointers on.
"""
from __future__ import annotations

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
MOE_SUMS_WHOLE = 0x100   # with an FP8 product's epilogue
MOE_LAYOUT_ROWMAJOR, MOE_LAYOUT_PACKED = 0, 1

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

"""Python binding of the C ABI in ``include/w4a4.h`` (ctypes).

Argument marshalling only: every step of the quantized linear runs in the
HIP kernels of ``libw4a4.so``.  PyTorch supplies device memory and the HIP
stream.  If the library is missing this module raises at import: there is
no fallback path.
"""
from __future__ import annotations

import ctypes
import functools
import math
import os
import struct
from typing import Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libw4a4.so")

FMT_INT4, FMT_INT8, FMT_NVFP4, FMT_W4A8, FMT_FP8 = 0, 1, 2, 3, 4
DT_F32, DT_BF16, DT_I32 = 0, 1, 2
ORDER_SMOOTH_THEN_ROTATE, ORDER_ROTATE_THEN_SMOOTH = 0, 1
BRANCH_NONE, BRANCH_BF16 = 0, 1
# w4a8: quantize_act writes W4A8-layout int8 activations; the weights are int4
FMTS = {"int4": FMT_INT4, "int8": FMT_INT8, "nvfp4": FMT_NVFP4, "w4a8": FMT_W4A8, "fp8": FMT_FP8}
ORDERS = {"smooth_then_rotate": ORDER_SMOOTH_THEN_ROTATE,
          "rotate_then_smooth": ORDER_ROTATE_THEN_SMOOTH}
# activations of the 16-bit operators (swiglu: bf16_linear only)
ACTS = {"none": 0, "relu": 1, "gelu": 2, "gelu_tanh": 3, "silu": 4, "swiglu": 5}
ABI_VERSION = 3
MAX_BRANCH = 128   # W4A4_MAX_BRANCH: largest branch width (rank or kept channels)

EXPORTS = ["quantize_act", "quantize_act_gather", "quantize_act_lowrank", "quantize_act_project", "pack_weights", "pack_weights_gptq", "w4a4_gptq_workspace_size", "w4a4_linear", "w4a4_linear_noalloc", "w8a8_linear", "w4a8_linear", "fp8_linear", "lowrank_add",
           "w4a4_lowrank_project", "w4a4_lowrank_width", "w4a4_transform_amax", "w4a4_linear_plan",
           "w4a4_workspace_size", "w4a4_status_string",
           "w4a4_prefix_attention", "w4a4_prefix_attention_workspace", "bf16_linear", "w4a4_bf16_workspace_size",
           "w4a4_group_norm_act", "w4a4_group_norm_workspace",
           "w4a4_cache_append", "w4a4_cache_read", "w4a4_cache_attention", "w4a4_cache_attention_workspace",
           "w4a4_rotary_axes", "w4a4_gated_norm",
           "w4a4_last_error", "w4a4_abi_version"]


class QDesc(ctypes.Structure):
    _fields_ = [("fmt", ctypes.c_int32), ("fwht_block", ctypes.c_int32),
                ("order", ctypes.c_int32), ("tensor_scale", ctypes.c_float)]


class BranchDesc(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int32), ("r", ctypes.c_int32), ("ra", ctypes.c_int32),
                ("reserved", ctypes.c_int32), ("a", ctypes.c_void_p), ("lda", ctypes.c_int64),
                ("b", ctypes.c_void_p), ("ldb", ctypes.c_int64)]


# w4a4_attn, packed (filling a ctypes structure of 36 fields takes longer than a short kernel)
_ATTN = struct.Struct("7qfi" + "4q" + "3q3q" + "4q4q" + "2q" + "4q")


_EPILOGUE = struct.Struct("2i3q")   # w4a4_epilogue
_KVCACHE = struct.Struct("4q2f8q")   # w4a4_kvcache
_CACHE_ATTN = struct.Struct("4qfi" + "4q" + "3q" + "q" + "4q")   # w4a4_cache_attn
_ROTARY = struct.Struct("4q4i4i" + "3q" + "12q")   # w4a4_rotary
_GATED = struct.Struct("3q2f4i" + "4q" + "6q" + "3q" + "4q")   # w4a4_gated


class W4A4Error(RuntimeError):
    def __init__(self, fn, status, msg):
        super().__init__(f"{fn} failed with status {status}: {msg}")
        self.status = status


def load_library(path: str = LIB_PATH) -> ctypes.CDLL:
    if not os.path.exists(path):
        raise ImportError(f"{path} not built: run __graft_entry__.build() or "
                          f"python -m w4a4_post_quantized_channel_amd.build")
    lib = ctypes.CDLL(path)
    vp, i32, i64, f32, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t
    qd, br = ctypes.POINTER(QDesc), ctypes.POINTER(BranchDesc)
    sig = {
        "quantize_act": [vp, i32, i64, i64, i64, vp, qd, vp, vp, vp],
        "quantize_act_gather": [vp, i32, i64, i64, i64, vp, qd, vp, vp, vp, i64, vp, i64, vp],
        "quantize_act_lowrank": [vp, i32, i64, i64, i64, vp, qd, vp, vp, vp, i64, vp, i64, vp],
        "quantize_act_project": [vp, i32, i64, i64, i64, vp, qd, vp, vp, vp, i64, vp, i64, vp],
        "pack_weights": [vp, i32, i64, i64, i64, vp, qd, vp, vp, vp],
        "pack_weights_gptq": [vp, i32, i64, i64, i64, vp, qd, vp, vp, vp, vp, vp, sz, vp],
        "w4a4_gptq_workspace_size": [i64, i64],
        "w4a4_linear": [vp, vp, vp, vp, i64, i64, i64, i32, f32, br, vp, i32, i64, vp, sz, vp],
        "w4a4_linear_noalloc": [vp, vp, vp, vp, i64, i64, i64, i32, f32, br, vp, i32, i64, vp],
        "w8a8_linear": [vp, vp, vp, vp, i64, i64, i64, f32, br, vp, i32, i64, vp, sz, vp],
        "w4a8_linear": [vp, vp, vp, vp, i64, i64, i64, f32, br, vp, i32, i64, vp, sz, vp],
        "fp8_linear": [vp, vp, vp, vp, i64, i64, i64, f32, br, vp, i32, i64, vp, sz, vp],
        "w4a4_workspace_size": [i64, i64, i64, i32],
        "lowrank_add": [vp, i32, i64, i64, i64, vp, vp, vp, i64, i64, i64, vp, i32, i64, vp],
        "w4a4_lowrank_project": [vp, i32, i64, i64, i64, vp, vp, i64, vp, i64, vp],
        "w4a4_linear_plan": [i64, i64, i64, i32, i32, ctypes.POINTER(ctypes.c_int32)],
        "w4a4_lowrank_width": [i64, i64, i64],
        "w4a4_transform_amax": [vp, i32, i64, i64, i64, vp, qd, vp, vp],
        "w4a4_prefix_attention": [ctypes.c_char_p, vp, sz, vp],   # a packed w4a4_attn
        "w4a4_prefix_attention_workspace": [i64] * 7,
        "bf16_linear": [vp, i64, vp, i64, i64, i64, i64, ctypes.c_char_p, vp, i32, i64, vp, sz, vp],
        "w4a4_bf16_workspace_size": [i64, i64, i64, i32],
        "w4a4_group_norm_act": [vp, i32, i64, i64, i64, i64, i64, i64, vp, vp, f32, i32, vp, i64, i64, vp, sz, vp],
        "w4a4_group_norm_workspace": [i64] * 4,
        "w4a4_cache_append": [ctypes.c_char_p, vp, i64, i64, vp, i64, i64, i32, i64, vp, vp],   # a packed w4a4_kvcache
        "w4a4_cache_read": [ctypes.c_char_p, vp, i64, vp, i64, i64, vp, i64, i64, i32, vp],
        "w4a4_cache_attention": [ctypes.c_char_p, ctypes.c_char_p, vp, sz, vp],
        "w4a4_cache_attention_workspace": [i64] * 6,
        "w4a4_rotary_axes": [ctypes.c_char_p, vp],   # a packed w4a4_rotary
        "w4a4_gated_norm": [ctypes.c_char_p, vp],    # a packed w4a4_gated
        "w4a4_status_string": [ctypes.c_int],
        "w4a4_last_error": [],
        "w4a4_abi_version": [],
    }
    for name, args in sig.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = ctypes.c_int
    lib.w4a4_workspace_size.restype = ctypes.c_size_t
    lib.w4a4_gptq_workspace_size.restype = ctypes.c_size_t
    lib.w4a4_prefix_attention_workspace.restype = ctypes.c_size_t
    lib.w4a4_bf16_workspace_size.restype = ctypes.c_size_t
    lib.w4a4_group_norm_workspace.restype = ctypes.c_size_t
    lib.w4a4_cache_attention_workspace.restype = ctypes.c_size_t
    lib.w4a4_lowrank_width.restype = ctypes.c_int64
    lib.w4a4_status_string.restype = ctypes.c_char_p
    lib.w4a4_last_error.restype = ctypes.c_char_p
    if lib.w4a4_abi_version() != ABI_VERSION:
        raise ImportError("libw4a4.so ABI version mismatch")
    return lib


LIB = load_library()


def _check(fn: str, status: int):
    if status != 0:
        raise W4A4Error(fn, status, LIB.w4a4_last_error().decode())


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream) -> int:
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream


_DTYPES = {torch.bfloat16: DT_BF16, torch.float32: DT_F32, torch.int32: DT_I32}


def _dtype_code(t: torch.Tensor) -> int:
    code = _DTYPES.get(t.dtype)
    if code is None:
        raise TypeError(f"unsupported dtype {t.dtype}")
    return code


def _rowmajor(t: torch.Tensor):
    assert t.dim() == 2 and t.stride(1) == 1, "expect a 2-D row-major tensor"
    return t.shape[0], t.shape[1], t.stride(0)


def qdesc(fmt, fwht_block: int = 64, order="smooth_then_rotate", tensor_scale: float = 1.0) -> QDesc:
    f = FMTS[fmt] if isinstance(fmt, str) else int(fmt)
    o = ORDERS[order] if isinstance(order, str) else int(order)
    return QDesc(f, int(fwht_block), o, float(tensor_scale))


def code_shapes(fmt: str, R: int, K: int):
    """(codes shape, codes dtype, scales shape, scales dtype) of a packed operand."""
    if fmt == "int4":
        return (R, K // 2), torch.uint8, (R,), torch.float32
    if fmt in ("int8", "w4a8"):   # w4a8: activation side, int8 in the W4A8 layout
        return (R, K), torch.int8, (R,), torch.float32
    if fmt == "fp8":              # OCP E4M3 codes
        return (R, K), torch.uint8, (R,), torch.float32
    if fmt == "nvfp4":
        return (R, K // 2), torch.uint8, (R, K // 16), torch.uint8
    raise ValueError(fmt)


def _alloc_codes(fmt, R, K, device):
    cs, cd, ss, sd = code_shapes(fmt, R, K)
    return torch.empty(cs, dtype=cd, device=device), torch.empty(ss, dtype=sd, device=device)


def quantize_act(x: torch.Tensor, inv_smooth: Optional[torch.Tensor], fmt: str = "int4", *,
                 fwht_block: int = 64, order="smooth_then_rotate", tensor_scale: float = 1.0,
                 codes=None, scales=None, stream=None, M: Optional[int] = None):
    """Per-token quantization of the transformed activations (see include/w4a4.h)."""
    R, K, ld = _rowmajor(x)
    if M is not None:
        R = M
    if codes is None:
        codes, scales = _alloc_codes(fmt, R, K, x.device)
    q = qdesc(fmt, fwht_block, order, tensor_scale)
    _check("quantize_act", LIB.quantize_act(_ptr(x), _dtype_code(x), R, K, ld, _ptr(inv_smooth),
                                            ctypes.byref(q), _ptr(codes), _ptr(scales), _stream(stream)))
    return codes, scales


def pack_weights_gptq(w: torch.Tensor, smooth: Optional[torch.Tensor], u: torch.Tensor,
                      perm: Optional[torch.Tensor] = None, fmt: str = "int4", *, fwht_block: int = 64,
                      order="smooth_then_rotate", codes=None, scales=None, workspace=None, stream=None):
    """pack_weights with GPTQ-style rounding (u: float64 K x K upper factor, perm: int32[K] or None)."""
    R, K, ld = _rowmajor(w)
    if codes is None:
        codes, scales = _alloc_codes(fmt, R, K, w.device)
    if workspace is None:
        workspace = torch.empty(int(LIB.w4a4_gptq_workspace_size(R, K)), dtype=torch.uint8, device=w.device)
    assert u.dtype == torch.float64 and u.is_contiguous()
    q = qdesc(fmt, fwht_block, order)
    _check("pack_weights_gptq", LIB.pack_weights_gptq(
        _ptr(w), _dtype_code(w), R, K, ld, _ptr(smooth), ctypes.byref(q), _ptr(u), _ptr(perm), _ptr(codes),
        _ptr(scales), _ptr(workspace), workspace.numel(), _stream(stream)))
    return codes, scales


def quantize_act_gather(x: torch.Tensor, inv_smooth: Optional[torch.Tensor], idx: torch.Tensor,
                        fmt: str = "int4", *, fwht_block: int = 64, order="smooth_then_rotate",
                        tensor_scale: float = 1.0, codes=None, scales=None, xo=None, stream=None):
    """quantize_act plus the kept-channel operand xo = x[:, idx] from the same pass."""
    R, K, ld = _rowmajor(x)
    r = idx.shape[0]
    if codes is None:
        codes, scales = _alloc_codes(fmt, R, K, x.device)
    if xo is None:
        xo = torch.empty((R, r), dtype=torch.bfloat16, device=x.device)
    q = qdesc(fmt, fwht_block, order, tensor_scale)
    _check("quantize_act_gather",
           LIB.quantize_act_gather(_ptr(x), _dtype_code(x), R, K, ld, _ptr(inv_smooth), ctypes.byref(q),
                                   _ptr(codes), _ptr(scales), _ptr(idx), r, _ptr(xo), xo.stride(0),
                                   _stream(stream)))
    return codes, scales, xo


def lowrank_fusable(x: torch.Tensor, l1t: torch.Tensor) -> bool:
    """Whether quantize_act_lowrank takes this activation / rank (see the header)."""
    r, K = l1t.shape
    return x.dtype == torch.bfloat16 and K % 64 == 0 and K <= 4096 and r in (16, 32)


def quantize_act_lowrank(x: torch.Tensor, inv_smooth: Optional[torch.Tensor], l1t: torch.Tensor,
                         fmt: str = "int4", *, fwht_block: int = 64, order="smooth_then_rotate",
                         tensor_scale: float = 1.0, codes=None, scales=None, out=None, stream=None):
    """quantize_act plus the low-rank operand [bf16(x L1) | residual] from the same pass."""
    R, K, ld = _rowmajor(x)
    r = l1t.shape[0]
    if codes is None:
        codes, scales = _alloc_codes(fmt, R, K, x.device)
    if out is None:
        out = torch.empty((R, 2 * r), dtype=torch.bfloat16, device=x.device)
    q = qdesc(fmt, fwht_block, order, tensor_scale)
    _check("quantize_act_lowrank",
           LIB.quantize_act_lowrank(_ptr(x), _dtype_code(x), R, K, ld, _ptr(inv_smooth), ctypes.byref(q),
                                    _ptr(codes), _ptr(scales), _ptr(l1t), r, _ptr(out), out.stride(0),
                                    _stream(stream)))
    return codes, scales, out


def project_fusable(x: torch.Tensor, l1t: torch.Tensor) -> bool:
    """Whether quantize_act_project takes this activation / rank (see the header)."""
    r, K = l1t.shape
    return x.dtype == torch.bfloat16 and K % 16 == 0 and K <= 5120 and 1 <= r <= MAX_BRANCH


def quantize_act_project(x: torch.Tensor, inv_smooth: Optional[torch.Tensor], l1t: torch.Tensor,
                         fmt: str = "int4", *, fwht_block: int = 64, order="smooth_then_rotate",
                         tensor_scale: float = 1.0, codes=None, scales=None, out=None, stream=None):
    """quantize_act and lowrank_project (low-rank form) in one launch."""
    R, K, ld = _rowmajor(x)
    r = l1t.shape[0]
    if codes is None:
        codes, scales = _alloc_codes(fmt, R, K, x.device)
    if out is None:
        out = torch.empty((R, 2 * r), dtype=torch.bfloat16, device=x.device)
    q = qdesc(fmt, fwht_block, order, tensor_scale)
    _check("quantize_act_project",
           LIB.quantize_act_project(_ptr(x), _dtype_code(x), R, K, ld, _ptr(inv_smooth), ctypes.byref(q),
                                    _ptr(codes), _ptr(scales), _ptr(l1t), r, _ptr(out), out.stride(0),
                                    _stream(stream)))
    return codes, scales, out


def pack_weights(w: torch.Tensor, smooth: Optional[torch.Tensor], fmt: str = "int4", *,
                 fwht_block: int = 64, order="smooth_then_rotate", tensor_scale: float = 1.0,
                 codes=None, scales=None, stream=None):
    """Per-output-channel quantization of W S R (inverse transform folded in)."""
    R, K, ld = _rowmajor(w)
    if codes is None:
        codes, scales = _alloc_codes(fmt, R, K, w.device)
    q = qdesc(fmt, fwht_block, order, tensor_scale)
    _check("pack_weights", LIB.pack_weights(_ptr(w), _dtype_code(w), R, K, ld, _ptr(smooth),
                                            ctypes.byref(q), _ptr(codes), _ptr(scales), _stream(stream)))
    return codes, scales


def transform_amax(x: torch.Tensor, scale: Optional[torch.Tensor], *, fwht_block: int = 64,
                   order="smooth_then_rotate", out=None, stream=None) -> torch.Tensor:
    R, K, ld = _rowmajor(x)
    if out is None:
        out = torch.empty(1, dtype=torch.float32, device=x.device)
    q = qdesc("int4", fwht_block, order, 1.0)
    _check("w4a4_transform_amax", LIB.w4a4_transform_amax(_ptr(x), _dtype_code(x), R, K, ld, _ptr(scale),
                                                          ctypes.byref(q), _ptr(out), _stream(stream)))
    return out


def branch_desc(a: Optional[torch.Tensor], b: Optional[torch.Tensor], r: Optional[int] = None) -> BranchDesc:
    """Fused-branch descriptor: a is bf16 M x ra (ra = r, or 2 P r from lowrank_project), b is bf16 N x r."""
    if a is None:
        return BranchDesc(BRANCH_NONE, 0, 0, 0, None, 0, None, 0)
    r = b.shape[1] if r is None else r
    return BranchDesc(BRANCH_BF16, r, a.shape[1], 0, a.data_ptr(), a.stride(0), b.data_ptr(), b.stride(0))


PLAN_FAMILIES = {1: "decode", 2: "decode_split", 3: "tile", 4: "nvfp4_shared"}


def linear_plan(M: int, N: int, K: int, fmt: str, with_workspace: bool = True) -> dict:
    """The kernel the linear entry point runs for this shape (host query)."""
    out = (ctypes.c_int32 * 4)()
    _check("w4a4_linear_plan", LIB.w4a4_linear_plan(M, N, K, FMTS[fmt], int(with_workspace), out))
    return {"family": PLAN_FAMILIES[out[0]], "tile": (out[1], out[2]), "splits": out[3]}


def workspace_size(M: int, N: int, K: int, fmt: str) -> int:
    return int(LIB.w4a4_workspace_size(M, N, K, FMTS[fmt]))


def make_workspace(M: int, N: int, K: int, fmt: str, device="cuda") -> Optional[torch.Tensor]:
    n = workspace_size(M, N, K, fmt)
    return None if n == 0 else torch.empty(n, dtype=torch.uint8, device=device)


def _linear(fn: str, fmt: str, a_codes, a_scales, w_codes, w_scales, K: int, *, alpha=1.0,
            branch: Optional[BranchDesc] = None, y=None, y_dtype=torch.bfloat16, workspace=None,
            stream=None, M: Optional[int] = None):
    M = a_codes.shape[0] if M is None else M
    N = w_codes.shape[0]
    if y is None:
        y = torch.empty((M, N), dtype=y_dtype, device=a_codes.device)
    br = branch if branch is not None else branch_desc(None, None)
    args = (_ptr(a_codes), _ptr(a_scales), _ptr(w_codes), _ptr(w_scales), M, N, K)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    tail = (ctypes.byref(br), _ptr(y), _dtype_code(y), y.stride(0), _ptr(workspace), ws_bytes, _stream(stream))
    if fn in ("w8a8_linear", "w4a8_linear", "fp8_linear"):
        st = getattr(LIB, fn)(*args, float(alpha), *tail)
    else:
        st = LIB.w4a4_linear(*args, FMTS[fmt], float(alpha), *tail)
    _check(fn, st)
    return y


def w4a4_linear(a_codes, a_scales, w_codes, w_scales, K: int, fmt: str = "int4", **kw):
    """y = alpha * dequant(A . W^T) (+ fused bf16 branch); fmt int4 or nvfp4."""
    return _linear("w4a4_linear", fmt, a_codes, a_scales, w_codes, w_scales, K, **kw)


def linear_noalloc(a_codes, a_scales, w_codes, w_scales, K: int, fmt: str = "int4", *, alpha=1.0,
                   branch: Optional[BranchDesc] = None, y=None, y_dtype=torch.bfloat16, stream=None,
                   M: Optional[int] = None):
    """The linear of ``fmt`` with split-K partials in the library's static
    per-GPU buffer (no workspace, no allocation inside the call; ``y`` must
    be given by callers that cannot allocate)."""
    M = a_codes.shape[0] if M is None else M
    N = w_codes.shape[0]
    if y is None:
        y = torch.empty((M, N), dtype=y_dtype, device=a_codes.device)
    br = branch if branch is not None else branch_desc(None, None)
    _check("w4a4_linear_noalloc", LIB.w4a4_linear_noalloc(
        _ptr(a_codes), _ptr(a_scales), _ptr(w_codes), _ptr(w_scales), M, N, K, FMTS[fmt], float(alpha),
        ctypes.byref(br), _ptr(y), _dtype_code(y), y.stride(0), _stream(stream)))
    return y


def w8a8_linear(a_codes, a_scales, w_codes, w_scales, K: int, **kw):
    """INT8 W8A8 sibling of w4a4_linear."""
    return _linear("w8a8_linear", "int8", a_codes, a_scales, w_codes, w_scales, K, **kw)


def w4a8_linear(a_codes, a_scales, w_codes, w_scales, K: int, **kw):
    """INT8 activation codes x packed INT4 weight codes (W4A8)."""
    return _linear("w4a8_linear", "w4a8", a_codes, a_scales, w_codes, w_scales, K, **kw)


def fp8_linear(a_codes, a_scales, w_codes, w_scales, K: int, **kw):
    """FP8 (OCP E4M3) W8A8, fp32 accumulation."""
    return _linear("fp8_linear", "fp8", a_codes, a_scales, w_codes, w_scales, K, **kw)


def _check_branch_inputs(x, l1t, idx, lw=None):
    if x.dtype != torch.bfloat16:
        raise TypeError("the 16-bit branch takes bf16 activations")
    if l1t is not None and (l1t.dtype != torch.bfloat16 or not l1t.is_contiguous()
                            or l1t.shape[1] != x.shape[1]):
        raise TypeError("l1t must be a contiguous bf16 r x K tensor (L1 transposed)")
    if idx is not None and idx.dtype != torch.int32:
        raise TypeError("idx must be int32")
    if lw is not None and lw.dtype != torch.bfloat16:
        raise TypeError("lw must be bf16")


def lowrank_add(x: torch.Tensor, y: torch.Tensor, lw: torch.Tensor, *, l1t: Optional[torch.Tensor] = None,
                idx: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """y += (x L1) lw^T  or  y += x[:, idx] lw^T, in place (l1t = L1 transposed, r x K)."""
    _check_branch_inputs(x, l1t, idx, lw)
    M, K, ldx = _rowmajor(x)
    N, r = lw.shape
    _check("lowrank_add", LIB.lowrank_add(_ptr(x), _dtype_code(x), M, K, ldx, _ptr(l1t), _ptr(idx), _ptr(lw),
                                          lw.stride(0), r, N, _ptr(y), _dtype_code(y), y.stride(0), _stream(stream)))
    return y


def lowrank_width(M: int, K: int, r: int) -> int:
    """Columns lowrank_project needs in its output: 2 P r for a rank-r
    projection (r > 0; the result is the first 2r), or |r| for a gather of
    |r| kept channels (r < 0)."""
    return int(LIB.w4a4_lowrank_width(M, K, r))


def lowrank_project(x: torch.Tensor, *, l1t: Optional[torch.Tensor] = None, idx: Optional[torch.Tensor] = None,
                    out=None, stream=None) -> torch.Tensor:
    """The fused branch's ``a`` operand: [hi | lo] bf16 halves of x L1 (a view of
    the first 2r columns of ``out``), or x[:, idx]."""
    _check_branch_inputs(x, l1t, idx)
    M, K, ldx = _rowmajor(x)
    r = l1t.shape[0] if l1t is not None else idx.shape[0]
    width = lowrank_width(M, K, r if l1t is not None else -r)
    if out is None:
        out = torch.empty((M, width), dtype=torch.bfloat16, device=x.device)
    _check("w4a4_lowrank_project", LIB.w4a4_lowrank_project(_ptr(x), _dtype_code(x), M, K, ldx, _ptr(l1t), _ptr(idx),
                                                            r, _ptr(out), out.stride(0), _stream(stream)))
    return out[:, :2 * r] if l1t is not None else out


# ---------------------------------------------------------------------------
# 16-bit operators beside the quantized linears
#
# Each takes the workspace that its make_*_workspace gives for the same sizes
# (None where none is needed).  Called without, it computes the same on an
# unsplit plan: right for small shapes, many times slower for those that the
# split spreads over the card (prefix_attention over 8192 keys 3 times,
# group_norm_act of full frames 250 times).
# ---------------------------------------------------------------------------
def _matrix(name: str, t: torch.Tensor):
    """(rows, columns, row stride) of a row-major matrix; the stride of a single row is not used."""
    if t.dim() != 2 or (t.stride(1) != 1 and t.shape[1] > 1):
        raise ValueError(f"{name} must be a 2-D row-major tensor")
    rows, cols = t.shape
    return rows, cols, t.stride(0) if rows > 1 else cols


def _act_code(act: str) -> int:
    if act not in ACTS:
        raise ValueError(f"unknown activation {act!r}: one of {sorted(ACTS)}")
    return ACTS[act]


def _ws(nbytes: int, device) -> Optional[torch.Tensor]:
    return None if nbytes == 0 else torch.empty(nbytes, dtype=torch.uint8, device=device)


def _together(names: str, first: torch.Tensor, *others) -> int:
    """The address of ``first``, with every other operand (``names``) on its
    device.  An operand in host memory would fault the kernel: if ``first`` lies
    there the address is NULL, which the library refuses after its checks of
    sizes."""
    index = first.get_device()
    if index >= 0:
        for t in others:
            if t is not None and t.get_device() != index:
                break
        else:
            return first.data_ptr()
    device = first.device
    for t in others:
        if t is not None and t.device != device:
            name = next(n for n, o in zip(names.split(), others) if o is t)
            raise ValueError(f"{name} is on {t.device}, the first operand on {device}")
    return first.data_ptr() if first.is_cuda else 0


def _ws_args(workspace):
    return (None, 0) if workspace is None else (workspace.data_ptr(), workspace.nbytes)


def _attn_operand(name: str, t: torch.Tensor, shape):
    if t.dtype is not torch.bfloat16:
        raise TypeError(f"{name} must be bf16")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {shape}")
    st = t.stride()
    if st[-1] != 1:
        raise ValueError(f"the last dimension of {name} must be contiguous")
    return st


def prefix_attention_workspace_size(B: int, T: int, Hq: int, Hkv: int, D: int, P: int, S: int) -> int:
    return int(LIB.w4a4_prefix_attention_workspace(B, T, Hq, Hkv, D, P, S))


def make_prefix_attention_workspace(B: int, T: int, Hq: int, Hkv: int, D: int, P: int, S: int,
                                    device="cuda") -> Optional[torch.Tensor]:
    return _ws(prefix_attention_workspace_size(B, T, Hq, Hkv, D, P, S), device)


def prefix_attention(q: torch.Tensor, k_prefix: torch.Tensor, v_prefix: torch.Tensor, k_own: torch.Tensor,
                     v_own: torch.Tensor, *, own_len: Optional[torch.Tensor] = None,
                     prefix_keep: Optional[torch.Tensor] = None, causal: bool = False,
                     scale: Optional[float] = None, out: Optional[torch.Tensor] = None, workspace=None,
                     stream=None) -> torch.Tensor:
    """Attention of a batch over one shared prefix and each sequence's own keys.

    q [B, T, Hq, D]; k_prefix, v_prefix [P, Hkv, D]; k_own, v_own [B, S, Hkv, D]
    (all bf16, any strides that are multiples of 8, last dimension contiguous);
    own_len int32[B] or None; prefix_keep bool / uint8 [P] or None; scale
    defaults to 1 / sqrt(D).  Pass workspace=make_prefix_attention_workspace(...)
    unless the prefix is short.  See include/w4a4.h for the formula and the masks.
    """
    B, T, Hq, D = q.shape
    P, Hkv, _ = k_prefix.shape
    S = k_own.shape[1]
    if out is None:
        out = torch.empty((B, T, Hq, D), dtype=torch.bfloat16, device=q.device)
    qb, qt, qh, _ = _attn_operand("q", q, (B, T, Hq, D))
    ob, ot, oh, _ = _attn_operand("out", out, (B, T, Hq, D))
    kpp, kph, _ = _attn_operand("k_prefix", k_prefix, (P, Hkv, D))
    vpp, vph, _ = _attn_operand("v_prefix", v_prefix, (P, Hkv, D))
    kob, kos, koh, _ = _attn_operand("k_own", k_own, (B, S, Hkv, D))
    vob, vos, voh, _ = _attn_operand("v_own", v_own, (B, S, Hkv, D))
    if own_len is not None and (own_len.dtype is not torch.int32 or own_len.shape != (B,)
                                or not own_len.is_contiguous()):
        raise TypeError("own_len must be a contiguous int32[B] tensor")
    if prefix_keep is not None and (prefix_keep.dtype not in (torch.bool, torch.uint8) or prefix_keep.shape != (P,)
                                    or not prefix_keep.is_contiguous()):
        raise TypeError("prefix_keep must be a contiguous bool or uint8 [P] tensor")
    qp = _together("k_prefix v_prefix k_own v_own own_len prefix_keep out workspace", q, k_prefix, v_prefix, k_own,
                   v_own, own_len, prefix_keep, out, workspace)
    desc = _ATTN.pack(B, T, Hq, Hkv, D, P, S, D ** -0.5 if scale is None else scale, causal,
                      qp, qb, qt, qh, k_prefix.data_ptr(), kpp, kph, v_prefix.data_ptr(), vpp, vph,
                      k_own.data_ptr(), kob, kos, koh, v_own.data_ptr(), vob, vos, voh,
                      0 if own_len is None else own_len.data_ptr(),
                      0 if prefix_keep is None else prefix_keep.data_ptr(), out.data_ptr(), ob, ot, oh)
    st = LIB.w4a4_prefix_attention(desc, *_ws_args(workspace), _stream(stream))
    if st != 0:
        _check("w4a4_prefix_attention", st)
    return out


def bf16_linear_workspace_size(M: int, N: int, K: int, act: str = "none") -> int:
    return int(LIB.w4a4_bf16_workspace_size(M, N, K, _act_code(act)))


def make_bf16_linear_workspace(M: int, N: int, K: int, act: str = "none", device="cuda") -> Optional[torch.Tensor]:
    return _ws(bf16_linear_workspace_size(M, N, K, act), device)


def bf16_linear(x: torch.Tensor, w: torch.Tensor, *, bias: Optional[torch.Tensor] = None, act: str = "none",
                residual: Optional[torch.Tensor] = None, y: Optional[torch.Tensor] = None, y_dtype=torch.bfloat16,
                workspace=None, stream=None) -> torch.Tensor:
    """y = act(x w^T + bias) + residual in bf16 with fp32 sums (see include/w4a4.h).

    w holds N rows, or 2 N for act="swiglu" (gate rows, then up rows); bias is
    fp32 or bf16 with one entry per row of w; residual has y's shape and type
    and may be y itself.  Without workspace=make_bf16_linear_workspace(...) K is
    not split, which few rows of a long K need.
    """
    M, K, ldx = _matrix("x", x)
    NW, Kw, ldw = _matrix("w", w)
    code = _act_code(act)
    if x.dtype is not torch.bfloat16 or w.dtype is not torch.bfloat16:
        raise TypeError("bf16_linear takes bf16 x and w")
    if Kw != K or (code == 5 and NW % 2):
        raise ValueError(f"w of shape {tuple(w.shape)} does not fit x of shape {tuple(x.shape)} with act={act!r}")
    N = NW // 2 if code == 5 else NW
    if y is None:
        y = torch.empty((M, N), dtype=y_dtype, device=x.device)
    My, Ny, ldy = _matrix("y", y)
    if My != M or Ny != N:
        raise ValueError(f"y has shape {tuple(y.shape)}, expected {(M, N)}")
    bdt, bp, rp, ldr = DT_F32, 0, 0, 0
    if bias is not None:
        if bias.shape != (NW,) or not bias.is_contiguous():
            raise ValueError("bias must be contiguous, one entry per row of w")
        bdt, bp = _dtype_code(bias), bias.data_ptr()
    if residual is not None:
        Mr, Nr, ldr = _matrix("residual", residual)
        if residual.dtype is not y.dtype or Mr != M or Nr != N:
            raise TypeError("residual must have y's shape and dtype")
        rp = residual.data_ptr()
    xp = _together("w bias residual y workspace", x, w, bias, residual, y, workspace)
    st = LIB.bf16_linear(xp, ldx, w.data_ptr(), ldw, M, N, K, _EPILOGUE.pack(code, bdt, bp, rp, ldr),
                         y.data_ptr(), _dtype_code(y), ldy, *_ws_args(workspace), _stream(stream))
    if st != 0:
        _check("bf16_linear", st)
    return y


def make_group_norm_workspace(N: int, S: int, C: int, groups: int, device="cuda") -> Optional[torch.Tensor]:
    return _ws(int(LIB.w4a4_group_norm_workspace(N, S, C, groups)), device)


def group_norm_act(x: torch.Tensor, groups: int, weight: Optional[torch.Tensor] = None,
                   bias: Optional[torch.Tensor] = None, *, eps: float = 1e-5, act: str = "silu",
                   out: Optional[torch.Tensor] = None, workspace=None, stream=None) -> torch.Tensor:
    """Group normalisation with an activation on channels-last features x [N, S, C]
    (fp32 or bf16, channels contiguous; weight, bias fp32[C] or None; out may be x).
    Without workspace=make_group_norm_workspace(...) one workgroup takes whole
    groups of a sample, which is for small samples only."""
    if x.dim() != 3 or x.stride(2) != 1 or x.dtype not in (torch.float32, torch.bfloat16):
        raise TypeError("x must be an fp32 or bf16 [N, S, C] tensor with contiguous channels")
    N, S, C = x.shape
    if out is None:
        out = torch.empty((N, S, C), dtype=x.dtype, device=x.device)
    if out.shape != x.shape or out.dtype != x.dtype or out.stride(2) != 1:
        raise TypeError("out must have x's shape and dtype, with contiguous channels")
    for name, v in (("weight", weight), ("bias", bias)):
        if v is not None and (v.dtype != torch.float32 or v.shape != (C,) or not v.is_contiguous()):
            raise TypeError(f"{name} must be a contiguous fp32[C] tensor")
    xp = _together("weight bias out workspace", x, weight, bias, out, workspace)
    st = LIB.w4a4_group_norm_act(xp, _dtype_code(x), N, S, C, groups, x.stride(0),
                                 x.stride(1) if S > 1 else C, _ptr(weight), _ptr(bias), float(eps), _act_code(act),
                                 out.data_ptr(), out.stride(0), out.stride(1) if S > 1 else C, *_ws_args(workspace),
                                 _stream(stream))
    if st != 0:
        _check("w4a4_group_norm_act", st)
    return out


# ---------------------------------------------------------------------------
# Operators around a 4-bit key/value cache
#
# These check that their operands lie on the current device, whose stream they
# take.  With ``stream`` (a torch.cuda.Stream) the outputs that a call makes come
# from that stream's memory; the caller orders it with the streams that wrote the
# operands and that read the outputs.
# ---------------------------------------------------------------------------
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)   # (there is a CUDA tensor by then)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)   # the handle alone, without a Stream object


def _stream_for(t, stream) -> int:
    """The stream of a call on ``t``'s device, which has to be the current one."""
    index = t.get_device()                       # -1 in host memory
    if index >= 0:
        if index != _current_device():
            raise ValueError(f"the operands are on {t.device}, the current device is cuda:{_current_device()}: "
                             f"call under torch.cuda.device({index})")
        if stream is None:
            if _raw_stream is not None:
                return _raw_stream(index)
        elif getattr(stream, "device_index", index) != index:    # it would read this device's addresses on its own
            raise ValueError(f"the stream is on cuda:{stream.device_index}, the operands are on {t.device}")
    return _stream(stream)


def _empty(shape, dtype, device, stream) -> torch.Tensor:
    """An output of a call on ``stream``, from that stream's memory: work that other streams have queued may still
    use what they freed."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    if not isinstance(stream, torch.cuda.Stream):        # (something with a handle alone)
        stream = torch.cuda.ExternalStream(stream.cuda_stream, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


class _Fixed:
    """Attributes that a call's arguments were packed from are set once: a change would not reach the calls."""
    _packed = None

    def __setattr__(self, name, value):
        if self._packed is not None:
            raise AttributeError(f"a {type(self).__name__} is fixed: make a new one to change {name}")
        object.__setattr__(self, name, value)


class KVCache(_Fixed):
    """A paged cache of keys and values in NVFP4 (see w4a4_kvcache in include/w4a4.h).

    k_codes, v_codes uint8 [n_pages, Hkv, page, D / 2]; k_scales, v_scales uint8
    [n_pages, Hkv, page, D / 16]; pages contiguous inside, any stride from page to
    page that is a multiple of 16 bytes.  k_scale, v_scale: the static tensor scales
    (nvfp4_scale_from_amax of calibration data; rounded up to a power of two, every
    value is exact in bf16).  The tensors may be written between calls, not replaced.
    """

    def __init__(self, k_codes: torch.Tensor, k_scales: torch.Tensor, v_codes: torch.Tensor, v_scales: torch.Tensor,
                 k_scale: float = 1.0, v_scale: float = 1.0):
        if k_codes.dim() != 4:
            raise ValueError("k_codes must be [n_pages, Hkv, page, D / 2]")
        n, H, page, half = k_codes.shape
        self.n_pages, self.Hkv, self.page, self.D = n, H, page, 2 * half
        self.k_codes, self.k_scales, self.v_codes, self.v_scales = k_codes, k_scales, v_codes, v_scales
        self.k_scale, self.v_scale = float(k_scale), float(v_scale)
        self.device, self._index = k_codes.device, k_codes.get_device()
        strides = []
        for name, width in (("k_codes", half), ("k_scales", half // 8), ("v_codes", half), ("v_scales", half // 8)):
            t = getattr(self, name)
            if t.dtype is not torch.uint8:
                raise TypeError(f"{name} must be uint8")
            if t.shape != (n, H, page, width):
                raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {(n, H, page, width)}")
            if not t[:1].is_contiguous():
                raise ValueError(f"a page of {name} must be contiguous")
            strides.append(t.stride(0) if n > 1 else H * page * width)
        _together("k_scales v_codes v_scales", k_codes, k_scales, v_codes, v_scales)
        at = [t.data_ptr() if t.is_cuda else 0 for t in (k_codes, k_scales, v_codes, v_scales)]
        self._packed = _KVCACHE.pack(n, page, H, 2 * half, self.k_scale, self.v_scale, at[0], strides[0], at[1], strides[1],
                                   at[2], strides[2], at[3], strides[3])

    def __reduce__(self):                        # a copy is packed from its own tensors
        return KVCache, (self.k_codes, self.k_scales, self.v_codes, self.v_scales, self.k_scale, self.v_scale)

    def get_device(self) -> int:
        return self._index


def make_kv_cache(n_pages: int, page: int, Hkv: int, D: int, k_scale: float = 1.0, v_scale: float = 1.0,
                  device="cuda") -> KVCache:
    """An empty cache (its bytes are whatever the allocator gave; only slots that were appended mean anything)."""
    def new(width):
        return torch.empty((n_pages, Hkv, page, width), dtype=torch.uint8, device=device)

    return KVCache(new(D // 2), new(D // 16), new(D // 2), new(D // 16), k_scale, v_scale)


def _cache_rows(name: str, t: torch.Tensor, shape, dtype):
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    st = t.stride()
    if st[2] != 1:
        raise ValueError(f"the last dimension of {name} must be contiguous")
    return st


def _check_slots(slots: torch.Tensor) -> int:
    if slots.dtype is not torch.int32 or slots.dim() != 1 or not slots.is_contiguous():
        raise TypeError("slots must be a contiguous int32 vector")
    return slots.shape[0]


def cache_append(cache: KVCache, k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor, *, stream=None) -> None:
    """Quantises k, v [M, Hkv, D] (both fp32 or bf16, strides multiples of 8) into the token slots int32[M]
    of the cache (slot = page * cache.page + token of the page; one outside the cache skips its row; distinct)."""
    M = _check_slots(slots)
    shape = (M, cache.Hkv, cache.D)
    km, kh, _ = _cache_rows("k", k, shape, k.dtype)
    vm, vh, _ = _cache_rows("v", v, shape, k.dtype)
    kp = _together("v slots cache", k, v, slots, cache)
    st = LIB.w4a4_cache_append(cache._packed, kp, km, kh, v.data_ptr(), vm, vh, _dtype_code(k), M, slots.data_ptr(),
                               _stream_for(k, stream))
    if st != 0:
        _check("w4a4_cache_append", st)


def cache_read(cache: KVCache, slots: torch.Tensor, *, k: Optional[torch.Tensor] = None,
               v: Optional[torch.Tensor] = None, dtype=torch.bfloat16, stream=None):
    """Keys and values [M, Hkv, D] of the slots int32[M] (zeros for a slot outside the cache), as bf16 or fp32."""
    M = _check_slots(slots)
    shape = (M, cache.Hkv, cache.D)
    if k is None:
        k = _empty(shape, dtype if v is None else v.dtype, slots.device, stream)
    if v is None:
        v = _empty(shape, k.dtype, slots.device, stream)
    km, kh, _ = _cache_rows("k", k, shape, k.dtype)
    vm, vh, _ = _cache_rows("v", v, shape, k.dtype)
    kp = _together("v slots cache", k, v, slots, cache)
    st = LIB.w4a4_cache_read(cache._packed, slots.data_ptr(), M, kp, km, kh, v.data_ptr(), vm, vh, _dtype_code(k),
                             _stream_for(k, stream))
    if st != 0:
        _check("w4a4_cache_read", st)
    return k, v


@functools.lru_cache(maxsize=256)
def cache_attention_workspace_size(B: int, T: int, Hq: int, Hkv: int, D: int, max_len: int) -> int:
    """Bytes that cache_attention uses with these sizes for histories of up to max_len keys (the host looks at the
    plan of every length: 0.1 ms)."""
    return int(LIB.w4a4_cache_attention_workspace(B, T, Hq, Hkv, D, max_len))


def make_cache_attention_workspace(B: int, T: int, Hq: int, Hkv: int, D: int, max_len: int,
                                   device="cuda") -> Optional[torch.Tensor]:
    return _ws(cache_attention_workspace_size(B, T, Hq, Hkv, D, max_len), device)


def cache_attention(q: torch.Tensor, cache: KVCache, table: torch.Tensor, lens: torch.Tensor, *, causal: bool = False,
                    scale: Optional[float] = None, max_len: Optional[int] = None, out: Optional[torch.Tensor] = None,
                    workspace=None, stream=None) -> torch.Tensor:
    """Attention of q [B, T, Hq, D] (bf16) over each sequence's history in the cache.

    table int32 [B, pages] lists a sequence's pages (an entry outside the cache is an
    absent page, whose keys nobody sees), lens int32[B] its keys; causal: the T queries
    are its last T positions.  max_len (default: the table's reach) is a bound of lens
    that the host knows.  Pass workspace=make_cache_attention_workspace(...) for the
    same max_len or a larger one: without, the keys are not split, and few queries over
    a long history take several times as long.  scale defaults to 1 / sqrt(D).  See
    include/w4a4.h.
    """
    B, T, Hq, D = q.shape
    if D != cache.D:
        raise ValueError(f"q has head width {D}, the cache {cache.D}")
    if out is None:
        out = _empty((B, T, Hq, D), torch.bfloat16, q.device, stream)
    qb, qt, qh, _ = _attn_operand("q", q, (B, T, Hq, D))
    ob, ot, oh, _ = _attn_operand("out", out, (B, T, Hq, D))
    if table.dtype is not torch.int32 or table.dim() != 2 or table.shape[0] != B or (
            table.shape[1] > 1 and table.stride(1) != 1):
        raise TypeError("table must be an int32 [B, pages] tensor with contiguous rows")
    if lens.dtype is not torch.int32 or lens.shape != (B,) or not lens.is_contiguous():
        raise TypeError("lens must be a contiguous int32[B] tensor")
    pages = table.shape[1]
    qp = _together("table lens out workspace cache", q, table, lens, out, workspace, cache)
    desc = _CACHE_ATTN.pack(B, T, Hq, pages * cache.page if max_len is None else max_len,
                            D ** -0.5 if scale is None else scale, causal, qp, qb, qt, qh, table.data_ptr(),
                            table.stride(0), pages, lens.data_ptr(), out.data_ptr(), ob, ot, oh)
    st = LIB.w4a4_cache_attention(cache._packed, desc, *_ws_args(workspace), _stream_for(q, stream))
    if st != 0:
        _check("w4a4_cache_attention", st)
    return out


class RotaryTable(_Fixed):
    """Frequencies of rotary_axes: ``sections`` pairs of each axis, ``turns`` fp32 [pairs, 2] (see make_rotary_table)."""

    def __init__(self, sections, turns: torch.Tensor):
        self.sections, self.turns = tuple(int(s) for s in sections), turns
        if not 1 <= len(self.sections) <= 4:
            raise ValueError("one to four axes")
        if turns.dtype is not torch.float32 or turns.shape != (sum(self.sections), 2) or not turns.is_contiguous():
            raise TypeError("turns must be a contiguous fp32 [sum(sections), 2] tensor")
        self._packed = self.sections + (0,) * (4 - len(self.sections))


def make_rotary_table(sections, theta: float = 10000.0, *, freqs=None, device="cuda") -> RotaryTable:
    """The table of rotary_axes for ``sections`` pairs of each axis: pair i of an axis with s pairs turns by
    theta ** (-i / s) a position.  ``freqs`` gives the frequencies of all pairs instead (radians a position)."""
    sections = [int(s) for s in sections]
    if freqs is None:
        freqs = [theta ** (-i / s) for s in sections for i in range(s)]
    turns = torch.as_tensor(freqs, dtype=torch.float64).cpu() / (2.0 * math.pi)
    if turns.shape != (sum(sections),):
        raise ValueError(f"{tuple(turns.shape)} frequencies for {sum(sections)} pairs")
    hi = turns.float()
    return RotaryTable(sections, torch.stack([hi, (turns - hi.double()).float()], dim=1).contiguous().to(device))


def rotary_axes(q: torch.Tensor, k: Optional[torch.Tensor], pos: torch.Tensor, table: RotaryTable, *,
                interleaved: bool = True, q_out: Optional[torch.Tensor] = None, k_out: Optional[torch.Tensor] = None,
                stream=None):
    """Rotary positions with one to four axes on q [M, Hq, D] and k [M, Hk, D] (or None), fp32 or bf16.

    pos int32 or fp32 [M, axes]; interleaved: pairs are channels 2 i and 2 i + 1, otherwise i and
    i + pairs; channels behind the pairs are copied.  q_out / k_out may be q / k themselves.
    Returns (q_out, k_out).
    """
    shape, dtype = q.shape, q.dtype
    M, Hq, D = shape
    if q_out is None:
        q_out = _empty(shape, dtype, q.device, stream)
    qm, qh, _ = _cache_rows("q", q, shape, dtype)
    qom, qoh, _ = _cache_rows("q_out", q_out, shape, dtype)
    Hk = kp = km = kh = kop = kom = koh = 0
    if k is not None:
        Hk = k.shape[1]
        kshape = (M, Hk, D)
        if k_out is None:
            k_out = _empty(kshape, dtype, q.device, stream)
        km, kh, _ = _cache_rows("k", k, kshape, dtype)
        kom, koh, _ = _cache_rows("k_out", k_out, kshape, dtype)
        kp, kop = k.data_ptr(), k_out.data_ptr()
    axes = len(table.sections)
    if pos.dtype not in (torch.int32, torch.float32) or pos.shape != (M, axes) or (axes > 1 and pos.stride(1) != 1):
        raise TypeError(f"pos must be an int32 or fp32 [{M}, {axes}] tensor with contiguous rows")
    qp = _together("k pos table q_out k_out", q, k, pos, table.turns, q_out, k_out)
    st = LIB.w4a4_rotary_axes(
        _ROTARY.pack(M, Hq, Hk, D, _dtype_code(q), _dtype_code(pos), axes, 0 if interleaved else 1, *table._packed,
                     pos.data_ptr(), pos.stride(0), table.turns.data_ptr(), qp, qm, qh, q_out.data_ptr(), qom, qoh,
                     kp, km, kh, kop, kom, koh), _stream_for(q, stream))
    if st != 0:
        _check("w4a4_rotary_axes", st)
    return q_out, k_out


NORMS = {"layer": 0, "rms": 1}


def _like(name: str, t: torch.Tensor, shape):
    """(address, row stride) of a row-major matrix of that shape."""
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    ld, inner = t.stride()
    if inner != 1 and shape[1] > 1:
        raise ValueError(f"{name} must be row-major")
    return t.data_ptr(), ld if shape[0] > 1 else shape[1]


def _fp32(name: str, t: Optional[torch.Tensor], shape):
    """(address, row stride) of an fp32 matrix or vector of that shape; (0, 0) for None."""
    if t is None:
        return 0, 0
    if t.dtype is not torch.float32:
        raise TypeError(f"{name} must be fp32")
    if t.shape != shape:
        raise (ValueError if len(shape) == 2 else TypeError)(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    st = t.stride()
    if st[-1] != 1 and shape[-1] > 1:
        raise (ValueError if len(shape) == 2 else TypeError)(f"{name} must have contiguous channels")
    return t.data_ptr(), st[0]


def gated_norm(x: torch.Tensor, h: Optional[torch.Tensor] = None, *, gate: Optional[torch.Tensor] = None,
               alpha: float = 1.0, post_weight: Optional[torch.Tensor] = None, kind: str = "layer",
               weight: Optional[torch.Tensor] = None, bias: Optional[torch.Tensor] = None,
               scale: Optional[torch.Tensor] = None, shift: Optional[torch.Tensor] = None, eps: float = 1e-6,
               x_out: Optional[torch.Tensor] = None, y: Optional[torch.Tensor] = None, y_dtype=torch.bfloat16,
               norm: bool = True, stream=None):
    """The residual step behind a block and the norm in front of the next one:

        x' = alpha x + gate * h              (h: rms-normed with post_weight first, if that is given)
        y  = (norm(x') weight + bias) (1 + scale) + shift

    x, h [M, C] (fp32 or bf16 each); gate, scale, shift fp32 [R, C], M a multiple of R (R = 1: one for
    all rows, R = M: one a row); post_weight, weight, bias fp32[C]; kind "layer" or "rms".  x_out may be
    x itself.  norm=False leaves y out, and without h there is no x_out unless it is passed.
    Returns (x_out, y).
    """
    code = NORMS.get(kind)
    if code is None:
        raise ValueError(f"unknown norm {kind!r}: one of {sorted(NORMS)}")
    shape = x.shape
    M, C, ldx = _matrix("x", x)
    if x_out is None and h is not None:
        x_out = _empty((M, C), x.dtype, x.device, stream)
    if y is None and norm:
        y = _empty((M, C), y_dtype, x.device, stream)
    hp = ldh = xop = ldxo = yp = ldy = 0
    if h is not None:
        hp, ldh = _like("h", h, shape)
    if x_out is not None:
        xop, ldxo = _like("x_out", x_out, shape)
        if x_out.dtype is not x.dtype:
            raise TypeError("x_out must have x's dtype")
    if y is not None:
        yp, ldy = _like("y", y, shape)
    first = gate if gate is not None else scale if scale is not None else shift
    R, mods = 1, (0, 0, 0, 0, 0, 0)
    if first is not None:
        if first.dim() != 2 or first.shape[1] != C:
            raise ValueError(f"modulations must be [R, {C}], got {tuple(first.shape)}")
        mshape = first.shape
        R = mshape[0]
        mods = (*_fp32("gate", gate, mshape), *_fp32("scale", scale, mshape), *_fp32("shift", shift, mshape))
    vshape = shape[1:]
    pw, wp, bp = (_fp32("post_weight", post_weight, vshape)[0], _fp32("weight", weight, vshape)[0],
                  _fp32("bias", bias, vshape)[0])
    xp = _together("h gate scale shift post_weight weight bias x_out y", x, h, gate, scale, shift, post_weight, weight,
                   bias, x_out, y)
    xdt = _dtype_code(x)
    st = LIB.w4a4_gated_norm(
        _GATED.pack(M, C, R, alpha, eps, code, xdt, xdt if h is None else _dtype_code(h),
                    xdt if y is None else _dtype_code(y), xp, ldx, hp, ldh, *mods, pw, wp, bp, xop, ldxo, yp, ldy),
        _stream_for(x, stream))
    if st != 0:
        _check("w4a4_gated_norm", st)
    return x_out, y

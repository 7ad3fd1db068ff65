"""Thin Python binding of the C ABI in ``include/moe_layer_route.h``.

Argument marshalling only: every step of the MoE block runs in the HIP kernels
of ``libmoe_layer_route.so``.  PyTorch provides device memory (``torch.empty``)
and the current stream; nothing here computes on tensor values.  If the
library has not been built, every call raises ``MoEError`` -- there is no
fallback implementation.
"""
from __future__ import annotations

import contextlib
import ctypes
import os

import torch

PATH_AUTO, PATH_GEMV, PATH_GEMM = 0, 1, 2
_PATHS = {"auto": PATH_AUTO, "gemv": PATH_GEMV, "gemm": PATH_GEMM}
ROUTE_AUTO, ROUTE_EXACT, ROUTE_MFMA = 0, 1, 2
_ROUTES = {"auto": ROUTE_AUTO, "exact": ROUTE_EXACT, "mfma": ROUTE_MFMA}

# The in-tree build; MOE_LAYER_ROUTE_LIB may name another build of the same library.
LIB_PATH = os.environ.get("MOE_LAYER_ROUTE_LIB") or os.path.join(
    os.path.dirname(os.path.abspath(__file__)), "libmoe_layer_route.so")

EXPORTS = ("moe_abi_version", "moe_status_str", "moe_last_error", "moe_workspace_bytes", "moe_expert_path",
           "moe_route", "moe_route_ex",
           "moe_forward", "moe_forward_ex", "moe_forward_ep", "moe_permute", "moe_gate_up", "moe_down",
           "moe_combine", "moe_quantize_mxfp4", "moe_forward_mxfp4", "moe_forward_mxfp4_ex", "moe_gate_up_mxfp4",
           "moe_down_mxfp4", "moe_quantize_fp8", "moe_quantize_rows_fp8", "moe_workspace_bytes_fp8",
           "moe_forward_fp8", "moe_forward_fp8_ex", "moe_gate_up_fp8", "moe_down_fp8", "moe_forward_padded",
           "moe_probe_mfma_bf16", "moe_probe_read", "moe_forward_padded_mxfp4", "moe_forward_padded_fp8",
           "moe_forward_ep_mxfp4", "moe_forward_ep_fp8", "moe_probe_mfma_dot_bf16",
           "moe_forward_noalloc",
           "moe_add_rmsnorm", "moe_add_rmsnorm_fp8", "moe_workspace_bytes_norm_fp8", "moe_forward_norm_fp8",
           "moe_quantize_int4", "moe_pack_int4", "moe_forward_int4", "moe_forward_int4_ex", "moe_gate_up_int4",
           "moe_down_int4", "moe_forward_padded_int4", "moe_forward_ep_int4",
           "moe_quantize_rows_mxfp4", "moe_dequantize_rows_mxfp4", "moe_workspace_bytes_w4a4", "moe_forward_w4a4",
           "moe_forward_padded_w4a4", "moe_forward_ep_w4a4", "moe_gate_up_w4a4", "moe_down_w4a4",
           "moe_workspace_bytes_backward", "moe_backward")


class MoEError(RuntimeError):
    """A call into the native library failed (or the library is missing)."""


_lib = None

_vp, _i64, _i32, _sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_size_t
_f32 = ctypes.c_float
_SIGS = {
    "moe_abi_version": (ctypes.c_int, []),
    "moe_status_str": (ctypes.c_char_p, [ctypes.c_int]),
    "moe_last_error": (ctypes.c_char_p, []),
    "moe_workspace_bytes": (_sz, [_i64, _i32, _i32, _i32, _i32]),
    "moe_expert_path": (ctypes.c_int, [_i64, _i32, _i32]),
    "moe_route": (ctypes.c_int, [_vp, _vp, _vp, _i64, _i32, _i32, _i32, _vp, _vp, _vp]),
    "moe_route_ex": (ctypes.c_int, [_vp, _vp, _vp, _i64, _i32, _i32, _i32, _vp, _vp, _i32, _vp]),
    "moe_forward": (ctypes.c_int, [_vp] * 7 + [_i64, _i32, _i32, _i32, _i32] + [_vp] * 4 + [_sz, _vp]),
    "moe_forward_ex": (ctypes.c_int, [_vp] * 7 + [_i64, _i32, _i32, _i32, _i32] + [_vp] * 4 + [_sz, _i32, _vp]),
    "moe_forward_ep": (ctypes.c_int, [_vp] * 7 + [_i64, _i32, _i32, _i32, _i32, _i32, _i32] + [_vp] * 4
                       + [_sz, _i32, _vp]),
    "moe_permute": (ctypes.c_int, [_vp, _i64, _i32, _i32, _vp, _vp, _vp, _vp, _vp]),
    "moe_gate_up": (ctypes.c_int, [_vp] * 6 + [_i64, _i32, _i32, _i32, _i32, _vp, _i32, _vp]),
    "moe_down": (ctypes.c_int, [_vp] * 5 + [_i64, _i32, _i32, _i32, _i32, _vp, _i32, _vp]),
    "moe_combine": (ctypes.c_int, [_vp, _vp, _vp, _i64, _i32, _i32, _vp, _vp]),
    "moe_quantize_mxfp4": (ctypes.c_int, [_vp, _i32, _i32, _i32, _vp, _vp, _vp]),
    "moe_forward_mxfp4": (ctypes.c_int, [_vp] * 9 + [_i64, _i32, _i32, _i32, _i32] + [_vp] * 4 + [_sz, _vp]),
    "moe_forward_mxfp4_ex": (ctypes.c_int, [_vp] * 9 + [_i64, _i32, _i32, _i32, _i32] + [_vp] * 4 + [_sz, _i32, _vp]),
    "moe_gate_up_mxfp4": (ctypes.c_int, [_vp] * 7 + [_i64, _i32, _i32, _i32, _i32, _vp, _i32, _vp]),
    "moe_down_mxfp4": (ctypes.c_int, [_vp] * 6 + [_i64, _i32, _i32, _i32, _i32, _vp, _i32, _vp]),
    "moe_quantize_fp8": (ctypes.c_int, [_vp, _i32, _i32, _i32, _vp, _vp, _vp]),
    "moe_forward_padded": (ctypes.c_int, [_vp] * 7 + [_i64, _i32, _i32, _i32, _i32] + [_vp] * 5 + [_vp, _sz, _i32, _vp]),
    "moe_quantize_rows_fp8": (ctypes.c_int, [_vp, _i64, _i32, _vp, _vp, _vp]),
    "moe_workspace_bytes_fp8": (_sz, [_i64, _i32, _i32, _i32, _i32]),
    "moe_forward_fp8": (ctypes.c_int, [_vp] * 9 + [_i64, _i32, _i32, _i32, _i32] + [_vp] * 4 + [_sz, _vp]),
    "moe_forward_fp8_ex": (ctypes.c_int, [_vp] * 9 + [_i64, _i32, _i32, _i32, _i32] + [_vp] * 4 + [_sz, _i32, _vp]),
    "moe_gate_up_fp8": (ctypes.c_int, [_vp] * 8 + [_i64, _i32, _i32, _i32, _i32, _vp, _i32, _vp]),
    "moe_down_fp8": (ctypes.c_int, [_vp] * 7 + [_i64, _i32, _i32, _i32, _i32, _vp, _i32, _vp]),
    "moe_forward_padded_mxfp4": (ctypes.c_int, [_vp] * 9 + [_i64, _i32, _i32, _i32, _i32] + [_vp] * 5
                                 + [_vp, _sz, _i32, _vp]),
    "moe_forward_padded_fp8": (ctypes.c_int, [_vp] * 9 + [_i64, _i32, _i32, _i32, _i32] + [_vp] * 5
                               + [_vp, _sz, _i32, _vp]),
    "moe_forward_ep_mxfp4": (ctypes.c_int, [_vp] * 9 + [_i64, _i32, _i32, _i32, _i32, _i32, _i32] + [_vp] * 4
                             + [_sz, _i32, _vp]),
    "moe_forward_ep_fp8": (ctypes.c_int, [_vp] * 9 + [_i64, _i32, _i32, _i32, _i32, _i32, _i32] + [_vp] * 4
                           + [_sz, _i32, _vp]),
    "moe_probe_mfma_bf16": (ctypes.c_int, [_i32, _i32, _vp, _vp]),
    "moe_probe_read": (ctypes.c_int, [_vp, _sz, _i32, _vp, _vp]),
    "moe_probe_mfma_dot_bf16": (ctypes.c_int, [_vp, _vp, _i32, _i32, _vp, _vp]),
    "moe_forward_noalloc": (ctypes.c_int, [_vp] * 7 + [_i64, _i32, _i32, _i32, _i32] + [_vp] * 4),
    "moe_add_rmsnorm": (ctypes.c_int, [_vp] * 3 + [_i64, _i32, _f32] + [_vp] * 3),
    "moe_add_rmsnorm_fp8": (ctypes.c_int, [_vp] * 3 + [_i64, _i32, _f32] + [_vp] * 5),
    "moe_workspace_bytes_norm_fp8": (_sz, [_i64, _i32, _i32, _i32, _i32]),
    "moe_forward_norm_fp8": (ctypes.c_int, [_vp] * 3 + [_f32] + [_vp] * 8 + [_i64, _i32, _i32, _i32, _i32] + [_vp] * 5
                             + [_sz, _i32, _vp]),
    "moe_quantize_int4": (ctypes.c_int, [_vp, _i32, _i32, _i32, _i32, _vp, _vp, _vp, _vp]),
    "moe_pack_int4": (ctypes.c_int, [_vp, _i32, _i32, _i32, _vp, _vp]),
    "moe_forward_int4": (ctypes.c_int, [_vp] * 11 + [_i64] + [_i32] * 5 + [_vp] * 4 + [_sz, _vp]),
    "moe_forward_int4_ex": (ctypes.c_int, [_vp] * 11 + [_i64] + [_i32] * 5 + [_vp] * 4 + [_sz, _i32, _vp]),
    "moe_forward_padded_int4": (ctypes.c_int, [_vp] * 11 + [_i64] + [_i32] * 5 + [_vp] * 6 + [_sz, _i32, _vp]),
    "moe_forward_ep_int4": (ctypes.c_int, [_vp] * 11 + [_i64] + [_i32] * 7 + [_vp] * 4 + [_sz, _i32, _vp]),
    "moe_gate_up_int4": (ctypes.c_int, [_vp] * 8 + [_i64] + [_i32] * 5 + [_vp, _i32, _vp]),
    "moe_down_int4": (ctypes.c_int, [_vp] * 7 + [_i64] + [_i32] * 5 + [_vp, _i32, _vp]),
    "moe_quantize_rows_mxfp4": (ctypes.c_int, [_vp, _i64, _i32, _vp, _vp, _vp]),
    "moe_dequantize_rows_mxfp4": (ctypes.c_int, [_vp, _vp, _i64, _i32, _vp, _vp]),
    "moe_workspace_bytes_w4a4": (_sz, [_i64, _i32, _i32, _i32, _i32]),
    "moe_forward_w4a4": (ctypes.c_int, [_vp] * 9 + [_i64] + [_i32] * 4 + [_vp] * 4 + [_sz, _i32, _vp]),
    "moe_forward_padded_w4a4": (ctypes.c_int, [_vp] * 9 + [_i64] + [_i32] * 4 + [_vp] * 6 + [_sz, _i32, _vp]),
    "moe_forward_ep_w4a4": (ctypes.c_int, [_vp] * 9 + [_i64] + [_i32] * 6 + [_vp] * 4 + [_sz, _i32, _vp]),
    "moe_workspace_bytes_backward": (_sz, [_i64, _i32, _i32, _i32, _i32]),
    "moe_backward": (ctypes.c_int, [_vp] * 9 + [_i64] + [_i32] * 4 + [_vp] * 8 + [_sz, _vp]),
    "moe_gate_up_w4a4": (ctypes.c_int, [_vp] * 8 + [_i64] + [_i32] * 4 + [_vp, _vp, _i32, _vp]),
    "moe_down_w4a4": (ctypes.c_int, [_vp] * 7 + [_i64] + [_i32] * 4 + [_vp, _i32, _vp]),
}


def library(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load the native library (once).  Raises MoEError if it is missing."""
    global _lib
    if _lib is None:
        if not os.path.exists(path):
            raise MoEError(f"native library not built: {path} (run __graft_entry__.build())")
        lib = ctypes.CDLL(path)
        for name, (res, args) in _SIGS.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _lib = lib
    return _lib


def _check(status: int, what: str):
    if status != 0:
        lib = library()
        msg = lib.moe_last_error().decode()
        raise MoEError(f"{what}: {lib.moe_status_str(status).decode()} ({status}): {msg}")


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _ptr(t):
    if t is None:
        return None
    return ctypes.c_void_p(t.data_ptr())


def _dev(*ts):
    for t in ts:
        if t is not None:
            if not t.is_cuda:
                raise MoEError("tensors must be on the GPU")
            if not t.is_contiguous():
                raise MoEError("tensors must be contiguous")


_HERE = contextlib.nullcontext()


def _on(t, stream):
    """Where a call runs: t's device, and stream (a torch stream or a raw handle; default: that device's current
    stream).  Within it both are current, so that what the call allocates belongs to the stream that uses it."""
    if stream is None:
        return _HERE if t.device.index == torch.cuda.current_device() else torch.cuda.device(t.device)
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(int(stream), t.device) if int(stream) else torch.cuda.default_stream(t.device)
    if stream.device != t.device:
        raise MoEError(f"stream is on {stream.device}, the tensors on {t.device}")
    return torch.cuda.stream(stream)


# torch's own generated code reads the raw handle this way; building a stream object for it takes 2 us longer
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _here(t):
    """Raw handle of the current stream of t's device."""
    index = t.get_device()
    return _raw_stream(index) if _raw_stream else torch.cuda.current_stream(index).cuda_stream


def _place(t, stream):
    """_here, if t's device is the current one and stream is not given; None where the caller has to go through _on."""
    index = t.get_device()
    if index < 0:
        _dev(t)   # raises
    return _here(t) if stream is None and index == _current_device() else None


def _at(t):
    """A tensor's address; one that is never read where it has no elements (a call for no tokens is valid)."""
    return None if t is None else t.data_ptr() or 4096


def _dev_as(first, *ts):
    """Raises: not every tensor is contiguous and on the device of the first, a GPU."""
    _dev(first, *ts)
    raise MoEError("tensors are on several devices: "
                   + ", ".join(sorted({str(t.device) for t in (first, *ts) if t is not None})))


def _ats(*ts):
    """Their addresses (_at), every tensor being contiguous and on the device of the first, a GPU."""
    index = ts[0].get_device()
    at = []
    for t in ts:
        if t is None:
            at.append(None)
        elif t.get_device() == index and t.is_contiguous() and index >= 0:
            at.append(t.data_ptr() or 4096)
        else:
            _dev_as(*ts)
    return at


# ---------------------------------------------------------------------------
# argument checks: shapes and dtypes are checked against the sizes the call
# passes to the library, before anything is enqueued (a short weight or a
# too-small output would otherwise be read or written out of bounds)
# ---------------------------------------------------------------------------
def _req(t, name, shape, dtype=None, bf16=False):
    """t has exactly this shape (and dtype, or 2-byte elements for bf16 bit patterns)."""
    if t is None:
        return
    if t.shape != shape and tuple(t.shape) != tuple(shape):
        raise MoEError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    if dtype is not None and t.dtype != dtype:
        raise MoEError(f"{name}: expected {dtype}, got {t.dtype}")
    if bf16 and t.element_size() != 2:
        raise MoEError(f"{name}: expected a 2-byte (bf16) tensor, got {t.dtype}")


def _req_rows(t, name, min_rows, cols, dtype):
    """A buffer of at least min_rows rows of cols elements (cols None: 1-D)."""
    if t is None:
        return
    ok = t.dim() == (1 if cols is None else 2) and t.shape[0] >= min_rows and (cols is None or t.shape[1] == cols)
    if not ok:
        want = f"({min_rows}+,)" if cols is None else f"({min_rows}+, {cols})"
        raise MoEError(f"{name}: expected shape {want}, got {tuple(t.shape)}")
    if t.dtype != dtype:
        raise MoEError(f"{name}: expected {dtype}, got {t.dtype}")


def _dims(t, name, n):
    if t.dim() != n:
        raise MoEError(f"{name}: expected {n} dimensions, got shape {tuple(t.shape)}")


def _route_args(x, Wr, br, k, topk_ids=None, topk_w=None):
    """x [T][H], Wr [E][H], br [E] (bf16); optional topk_ids int32 / topk_w float32 [T][k]."""
    _dims(x, "x", 2)
    _dims(Wr, "Wr", 2)
    T, H = x.shape
    E = Wr.shape[0]
    _req(x, "x", (T, H), bf16=True)
    _req(Wr, "Wr", (E, H), bf16=True)
    _req(br, "br", (E,), bf16=True)
    _req(topk_ids, "topk_ids", (T, k), torch.int32)
    _req(topk_w, "topk_w", (T, k), torch.float32)
    return T, H, E


def _bf16_experts(Wgu, bgu, Wd, bd, n, H):
    """Wgu [n][H][2I], bgu [n][2I], Wd [n][I][H], bd [n][H] (bf16); returns I."""
    _dims(Wd, "Wd", 3)
    I = Wd.shape[1]
    _req(Wgu, "Wgu", (n, H, 2 * I), bf16=True)
    _req(bgu, "bgu", (n, 2 * I), bf16=True)
    _req(Wd, "Wd", (n, I, H), bf16=True)
    _req(bd, "bd", (n, H), bf16=True)
    return I


def _mxfp4_experts(Wgu_q, Wgu_s, bgu, Wd_q, Wd_s, bd, n, H):
    """MXFP4 codes [n][N][K/2] and scales [n][K/32][N] (uint8), biases bf16; returns I."""
    _dims(Wd_q, "Wd_q", 3)
    I = 2 * Wd_q.shape[2]
    if H % 32 or I % 32:
        raise MoEError(f"MXFP4 weights need H and I divisible by 32, got H={H}, I={I}")
    _req(Wgu_q, "Wgu_q", (n, 2 * I, H // 2), torch.uint8)
    _req(Wgu_s, "Wgu_s", (n, H // 32, 2 * I), torch.uint8)
    _req(bgu, "bgu", (n, 2 * I), bf16=True)
    _req(Wd_q, "Wd_q", (n, H, I // 2), torch.uint8)
    _req(Wd_s, "Wd_s", (n, I // 32, H), torch.uint8)
    _req(bd, "bd", (n, H), bf16=True)
    return I


def _fp8_experts(Wgu_q, Wgu_s, bgu, Wd_q, Wd_s, bd, n, H):
    """FP8 codes [n][N][K] (uint8), one float32 scale per expert, biases bf16; returns I."""
    _dims(Wd_q, "Wd_q", 3)
    I = Wd_q.shape[2]
    _req(Wgu_q, "Wgu_q", (n, 2 * I, H), torch.uint8)
    _req(Wgu_s, "Wgu_s", (n,), torch.float32)
    _req(bgu, "bgu", (n, 2 * I), bf16=True)
    _req(Wd_q, "Wd_q", (n, H, I), torch.uint8)
    _req(Wd_s, "Wd_s", (n,), torch.float32)
    _req(bd, "bd", (n, H), bf16=True)
    return I


def _local_experts(e_begin, n_local, E):
    if e_begin < 0 or n_local < 1 or e_begin + n_local > E:
        raise MoEError(f"expert range [{e_begin}, {e_begin + n_local}) is not inside [0, {E})")


def _padded_args(n_valid, expert_counts, E):
    if n_valid is not None and (n_valid.dtype != torch.int32 or n_valid.numel() != 1):
        raise MoEError("n_valid must be a one-element int32 tensor")
    if expert_counts is not None and (expert_counts.dtype != torch.int32 or expert_counts.numel() != E):
        raise MoEError("expert_counts must be an int32 tensor of E elements")


def path_code(path) -> int:
    if isinstance(path, str):
        return _PATHS[path]
    return int(path)


def expert_path(T: int, E: int, k: int) -> str:
    """The expert path ("gemv" or "gemm") the library picks for these sizes."""
    return {PATH_GEMV: "gemv", PATH_GEMM: "gemm"}[int(library().moe_expert_path(T, E, k))]


def workspace_bytes(T: int, H: int, E: int, k: int, I: int) -> int:
    return int(library().moe_workspace_bytes(T, H, E, k, I))


def alloc_workspace(T: int, H: int, E: int, k: int, I: int, device=None) -> torch.Tensor:
    n = workspace_bytes(T, H, E, k, I)
    return torch.empty(max(n, 256), dtype=torch.uint8, device=device or "cuda")


def moe_route(x, Wr, br, k: int, topk_ids=None, topk_w=None, method="auto", stream=None):
    """Router: returns (topk_ids int32 [T,k], topk_w float32 [T,k]).

    method: "auto", "exact" or "mfma" (same decision; speed only)."""
    T, H, E = _route_args(x, Wr, br, k, topk_ids, topk_w)
    _dev(x, Wr, br)
    if topk_ids is None:
        topk_ids = torch.empty((T, k), dtype=torch.int32, device=x.device)
    if topk_w is None:
        topk_w = torch.empty((T, k), dtype=torch.float32, device=x.device)
    _dev(topk_ids, topk_w)
    m = _ROUTES[method] if isinstance(method, str) else int(method)
    _check(library().moe_route_ex(_ptr(x), _ptr(Wr), _ptr(br), T, H, E, k, _ptr(topk_ids), _ptr(topk_w), m,
                                  _stream(stream)), "moe_route")
    return topk_ids, topk_w


def moe_forward(x, Wr, br, Wgu, bgu, Wd, bd, k: int = 4, y=None, workspace=None, topk_ids=None,
                topk_w=None, path="auto", stream=None):
    """Whole MoE block forward; returns y (bf16 [T,H]).

    topk_ids / topk_w: optional preallocated outputs of the routing decision.
    workspace: optional uint8 device buffer of at least workspace_bytes(...)."""
    T, H, E = _route_args(x, Wr, br, k, topk_ids, topk_w)
    I = _bf16_experts(Wgu, bgu, Wd, bd, E, H)
    _req(y, "y", (T, H), torch.bfloat16)
    _dev(x, Wr, br, Wgu, bgu, Wd, bd)
    if y is None:
        y = torch.empty((T, H), dtype=torch.bfloat16, device=x.device)
    if workspace is None:
        workspace = alloc_workspace(T, H, E, k, I, x.device)
    _dev(y, workspace, topk_ids, topk_w)
    st = library().moe_forward_ex(_ptr(x), _ptr(Wr), _ptr(br), _ptr(Wgu), _ptr(bgu), _ptr(Wd), _ptr(bd),
                                  T, H, E, k, I, _ptr(y), _ptr(topk_ids), _ptr(topk_w), _ptr(workspace),
                                  workspace.numel() * workspace.element_size(), path_code(path),
                                  _stream(stream))
    _check(st, "moe_forward")
    return y


def moe_forward_noalloc(x, Wr, br, Wgu, bgu, Wd, bd, k: int = 4, y=None, topk_ids=None, topk_w=None, stream=None):
    """moe_forward on the library's own scratch array (no workspace argument;
    the call itself allocates nothing).  For T*k*(2I + 4H + 16) bytes up to
    64 MiB; calls that overlap on one GPU race.  Returns y (bf16 [T,H])."""
    T, H, E = _route_args(x, Wr, br, k, topk_ids, topk_w)
    _bf16_experts(Wgu, bgu, Wd, bd, E, H)
    I = Wd.shape[1]
    _req(y, "y", (T, H), torch.bfloat16)
    _dev(x, Wr, br, Wgu, bgu, Wd, bd)
    if y is None:
        y = torch.empty((T, H), dtype=torch.bfloat16, device=x.device)
    _dev(y, topk_ids, topk_w)
    _check(library().moe_forward_noalloc(_ptr(x), _ptr(Wr), _ptr(br), _ptr(Wgu), _ptr(bgu), _ptr(Wd), _ptr(bd),
                                         T, H, E, k, I, _ptr(y), _ptr(topk_ids), _ptr(topk_w), _stream(stream)),
           "moe_forward_noalloc")
    return y


def moe_forward_ex(*args, **kw):
    return moe_forward(*args, **kw)


def moe_forward_ep(x, Wr, br, Wgu_local, bgu_local, Wd_local, bd_local, e_begin: int, k: int = 4,
                   y_partial=None, workspace=None, topk_ids=None, topk_w=None, path="auto", stream=None):
    """One expert-parallel rank's share: experts [e_begin, e_begin + n_local) of the E
    routed ones (n_local = Wgu_local.shape[0]); returns y_partial (float32 [T,H])."""
    T, H, E = _route_args(x, Wr, br, k, topk_ids, topk_w)
    _dims(Wgu_local, "Wgu_local", 3)
    n_local = Wgu_local.shape[0]
    _local_experts(e_begin, n_local, E)
    I = _bf16_experts(Wgu_local, bgu_local, Wd_local, bd_local, n_local, H)
    _req(y_partial, "y_partial", (T, H), torch.float32)
    _dev(x, Wr, br, Wgu_local, bgu_local, Wd_local, bd_local)
    if y_partial is None:
        y_partial = torch.empty((T, H), dtype=torch.float32, device=x.device)
    if workspace is None:
        workspace = alloc_workspace(T, H, E, k, I, x.device)
    _dev(y_partial, workspace, topk_ids, topk_w)
    st = library().moe_forward_ep(_ptr(x), _ptr(Wr), _ptr(br), _ptr(Wgu_local), _ptr(bgu_local),
                                  _ptr(Wd_local), _ptr(bd_local), T, H, E, k, I, e_begin, n_local,
                                  _ptr(y_partial), _ptr(topk_ids), _ptr(topk_w), _ptr(workspace),
                                  workspace.numel() * workspace.element_size(), path_code(path),
                                  _stream(stream))
    _check(st, "moe_forward_ep")
    return y_partial


def moe_permute(topk_ids, E: int, stream=None):
    """Expert-contiguous order: returns (cnt [E], off [E+1], rows [T*k], pos [T*k]) int32."""
    _dims(topk_ids, "topk_ids", 2)
    T, k = topk_ids.shape
    _req(topk_ids, "topk_ids", (T, k), torch.int32)
    _dev(topk_ids)
    dev = topk_ids.device
    cnt = torch.empty(E, dtype=torch.int32, device=dev)
    off = torch.empty(E + 1, dtype=torch.int32, device=dev)
    rows = torch.empty(max(T * k, 1), dtype=torch.int32, device=dev)
    pos = torch.empty(max(T * k, 1), dtype=torch.int32, device=dev)
    _check(library().moe_permute(_ptr(topk_ids), T, E, k, _ptr(cnt), _ptr(off), _ptr(rows), _ptr(pos),
                                 _stream(stream)), "moe_permute")
    return cnt, off, rows[:T * k], pos[:T * k]


def moe_gate_up(x, Wgu, bgu, cnt, off, rows, k: int, path="auto", h=None, stream=None):
    """Per-expert gate_up GEMM + bias + GLU; returns h (bf16 [T*k, I], permuted order)."""
    _dims(x, "x", 2)
    _dims(Wgu, "Wgu", 3)
    T, H = x.shape
    E, I = Wgu.shape[0], Wgu.shape[2] // 2
    _req(x, "x", (T, H), bf16=True)
    _req(Wgu, "Wgu", (E, H, 2 * I), bf16=True)
    _req(bgu, "bgu", (E, 2 * I), bf16=True)
    _req(cnt, "cnt", (E,), torch.int32)
    _req(off, "off", (E + 1,), torch.int32)
    _req_rows(rows, "rows", T * k, None, torch.int32)
    _req_rows(h, "h", T * k, I, torch.bfloat16)
    _dev(x, Wgu, bgu, cnt, off, rows)
    if h is None:
        h = torch.empty((max(T * k, 1), I), dtype=torch.bfloat16, device=x.device)
    _check(library().moe_gate_up(_ptr(x), _ptr(Wgu), _ptr(bgu), _ptr(cnt), _ptr(off), _ptr(rows), T, H, E,
                                 k, I, _ptr(h), path_code(path), _stream(stream)), "moe_gate_up")
    return h[:T * k]


def moe_down(h, Wd, bd, cnt, off, T: int, k: int, path="auto", o=None, stream=None):
    """Per-expert down GEMM + bias; returns o (float32 [T*k, H], permuted order)."""
    _dims(Wd, "Wd", 3)
    E, I, H = Wd.shape
    _req(Wd, "Wd", (E, I, H), bf16=True)
    _req(bd, "bd", (E, H), bf16=True)
    _req(cnt, "cnt", (E,), torch.int32)
    _req(off, "off", (E + 1,), torch.int32)
    _req_rows(h, "h", T * k, I, torch.bfloat16)
    _req_rows(o, "o", T * k, H, torch.float32)
    _dev(h, Wd, bd, cnt, off)
    if o is None:
        o = torch.empty((max(T * k, 1), H), dtype=torch.float32, device=h.device)
    _check(library().moe_down(_ptr(h), _ptr(Wd), _ptr(bd), _ptr(cnt), _ptr(off), T, H, E, k, I, _ptr(o),
                              path_code(path), _stream(stream)), "moe_down")
    return o[:T * k]


def moe_combine(o, pos, topk_w, y=None, stream=None):
    """Weighted combine; returns y (bf16 [T, H])."""
    _dims(topk_w, "topk_w", 2)
    _dims(o, "o", 2)
    T, k = topk_w.shape
    H = o.shape[1]
    _req(topk_w, "topk_w", (T, k), torch.float32)
    _req_rows(o, "o", T * k, H, torch.float32)
    _req_rows(pos, "pos", T * k, None, torch.int32)
    _req(y, "y", (T, H), torch.bfloat16)
    _dev(o, pos, topk_w)
    if y is None:
        y = torch.empty((T, H), dtype=torch.bfloat16, device=o.device)
    _check(library().moe_combine(_ptr(o), _ptr(pos), _ptr(topk_w), T, H, k, _ptr(y), _stream(stream)),
           "moe_combine")
    return y


# ---------------------------------------------------------------------------
# MXFP4 expert weights: codes uint8 [E][N][K/2] and scales uint8 [E][K/32][N]
# (gate_up: K = H, N = 2I; down: K = I, N = H)
# ---------------------------------------------------------------------------
def _u8(*ts):
    for t in ts:
        if t.dtype != torch.uint8:
            raise MoEError(f"expected a uint8 tensor, got {t.dtype}")


def moe_quantize_mxfp4(W, codes=None, scales=None, stream=None):
    """bf16 weights [E][K][N] (x.W form) -> (codes uint8 [E][N][K/2], scales uint8 [E][K/32][N])."""
    _dims(W, "W", 3)
    E, K, N = W.shape
    _req(W, "W", (E, K, N), bf16=True)
    _req(codes, "codes", (E, N, K // 2), torch.uint8)
    _req(scales, "scales", (E, K // 32, N), torch.uint8)
    _dev(W)
    if codes is None:
        codes = torch.empty((E, N, K // 2), dtype=torch.uint8, device=W.device)
    if scales is None:
        scales = torch.empty((E, K // 32, N), dtype=torch.uint8, device=W.device)
    _dev(codes, scales)
    _u8(codes, scales)
    _check(library().moe_quantize_mxfp4(_ptr(W), E, K, N, _ptr(codes), _ptr(scales), _stream(stream)),
           "moe_quantize_mxfp4")
    return codes, scales


def moe_forward_mxfp4(x, Wr, br, Wgu_q, Wgu_s, bgu, Wd_q, Wd_s, bd, k: int = 4, y=None, workspace=None,
                      topk_ids=None, topk_w=None, path="auto", stream=None):
    """moe_forward with MXFP4 expert weights; returns y (bf16 [T,H])."""
    T, H, E = _route_args(x, Wr, br, k, topk_ids, topk_w)
    I = _mxfp4_experts(Wgu_q, Wgu_s, bgu, Wd_q, Wd_s, bd, E, H)
    _req(y, "y", (T, H), torch.bfloat16)
    _dev(x, Wr, br, Wgu_q, Wgu_s, bgu, Wd_q, Wd_s, bd)
    if y is None:
        y = torch.empty((T, H), dtype=torch.bfloat16, device=x.device)
    if workspace is None:
        workspace = alloc_workspace(T, H, E, k, I, x.device)
    _dev(y, workspace, topk_ids, topk_w)
    st = library().moe_forward_mxfp4_ex(_ptr(x), _ptr(Wr), _ptr(br), _ptr(Wgu_q), _ptr(Wgu_s), _ptr(bgu),
                                        _ptr(Wd_q), _ptr(Wd_s), _ptr(bd), T, H, E, k, I, _ptr(y), _ptr(topk_ids),
                                        _ptr(topk_w), _ptr(workspace), workspace.numel() * workspace.element_size(),
                                        path_code(path), _stream(stream))
    _check(st, "moe_forward_mxfp4")
    return y


def moe_gate_up_mxfp4(x, Wgu_q, Wgu_s, bgu, cnt, off, rows, k: int, h=None, path="auto", stream=None):
    """MXFP4 gate_up + bias + GLU; returns h (bf16 [T*k, I], permuted order)."""
    _dims(x, "x", 2)
    _dims(Wgu_q, "Wgu_q", 3)
    T, H = x.shape
    E, I = Wgu_q.shape[0], Wgu_q.shape[1] // 2
    _req(x, "x", (T, H), bf16=True)
    _req(Wgu_q, "Wgu_q", (E, 2 * I, H // 2), torch.uint8)
    _req(Wgu_s, "Wgu_s", (E, H // 32, 2 * I), torch.uint8)
    _req(bgu, "bgu", (E, 2 * I), bf16=True)
    _req(cnt, "cnt", (E,), torch.int32)
    _req(off, "off", (E + 1,), torch.int32)
    _req_rows(rows, "rows", T * k, None, torch.int32)
    _req_rows(h, "h", T * k, I, torch.bfloat16)
    _dev(x, Wgu_q, Wgu_s, bgu, cnt, off, rows)
    if h is None:
        h = torch.empty((max(T * k, 1), I), dtype=torch.bfloat16, device=x.device)
    _check(library().moe_gate_up_mxfp4(_ptr(x), _ptr(Wgu_q), _ptr(Wgu_s), _ptr(bgu), _ptr(cnt), _ptr(off),
                                       _ptr(rows), T, H, E, k, I, _ptr(h), path_code(path), _stream(stream)),
           "moe_gate_up_mxfp4")
    return h[:T * k]


def moe_down_mxfp4(h, Wd_q, Wd_s, bd, cnt, off, T: int, k: int, o=None, path="auto", stream=None):
    """MXFP4 down + bias; returns o (float32 [T*k, H], permuted order)."""
    _dims(Wd_q, "Wd_q", 3)
    E, H, I2 = Wd_q.shape
    I = 2 * I2
    _req(Wd_q, "Wd_q", (E, H, I2), torch.uint8)
    _req(Wd_s, "Wd_s", (E, I // 32, H), torch.uint8)
    _req(bd, "bd", (E, H), bf16=True)
    _req(cnt, "cnt", (E,), torch.int32)
    _req(off, "off", (E + 1,), torch.int32)
    _req_rows(h, "h", T * k, I, torch.bfloat16)
    _req_rows(o, "o", T * k, H, torch.float32)
    _dev(h, Wd_q, Wd_s, bd, cnt, off)
    if o is None:
        o = torch.empty((max(T * k, 1), H), dtype=torch.float32, device=h.device)
    _check(library().moe_down_mxfp4(_ptr(h), _ptr(Wd_q), _ptr(Wd_s), _ptr(bd), _ptr(cnt), _ptr(off), T, H, E,
                                    k, I, _ptr(o), path_code(path), _stream(stream)), "moe_down_mxfp4")
    return o[:T * k]


# ---------------------------------------------------------------------------
# FP8 W8A8
# ---------------------------------------------------------------------------
def workspace_bytes_fp8(T: int, H: int, E: int, k: int, I: int) -> int:
    return int(library().moe_workspace_bytes_fp8(T, H, E, k, I))


def alloc_workspace_fp8(T: int, H: int, E: int, k: int, I: int, device=None) -> torch.Tensor:
    n = workspace_bytes_fp8(T, H, E, k, I)
    return torch.empty(max(n, 256), dtype=torch.uint8, device=device or "cuda")


def moe_quantize_fp8(W, codes=None, scales=None, stream=None):
    """bf16 weights [E][K][N] (x.W form) -> (codes uint8 [E][N][K], scales float32 [E])."""
    _dims(W, "W", 3)
    E, K, N = W.shape
    _req(W, "W", (E, K, N), bf16=True)
    _req(codes, "codes", (E, N, K), torch.uint8)
    _req(scales, "scales", (E,), torch.float32)
    _dev(W)
    if codes is None:
        codes = torch.empty((E, N, K), dtype=torch.uint8, device=W.device)
    if scales is None:
        scales = torch.empty((E,), dtype=torch.float32, device=W.device)
    _dev(codes, scales)
    _check(library().moe_quantize_fp8(_ptr(W), E, K, N, _ptr(codes), _ptr(scales), _stream(stream)),
           "moe_quantize_fp8")
    return codes, scales


def moe_quantize_rows_fp8(a, codes=None, scales=None, stream=None):
    """bf16 rows [R][K] -> (codes uint8 [R][K], scales float32 [R])."""
    _dims(a, "a", 2)
    R, K = a.shape
    _req(a, "a", (R, K), bf16=True)
    _req(codes, "codes", (R, K), torch.uint8)
    _req(scales, "scales", (R,), torch.float32)
    _dev(a)
    if codes is None:
        codes = torch.empty((R, K), dtype=torch.uint8, device=a.device)
    if scales is None:
        scales = torch.empty((R,), dtype=torch.float32, device=a.device)
    _dev(codes, scales)
    _check(library().moe_quantize_rows_fp8(_ptr(a), R, K, _ptr(codes), _ptr(scales), _stream(stream)),
           "moe_quantize_rows_fp8")
    return codes, scales


def moe_forward_fp8(x, Wr, br, Wgu_q, Wgu_s, bgu, Wd_q, Wd_s, bd, k: int = 4, y=None, workspace=None,
                    topk_ids=None, topk_w=None, path="auto", stream=None):
    """moe_forward with FP8 W8A8 experts; returns y (bf16 [T,H])."""
    T, H, E = _route_args(x, Wr, br, k, topk_ids, topk_w)
    I = _fp8_experts(Wgu_q, Wgu_s, bgu, Wd_q, Wd_s, bd, E, H)
    _req(y, "y", (T, H), torch.bfloat16)
    _dev(x, Wr, br, Wgu_q, Wgu_s, bgu, Wd_q, Wd_s, bd)
    if y is None:
        y = torch.empty((T, H), dtype=torch.bfloat16, device=x.device)
    if workspace is None:
        workspace = alloc_workspace_fp8(T, H, E, k, I, x.device)
    _dev(y, workspace, topk_ids, topk_w)
    st = library().moe_forward_fp8_ex(_ptr(x), _ptr(Wr), _ptr(br), _ptr(Wgu_q), _ptr(Wgu_s), _ptr(bgu),
                                      _ptr(Wd_q), _ptr(Wd_s), _ptr(bd), T, H, E, k, I, _ptr(y), _ptr(topk_ids),
                                      _ptr(topk_w), _ptr(workspace), workspace.numel() * workspace.element_size(),
                                      path_code(path), _stream(stream))
    _check(st, "moe_forward_fp8")
    return y


def moe_gate_up_fp8(xq, sx, Wgu_q, Wgu_s, bgu, cnt, off, rows, k: int, h=None, path="auto", stream=None):
    """FP8 gate_up + bias + GLU from x codes and row scales; returns h (bf16 [T*k, I], permuted order)."""
    _dims(xq, "xq", 2)
    _dims(Wgu_q, "Wgu_q", 3)
    T, H = xq.shape
    E, I = Wgu_q.shape[0], Wgu_q.shape[1] // 2
    _req(xq, "xq", (T, H), torch.uint8)
    _req(sx, "sx", (T,), torch.float32)
    _req(Wgu_q, "Wgu_q", (E, 2 * I, H), torch.uint8)
    _req(Wgu_s, "Wgu_s", (E,), torch.float32)
    _req(bgu, "bgu", (E, 2 * I), bf16=True)
    _req(cnt, "cnt", (E,), torch.int32)
    _req(off, "off", (E + 1,), torch.int32)
    _req_rows(rows, "rows", T * k, None, torch.int32)
    _req_rows(h, "h", T * k, I, torch.bfloat16)
    _dev(xq, sx, Wgu_q, Wgu_s, bgu, cnt, off, rows)
    if h is None:
        h = torch.empty((T * k, I), dtype=torch.bfloat16, device=xq.device)
    _dev(h)
    _check(library().moe_gate_up_fp8(_ptr(xq), _ptr(sx), _ptr(Wgu_q), _ptr(Wgu_s), _ptr(bgu), _ptr(cnt), _ptr(off),
                                     _ptr(rows), T, H, E, k, I, _ptr(h), path_code(path), _stream(stream)),
           "moe_gate_up_fp8")
    return h


def moe_down_fp8(hq, sh, Wd_q, Wd_s, bd, cnt, off, T: int, k: int, o=None, path="auto", stream=None):
    """FP8 down + bias from h codes and row scales; returns o (float32 [T*k, H], permuted order)."""
    _dims(Wd_q, "Wd_q", 3)
    E, H, I = Wd_q.shape
    _req(Wd_q, "Wd_q", (E, H, I), torch.uint8)
    _req(Wd_s, "Wd_s", (E,), torch.float32)
    _req(bd, "bd", (E, H), bf16=True)
    _req(cnt, "cnt", (E,), torch.int32)
    _req(off, "off", (E + 1,), torch.int32)
    _req_rows(hq, "hq", T * k, I, torch.uint8)
    _req_rows(sh, "sh", T * k, None, torch.float32)
    _req_rows(o, "o", T * k, H, torch.float32)
    _dev(hq, sh, Wd_q, Wd_s, bd, cnt, off)
    if o is None:
        o = torch.empty((T * k, H), dtype=torch.float32, device=hq.device)
    _dev(o)
    _check(library().moe_down_fp8(_ptr(hq), _ptr(sh), _ptr(Wd_q), _ptr(Wd_s), _ptr(bd), _ptr(cnt), _ptr(off), T, H,
                                  E, k, I, _ptr(o), path_code(path), _stream(stream)), "moe_down_fp8")
    return o


def moe_forward_padded(x, Wr, br, Wgu, bgu, Wd, bd, k: int = 4, n_valid=None, y=None, workspace=None,
                       topk_ids=None, topk_w=None, expert_counts=None, path="auto", stream=None):
    """moe_forward over a batch whose rows from n_valid (a device int32
    tensor of one element, read when the call runs) are padding; returns y.
    expert_counts (device int32 [E]), if given, receives the per-expert loads."""
    T, H, E = _route_args(x, Wr, br, k, topk_ids, topk_w)
    I = _bf16_experts(Wgu, bgu, Wd, bd, E, H)
    _req(y, "y", (T, H), torch.bfloat16)
    _padded_args(n_valid, expert_counts, E)
    _dev(x, Wr, br, Wgu, bgu, Wd, bd)
    if y is None:
        y = torch.empty((T, H), dtype=torch.bfloat16, device=x.device)
    if workspace is None:
        workspace = alloc_workspace(T, H, E, k, I, x.device)
    _dev(y, workspace, topk_ids, topk_w, n_valid, expert_counts)
    st = library().moe_forward_padded(_ptr(x), _ptr(Wr), _ptr(br), _ptr(Wgu), _ptr(bgu), _ptr(Wd), _ptr(bd), T, H,
                                      E, k, I, _ptr(n_valid), _ptr(y), _ptr(topk_ids), _ptr(topk_w),
                                      _ptr(expert_counts), _ptr(workspace),
                                      workspace.numel() * workspace.element_size(), path_code(path), _stream(stream))
    _check(st, "moe_forward_padded")
    return y


def moe_forward_padded_mxfp4(x, Wr, br, Wgu_q, Wgu_s, bgu, Wd_q, Wd_s, bd, k: int = 4, n_valid=None, y=None,
                             workspace=None, topk_ids=None, topk_w=None, expert_counts=None, path="auto",
                             stream=None):
    """moe_forward_padded with MXFP4 expert weights; returns y (bf16 [T,H])."""
    T, H, E = _route_args(x, Wr, br, k, topk_ids, topk_w)
    I = _mxfp4_experts(Wgu_q, Wgu_s, bgu, Wd_q, Wd_s, bd, E, H)
    _req(y, "y", (T, H), torch.bfloat16)
    _padded_args(n_valid, expert_counts, E)
    _dev(x, Wr, br, Wgu_q, Wgu_s, bgu, Wd_q, Wd_s, bd)
    if y is None:
        y = torch.empty((T, H), dtype=torch.bfloat16, device=x.device)
    if workspace is None:
        workspace = alloc_workspace(T, H, E, k, I, x.device)
    _dev(y, workspace, topk_ids, topk_w, n_valid, expert_counts)
    st = library().moe_forward_padded_mxfp4(_ptr(x), _ptr(Wr), _ptr(br), _ptr(Wgu_q), _ptr(Wgu_s), _ptr(bgu),
                                            _ptr(Wd_q), _ptr(Wd_s), _ptr(bd), T, H, E, k, I, _ptr(n_valid), _ptr(y),
                                            _ptr(topk_ids), _ptr(topk_w), _ptr(expert_counts), _ptr(workspace),
                                            workspace.numel() * workspace.element_size(), path_code(path),
                                            _stream(stream))
    _check(st, "moe_forward_padded_mxfp4")
    return y


def moe_forward_padded_fp8(x, Wr, br, Wgu_q, Wgu_s, bgu, Wd_q, Wd_s, bd, k: int = 4, n_valid=None, y=None,
                           workspace=None, topk_ids=None, topk_w=None, expert_counts=None, path="auto", stream=None):
    """moe_forward_padded with FP8 W8A8 experts; returns y (bf16 [T,H])."""
    T, H, E = _route_args(x, Wr, br, k, topk_ids, topk_w)
    I = _fp8_experts(Wgu_q, Wgu_s, bgu, Wd_q, Wd_s, bd, E, H)
    _req(y, "y", (T, H), torch.bfloat16)
    _padded_args(n_valid, expert_counts, E)
    _dev(x, Wr, br, Wgu_q, Wgu_s, bgu, Wd_q, Wd_s, bd)
    if y is None:
        y = torch.empty((T, H), dtype=torch.bfloat16, device=x.device)
    if workspace is None:
        workspace = alloc_workspace_fp8(T, H, E, k, I, x.device)
    _dev(y, workspace, topk_ids, topk_w, n_valid, expert_counts)
    st = library().moe_forward_padded_fp8(_ptr(x), _ptr(Wr), _ptr(br), _ptr(Wgu_q), _ptr(Wgu_s), _ptr(bgu),
                                          _ptr(Wd_q), _ptr(Wd_s), _ptr(bd), T, H, E, k, I, _ptr(n_valid), _ptr(y),
                                          _ptr(topk_ids), _ptr(topk_w), _ptr(expert_counts), _ptr(workspace),
                                          workspace.numel() * workspace.element_size(), path_code(path),
                                          _stream(stream))
    _check(st, "moe_forward_padded_fp8")
    return y


def moe_forward_ep_mxfp4(x, Wr, br, Wgu_q_local, Wgu_s_local, bgu_local, Wd_q_local, Wd_s_local, bd_local,
                         e_begin: int, k: int = 4, y_partial=None, workspace=None, topk_ids=None, topk_w=None,
                         path="auto", stream=None):
    """moe_forward_ep with MXFP4 expert weights (the rank's n_local = Wgu_q_local.shape[0]
    experts from e_begin); returns y_partial (float32 [T,H])."""
    T, H, E = _route_args(x, Wr, br, k, topk_ids, topk_w)
    _dims(Wgu_q_local, "Wgu_q_local", 3)
    n_local = Wgu_q_local.shape[0]
    _local_experts(e_begin, n_local, E)
    I = _mxfp4_experts(Wgu_q_local, Wgu_s_local, bgu_local, Wd_q_local, Wd_s_local, bd_local, n_local, H)
    _req(y_partial, "y_partial", (T, H), torch.float32)
    _dev(x, Wr, br, Wgu_q_local, Wgu_s_local, bgu_local, Wd_q_local, Wd_s_local, bd_local)
    if y_partial is None:
        y_partial = torch.empty((T, H), dtype=torch.float32, device=x.device)
    if workspace is None:
        workspace = alloc_workspace(T, H, E, k, I, x.device)
    _dev(y_partial, workspace, topk_ids, topk_w)
    st = library().moe_forward_ep_mxfp4(_ptr(x), _ptr(Wr), _ptr(br), _ptr(Wgu_q_local), _ptr(Wgu_s_local),
                                        _ptr(bgu_local), _ptr(Wd_q_local), _ptr(Wd_s_local), _ptr(bd_local), T, H,
                                        E, k, I, e_begin, n_local, _ptr(y_partial), _ptr(topk_ids), _ptr(topk_w),
                                        _ptr(workspace), workspace.numel() * workspace.element_size(),
                                        path_code(path), _stream(stream))
    _check(st, "moe_forward_ep_mxfp4")
    return y_partial


def moe_forward_ep_fp8(x, Wr, br, Wgu_q_local, Wgu_s_local, bgu_local, Wd_q_local, Wd_s_local, bd_local,
                       e_begin: int, k: int = 4, y_partial=None, workspace=None, topk_ids=None, topk_w=None,
                       path="auto", stream=None):
    """moe_forward_ep with FP8 W8A8 experts (the rank's n_local = Wgu_q_local.shape[0]
    experts from e_begin); returns y_partial (float32 [T,H])."""
    T, H, E = _route_args(x, Wr, br, k, topk_ids, topk_w)
    _dims(Wgu_q_local, "Wgu_q_local", 3)
    n_local = Wgu_q_local.shape[0]
    _local_experts(e_begin, n_local, E)
    I = _fp8_experts(Wgu_q_local, Wgu_s_local, bgu_local, Wd_q_local, Wd_s_local, bd_local, n_local, H)
    _req(y_partial, "y_partial", (T, H), torch.float32)
    _dev(x, Wr, br, Wgu_q_local, Wgu_s_local, bgu_local, Wd_q_local, Wd_s_local, bd_local)
    if y_partial is None:
        y_partial = torch.empty((T, H), dtype=torch.float32, device=x.device)
    if workspace is None:
        workspace = alloc_workspace_fp8(T, H, E, k, I, x.device)
    _dev(y_partial, workspace, topk_ids, topk_w)
    st = library().moe_forward_ep_fp8(_ptr(x), _ptr(Wr), _ptr(br), _ptr(Wgu_q_local), _ptr(Wgu_s_local),
                                      _ptr(bgu_local), _ptr(Wd_q_local), _ptr(Wd_s_local), _ptr(bd_local), T, H, E,
                                      k, I, e_begin, n_local, _ptr(y_partial), _ptr(topk_ids), _ptr(topk_w),
                                      _ptr(workspace), workspace.numel() * workspace.element_size(),
                                      path_code(path), _stream(stream))
    _check(st, "moe_forward_ep_fp8")
    return y_partial


# ---------------------------------------------------------------------------
# residual addition and RMS norm in front of the block
# ---------------------------------------------------------------------------
def _norm_args(x, gamma, residual, residual_out, y):
    """x, residual, residual_out, y [T][H] and gamma [H], bf16; residual_out only beside a residual."""
    _dims(x, "x", 2)
    T, H = shape = x.shape
    bf16 = torch.bfloat16
    for t in (x, residual, residual_out, y):
        if t is not None and (t.shape != shape or t.dtype != bf16):
            for u, name in ((x, "x"), (residual, "residual"), (residual_out, "residual_out"), (y, "y")):
                _req(u, name, (T, H), bf16)
    _req(gamma, "gamma", (H,), bf16)
    if residual is None and residual_out is not None:
        raise MoEError("residual_out: given without a residual")
    return T, H


def moe_add_rmsnorm(x, gamma, residual=None, eps: float = 1e-5, y=None, residual_out=None, stream=None):
    """r = bf16(x + residual) and y = RMS norm of r times gamma; returns (y, r).

    y and residual_out may be the buffer of x or residual (in place).  Without a residual r is the tensor x itself; with
    y=x as well (a norm in place that no addition follows, such as a model's last) that tensor then holds y, and the
    rows as they were are gone."""
    T, H = _norm_args(x, gamma, residual, residual_out, y)
    here = _place(x, stream)
    if here is None:
        with _on(x, stream):
            return moe_add_rmsnorm(x, gamma, residual, eps, y, residual_out)
    if y is None:
        y = torch.empty_like(x)
    if residual is not None and residual_out is None:
        residual_out = torch.empty_like(x)
    a = _ats(x, residual, gamma, residual_out, y)
    st = library().moe_add_rmsnorm(a[0], a[1], a[2], T, H, eps, a[3], a[4], here)
    _check(st, "moe_add_rmsnorm")
    return y, x if residual is None else residual_out


def moe_add_rmsnorm_fp8(x, gamma, residual=None, eps: float = 1e-5, y=None, residual_out=None, codes=None, scales=None,
                        stream=None):
    """moe_add_rmsnorm that also quantises the normalised rows for the FP8 experts; returns (y, codes, scales, r):
    codes uint8 [T][H] and scales float32 [T] in moe_quantize_rows_fp8's format, from the unrounded values.  Without a
    residual r is x itself, which y must not overlap: the block behind these rows adds to it."""
    T, H = _norm_args(x, gamma, residual, residual_out, y)
    if residual is None and y is not None and abs(y.data_ptr() - x.data_ptr()) < 2 * T * H:
        raise MoEError("y overlaps x, the residual stream where no residual is given")
    _req(codes, "codes", (T, H), torch.uint8)
    _req(scales, "scales", (T,), torch.float32)
    here = _place(x, stream)
    if here is None:
        with _on(x, stream):
            return moe_add_rmsnorm_fp8(x, gamma, residual, eps, y, residual_out, codes, scales)
    if y is None:
        y = torch.empty_like(x)
    if residual is not None and residual_out is None:
        residual_out = torch.empty_like(x)
    if codes is None:
        codes = torch.empty((T, H), dtype=torch.uint8, device=x.device)
    if scales is None:
        scales = torch.empty((T,), dtype=torch.float32, device=x.device)
    a = _ats(x, residual, gamma, residual_out, y, codes, scales)
    st = library().moe_add_rmsnorm_fp8(a[0], a[1], a[2], T, H, eps, a[3], a[4], a[5], a[6], here)
    _check(st, "moe_add_rmsnorm_fp8")
    return y, codes, scales, x if residual is None else residual_out


def workspace_bytes_norm_fp8(T: int, H: int, E: int, k: int, I: int) -> int:
    return int(library().moe_workspace_bytes_norm_fp8(T, H, E, k, I))


def alloc_workspace_norm_fp8(T: int, H: int, E: int, k: int, I: int, device=None) -> torch.Tensor:
    n = workspace_bytes_norm_fp8(T, H, E, k, I)
    return torch.empty(max(n, 256), dtype=torch.uint8, device=device or "cuda")


def moe_forward_norm_fp8(x, gamma, Wr, br, Wgu_q, Wgu_s, bgu, Wd_q, Wd_s, bd, k: int = 4, residual=None,
                         eps: float = 1e-5, y=None, residual_out=None, workspace=None, topk_ids=None, topk_w=None,
                         path="auto", stream=None):
    """moe_add_rmsnorm_fp8 and the FP8 block on its rows, in one call; returns (y, r).  Without a residual r is x itself,
    which y must not overlap."""
    T, H = _norm_args(x, gamma, residual, residual_out, y)
    _, _, E = _route_args(x, Wr, br, k, topk_ids, topk_w)
    I = _fp8_experts(Wgu_q, Wgu_s, bgu, Wd_q, Wd_s, bd, E, H)
    here = _place(x, stream)
    if here is None:
        with _on(x, stream):
            return moe_forward_norm_fp8(x, gamma, Wr, br, Wgu_q, Wgu_s, bgu, Wd_q, Wd_s, bd, k, residual, eps, y,
                                        residual_out, workspace, topk_ids, topk_w, path)
    if y is None:
        y = torch.empty_like(x)
    if residual is not None and residual_out is None:
        residual_out = torch.empty_like(x)
    if workspace is None:
        workspace = alloc_workspace_norm_fp8(T, H, E, k, I, x.device)
    a = _ats(x, residual, gamma, Wr, br, Wgu_q, Wgu_s, bgu, Wd_q, Wd_s, bd, residual_out, y, topk_ids, topk_w, workspace)
    st = library().moe_forward_norm_fp8(a[0], a[1], a[2], eps, *a[3:11], T, H, E, k, I, *a[11:],
                                        workspace.numel() * workspace.element_size(), path_code(path), here)
    _check(st, "moe_forward_norm_fp8")
    return y, x if residual is None else residual_out


# ---------------------------------------------------------------------------
# 4-bit integer expert weights: codes uint8 [E][ceil(N/64)][K/32][1024] in tile
# order, scales bf16 and zero points uint8 (or None: 8) [E][ceil(K/G)][N]
# (gate_up: K = H, N = 2I; down: K = I, N = H); G = 32, 64 or 128 follows from
# the scales' shape
# ---------------------------------------------------------------------------
_GROUPS = (32, 64, 128)


def _int4_group(*pairs):
    """The group size with ceil(K / G) scales for every (K, scales) pair (several fit only where they mean the same)."""
    for G in _GROUPS:
        for K, n in pairs:
            if -(-K // G) != n:
                break
        else:
            return G
    raise MoEError("scales: no group size of " + ", ".join(map(str, _GROUPS)) + " gives "
                   + " and ".join(f"{n} scales for K={K}" for K, n in pairs))


def _int4_shape(n, K, N):
    return n, -(-N // 64), K // 32, 1024


def _int4_matrix(q, s, z, bias, names, n, K, N):
    groups = s.shape
    if (q.shape == (n, -(-N // 64), K // 32, 1024) and q.dtype is torch.uint8 and groups == (n, groups[1], N)
            and s.dtype is torch.bfloat16 and (z is None or (z.shape == groups and z.dtype is torch.uint8))
            and bias is not None and bias.shape == (n, N) and bias.element_size() == 2):
        return
    _req(q, names + "_q", _int4_shape(n, K, N), torch.uint8)
    _req(s, names + "_s", (n, s.shape[1], N), torch.bfloat16)
    _req(z, names + "_z", tuple(s.shape), torch.uint8)
    _req(bias, "b" + names[1:], (n, N), bf16=True)


def _int4_experts(Wgu_q, Wgu_s, Wgu_z, bgu, Wd_q, Wd_s, Wd_z, bd, n, H):
    """Codes, scales, zero points and biases of n experts; returns (I, G)."""
    _dims(Wgu_s, "Wgu_s", 3)
    _dims(Wd_s, "Wd_s", 3)
    I = Wgu_s.shape[2] // 2
    if H % 32 or I % 32:
        raise MoEError(f"int4 weights need H and I divisible by 32, got H={H}, I={I}")
    _int4_matrix(Wgu_q, Wgu_s, Wgu_z, bgu, "Wgu", n, H, 2 * I)
    _int4_matrix(Wd_q, Wd_s, Wd_z, bd, "Wd", n, I, H)
    return I, _int4_group((H, Wgu_s.shape[1]), (I, Wd_s.shape[1]))


def moe_quantize_int4(W, G: int = 64, zeros: bool = False, stream=None):
    """bf16 weights [E][K][N] (x.W form) -> (codes, scales, zero points or None), groups of G values of K."""
    _dims(W, "W", 3)
    E, K, N = W.shape
    _req(W, "W", (E, K, N), torch.bfloat16)
    if G not in _GROUPS:
        raise MoEError(f"G: expected one of {_GROUPS}, got {G}")
    _dev(W)
    with _on(W, stream):
        q = torch.empty(_int4_shape(E, K, N), dtype=torch.uint8, device=W.device)
        s = torch.empty((E, -(-K // G), N), dtype=torch.bfloat16, device=W.device)
        z = torch.empty((E, -(-K // G), N), dtype=torch.uint8, device=W.device) if zeros else None
        _check(library().moe_quantize_int4(_at(W), E, K, N, G, _at(q), _at(s), _at(z), _here(W)),
               "moe_quantize_int4")
    return q, s, z


def moe_pack_int4(codes, stream=None):
    """K-contiguous codes uint8 [E][N][K/2] (low nibble the even value) -> the tile order of the int4 calls."""
    _dims(codes, "codes", 3)
    E, N, K = codes.shape[0], codes.shape[1], 2 * codes.shape[2]
    _req(codes, "codes", (E, N, K // 2), torch.uint8)
    _dev(codes)
    with _on(codes, stream):
        q = torch.empty(_int4_shape(E, K, N), dtype=torch.uint8, device=codes.device)
        _check(library().moe_pack_int4(_at(codes), E, K, N, _at(q), _here(codes)), "moe_pack_int4")
    return q


def _scalar_or_at(v):
    return _at(v) if v is None or isinstance(v, torch.Tensor) else v


def _forward_int4(name, x, Wr, br, Wgu_q, Wgu_s, Wgu_z, bgu, Wd_q, Wd_s, Wd_z, bd, k, n, y, y_dtype, workspace, topk_ids,
                  topk_w, path, stream, before=(), between=()):
    """The int4 forwards: `before` y come further sizes or inputs, `between` the outputs and the workspace further
    outputs."""
    T, H, E = _route_args(x, Wr, br, k, topk_ids, topk_w)
    I, G = _int4_experts(Wgu_q, Wgu_s, Wgu_z, bgu, Wd_q, Wd_s, Wd_z, bd, E if n is None else n, H)
    _req(y, "y" if y_dtype == torch.bfloat16 else "y_partial", (T, H), y_dtype)
    here = _place(x, stream)
    if here is None:
        with _on(x, stream):
            return _forward_int4(name, x, Wr, br, Wgu_q, Wgu_s, Wgu_z, bgu, Wd_q, Wd_s, Wd_z, bd, k, n, y, y_dtype,
                                 workspace, topk_ids, topk_w, path, None, before, between)
    if y is None:
        y = torch.empty((T, H), dtype=y_dtype, device=x.device)
    if workspace is None:
        workspace = alloc_workspace(T, H, E, k, I, x.device)
    a = _ats(x, Wr, br, Wgu_q, Wgu_s, Wgu_z, bgu, Wd_q, Wd_s, Wd_z, bd, y, topk_ids, topk_w, workspace,
             *(t for t in before + between if isinstance(t, torch.Tensor)))
    st = getattr(library(), name)(*a[:11], T, H, E, k, I, G, *map(_scalar_or_at, before), *a[11:14],
                                  *map(_scalar_or_at, between), a[14], workspace.numel() * workspace.element_size(),
                                  path_code(path), here)
    _check(st, name.removesuffix("_ex"))
    return y


def moe_forward_int4(x, Wr, br, Wgu_q, Wgu_s, bgu, Wd_q, Wd_s, bd, k: int = 4, Wgu_z=None, Wd_z=None, y=None,
                     workspace=None, topk_ids=None, topk_w=None, path="auto", stream=None):
    """moe_forward with 4-bit integer expert weights; returns y (bf16 [T,H])."""
    return _forward_int4("moe_forward_int4_ex", x, Wr, br, Wgu_q, Wgu_s, Wgu_z, bgu, Wd_q, Wd_s, Wd_z, bd, k, None, y,
                         torch.bfloat16, workspace, topk_ids, topk_w, path, stream)


def moe_forward_padded_int4(x, Wr, br, Wgu_q, Wgu_s, bgu, Wd_q, Wd_s, bd, k: int = 4, Wgu_z=None, Wd_z=None,
                            n_valid=None, y=None, workspace=None, topk_ids=None, topk_w=None, expert_counts=None,
                            path="auto", stream=None):
    """moe_forward_padded with 4-bit integer expert weights; returns y (bf16 [T,H])."""
    _dims(Wr, "Wr", 2)
    _padded_args(n_valid, expert_counts, Wr.shape[0])
    return _forward_int4("moe_forward_padded_int4", x, Wr, br, Wgu_q, Wgu_s, Wgu_z, bgu, Wd_q, Wd_s, Wd_z, bd, k, None,
                         y, torch.bfloat16, workspace, topk_ids, topk_w, path, stream, before=(n_valid,),
                         between=(expert_counts,))


def moe_forward_ep_int4(x, Wr, br, Wgu_q_local, Wgu_s_local, bgu_local, Wd_q_local, Wd_s_local, bd_local, e_begin: int,
                        k: int = 4, Wgu_z_local=None, Wd_z_local=None, y_partial=None, workspace=None, topk_ids=None,
                        topk_w=None, path="auto", stream=None):
    """moe_forward_ep with 4-bit integer expert weights (the rank's n_local = Wgu_q_local.shape[0] experts from
    e_begin); returns y_partial (float32 [T,H])."""
    _dims(Wr, "Wr", 2)
    _dims(Wgu_q_local, "Wgu_q_local", 4)
    n_local = Wgu_q_local.shape[0]
    _local_experts(e_begin, n_local, Wr.shape[0])
    return _forward_int4("moe_forward_ep_int4", x, Wr, br, Wgu_q_local, Wgu_s_local, Wgu_z_local, bgu_local, Wd_q_local,
                         Wd_s_local, Wd_z_local, bd_local, k, n_local, y_partial, torch.float32, workspace, topk_ids,
                         topk_w, path, stream, before=(e_begin, n_local))


def _permutation(cnt, off, rows, E, S):
    _req(cnt, "cnt", (E,), torch.int32)
    _req(off, "off", (E + 1,), torch.int32)
    if rows is not None:
        _req_rows(rows, "rows", S, None, torch.int32)


def moe_gate_up_int4(x, Wgu_q, Wgu_s, bgu, cnt, off, rows, k: int, Wgu_z=None, h=None, path="auto", stream=None):
    """int4 gate_up + bias + GLU; returns h (bf16 [T*k, I], permuted order)."""
    _dims(x, "x", 2)
    _dims(Wgu_s, "Wgu_s", 3)
    T, H = x.shape
    E, I = Wgu_s.shape[0], Wgu_s.shape[2] // 2
    _req(x, "x", (T, H), bf16=True)
    _int4_matrix(Wgu_q, Wgu_s, Wgu_z, bgu, "Wgu", E, H, 2 * I)
    G = _int4_group((H, Wgu_s.shape[1]))
    _permutation(cnt, off, rows, E, T * k)
    _req_rows(h, "h", T * k, I, torch.bfloat16)
    here = _place(x, stream)
    if here is None:
        with _on(x, stream):
            return moe_gate_up_int4(x, Wgu_q, Wgu_s, bgu, cnt, off, rows, k, Wgu_z, h, path)
    if h is None:
        h = torch.empty((max(T * k, 1), I), dtype=torch.bfloat16, device=x.device)
    a = _ats(x, Wgu_q, Wgu_s, Wgu_z, bgu, cnt, off, rows, h)
    st = library().moe_gate_up_int4(*a[:8], T, H, E, k, I, G, a[8], path_code(path), here)
    _check(st, "moe_gate_up_int4")
    return h if h.shape[0] == T * k else h[:T * k]


def moe_down_int4(h, Wd_q, Wd_s, bd, cnt, off, T: int, k: int, Wd_z=None, o=None, path="auto", stream=None):
    """int4 down + bias; returns o (float32 [T*k, H], permuted order)."""
    _dims(h, "h", 2)
    _dims(Wd_s, "Wd_s", 3)
    E, H, I = Wd_s.shape[0], Wd_s.shape[2], h.shape[1]
    _int4_matrix(Wd_q, Wd_s, Wd_z, bd, "Wd", E, I, H)
    G = _int4_group((I, Wd_s.shape[1]))
    _permutation(cnt, off, None, E, T * k)
    _req_rows(h, "h", T * k, I, torch.bfloat16)
    _req_rows(o, "o", T * k, H, torch.float32)
    here = _place(h, stream)
    if here is None:
        with _on(h, stream):
            return moe_down_int4(h, Wd_q, Wd_s, bd, cnt, off, T, k, Wd_z, o, path)
    if o is None:
        o = torch.empty((max(T * k, 1), H), dtype=torch.float32, device=h.device)
    a = _ats(h, Wd_q, Wd_s, Wd_z, bd, cnt, off, o)
    st = library().moe_down_int4(*a[:7], T, H, E, k, I, G, a[7], path_code(path), here)
    _check(st, "moe_down_int4")
    return o if o.shape[0] == T * k else o[:T * k]


# ---------------------------------------------------------------------------
# MXFP4 on both sides: rows as codes uint8 [R][K/2] and scales uint8
# [ceil(K/128)][R][4], weights as in the MXFP4 section above
# ---------------------------------------------------------------------------
def _mx_rows(codes, scales, name, R, K):
    """Codes and scales of exactly R rows (the scales' layout goes by their number)."""
    _req(codes, name + "q", (R, K // 2), torch.uint8)
    _req(scales, "s" + name, (-(-K // 128), R, 4), torch.uint8)


def _mx_matrix(q, s, bias, names, E, K, N):
    _req(q, names + "_q", (E, N, K // 2), torch.uint8)
    _req(s, names + "_s", (E, K // 32, N), torch.uint8)
    _req(bias, "b" + names[1:], (E, N), bf16=True)


def moe_quantize_rows_mxfp4(a, codes=None, scales=None, stream=None):
    """bf16 rows [R][K] -> (codes uint8 [R][K/2], scales uint8 [ceil(K/128)][R][4])."""
    _dims(a, "a", 2)
    R, K = a.shape
    _req(a, "a", (R, K), torch.bfloat16)
    _req(codes, "codes", (R, K // 2), torch.uint8)
    _req(scales, "scales", (-(-K // 128), R, 4), torch.uint8)
    here = _place(a, stream)
    if here is None:
        with _on(a, stream):
            return moe_quantize_rows_mxfp4(a, codes, scales)
    if codes is None:
        codes = torch.empty((R, K // 2), dtype=torch.uint8, device=a.device)
    if scales is None:
        scales = torch.empty((-(-K // 128), R, 4), dtype=torch.uint8, device=a.device)
    at = _ats(a, codes, scales)
    _check(library().moe_quantize_rows_mxfp4(at[0], R, K, at[1], at[2], here), "moe_quantize_rows_mxfp4")
    return codes, scales


def moe_dequantize_rows_mxfp4(codes, scales, out=None, stream=None):
    """Codes and scales of rows -> their values, bf16 [R][K] (exact)."""
    _dims(codes, "codes", 2)
    R, K = codes.shape[0], 2 * codes.shape[1]
    _req(codes, "codes", (R, K // 2), torch.uint8)
    _req(scales, "scales", (-(-K // 128), R, 4), torch.uint8)
    _req(out, "out", (R, K), torch.bfloat16)
    here = _place(codes, stream)
    if here is None:
        with _on(codes, stream):
            return moe_dequantize_rows_mxfp4(codes, scales, out)
    if out is None:
        out = torch.empty((R, K), dtype=torch.bfloat16, device=codes.device)
    at = _ats(codes, scales, out)
    _check(library().moe_dequantize_rows_mxfp4(at[0], at[1], R, K, at[2], here), "moe_dequantize_rows_mxfp4")
    return out


def workspace_bytes_w4a4(T: int, H: int, E: int, k: int, I: int) -> int:
    return int(library().moe_workspace_bytes_w4a4(T, H, E, k, I))


def alloc_workspace_w4a4(T: int, H: int, E: int, k: int, I: int, device=None) -> torch.Tensor:
    n = workspace_bytes_w4a4(T, H, E, k, I)
    return torch.empty(max(n, 256), dtype=torch.uint8, device=device or "cuda")


def _forward_w4a4(name, x, Wr, br, Wgu_q, Wgu_s, bgu, Wd_q, Wd_s, bd, k, n, y, y_dtype, workspace, topk_ids, topk_w,
                  path, stream, before=(), between=()):
    """The forwards with MXFP4 on both sides: `before` y come further sizes or inputs, `between` the outputs and the
    workspace further outputs."""
    T, H, E = _route_args(x, Wr, br, k, topk_ids, topk_w)
    I = _mxfp4_experts(Wgu_q, Wgu_s, bgu, Wd_q, Wd_s, bd, E if n is None else n, H)
    _req(y, "y" if y_dtype == torch.bfloat16 else "y_partial", (T, H), y_dtype)
    here = _place(x, stream)
    if here is None:
        with _on(x, stream):
            return _forward_w4a4(name, x, Wr, br, Wgu_q, Wgu_s, bgu, Wd_q, Wd_s, bd, k, n, y, y_dtype, workspace,
                                 topk_ids, topk_w, path, None, before, between)
    if y is None:
        y = torch.empty((T, H), dtype=y_dtype, device=x.device)
    if workspace is None:
        workspace = alloc_workspace_w4a4(T, H, E, k, I, x.device)
    a = _ats(x, Wr, br, Wgu_q, Wgu_s, bgu, Wd_q, Wd_s, bd, y, topk_ids, topk_w, workspace,
             *(t for t in before + between if isinstance(t, torch.Tensor)))
    st = getattr(library(), name)(*a[:9], T, H, E, k, I, *map(_scalar_or_at, before), *a[9:12],
                                  *map(_scalar_or_at, between), a[12], workspace.numel() * workspace.element_size(),
                                  path_code(path), here)
    _check(st, name)
    return y


def moe_forward_w4a4(x, Wr, br, Wgu_q, Wgu_s, bgu, Wd_q, Wd_s, bd, k: int = 4, y=None, workspace=None, topk_ids=None,
                     topk_w=None, path="auto", stream=None):
    """moe_forward with MXFP4 weights and MXFP4 activations; returns y (bf16 [T,H])."""
    return _forward_w4a4("moe_forward_w4a4", x, Wr, br, Wgu_q, Wgu_s, bgu, Wd_q, Wd_s, bd, k, None, y, torch.bfloat16,
                         workspace, topk_ids, topk_w, path, stream)


def moe_forward_padded_w4a4(x, Wr, br, Wgu_q, Wgu_s, bgu, Wd_q, Wd_s, bd, k: int = 4, n_valid=None, y=None,
                            workspace=None, topk_ids=None, topk_w=None, expert_counts=None, path="auto", stream=None):
    """moe_forward_padded with MXFP4 weights and MXFP4 activations; returns y (bf16 [T,H])."""
    _dims(Wr, "Wr", 2)
    _padded_args(n_valid, expert_counts, Wr.shape[0])
    return _forward_w4a4("moe_forward_padded_w4a4", x, Wr, br, Wgu_q, Wgu_s, bgu, Wd_q, Wd_s, bd, k, None, y,
                         torch.bfloat16, workspace, topk_ids, topk_w, path, stream, before=(n_valid,),
                         between=(expert_counts,))


def moe_forward_ep_w4a4(x, Wr, br, Wgu_q_local, Wgu_s_local, bgu_local, Wd_q_local, Wd_s_local, bd_local, e_begin: int,
                        k: int = 4, y_partial=None, workspace=None, topk_ids=None, topk_w=None, path="auto",
                        stream=None):
    """moe_forward_ep with MXFP4 weights and MXFP4 activations (the rank's n_local = Wgu_q_local.shape[0] experts from
    e_begin); returns y_partial (float32 [T,H])."""
    _dims(Wr, "Wr", 2)
    _dims(Wgu_q_local, "Wgu_q_local", 3)
    n_local = Wgu_q_local.shape[0]
    _local_experts(e_begin, n_local, Wr.shape[0])
    return _forward_w4a4("moe_forward_ep_w4a4", x, Wr, br, Wgu_q_local, Wgu_s_local, bgu_local, Wd_q_local, Wd_s_local,
                         bd_local, k, n_local, y_partial, torch.float32, workspace, topk_ids, topk_w, path, stream,
                         before=(e_begin, n_local))


def moe_gate_up_w4a4(xq, sx, Wgu_q, Wgu_s, bgu, cnt, off, rows, k: int, hq=None, sh=None, path="auto", stream=None):
    """gate_up + bias + GLU of MXFP4 rows; returns (hq uint8 [T*k, I/2], sh uint8 [ceil(I/128), T*k, 4]): h as MXFP4
    rows, permuted order."""
    _dims(xq, "xq", 2)
    _dims(Wgu_q, "Wgu_q", 3)
    T, H = xq.shape[0], 2 * xq.shape[1]
    E, I = Wgu_q.shape[0], Wgu_q.shape[1] // 2
    _mx_rows(xq, sx, "x", T, H)
    _mx_matrix(Wgu_q, Wgu_s, bgu, "Wgu", E, H, 2 * I)
    _permutation(cnt, off, rows, E, T * k)
    _mx_rows(hq, sh, "h", T * k, I)
    here = _place(xq, stream)
    if here is None:
        with _on(xq, stream):
            return moe_gate_up_w4a4(xq, sx, Wgu_q, Wgu_s, bgu, cnt, off, rows, k, hq, sh, path)
    if hq is None:
        hq = torch.empty((T * k, I // 2), dtype=torch.uint8, device=xq.device)
    if sh is None:
        sh = torch.empty((-(-I // 128), T * k, 4), dtype=torch.uint8, device=xq.device)
    a = _ats(xq, sx, Wgu_q, Wgu_s, bgu, cnt, off, rows, hq, sh)
    st = library().moe_gate_up_w4a4(*a[:8], T, H, E, k, I, a[8], a[9], path_code(path), here)
    _check(st, "moe_gate_up_w4a4")
    return hq, sh


def moe_down_w4a4(hq, sh, Wd_q, Wd_s, bd, cnt, off, T: int, k: int, o=None, path="auto", stream=None):
    """down + bias of MXFP4 rows h; returns o (float32 [T*k, H], permuted order)."""
    _dims(hq, "hq", 2)
    _dims(Wd_q, "Wd_q", 3)
    E, H, I = Wd_q.shape[0], Wd_q.shape[1], 2 * hq.shape[1]
    _mx_rows(hq, sh, "h", T * k, I)
    _mx_matrix(Wd_q, Wd_s, bd, "Wd", E, I, H)
    _permutation(cnt, off, None, E, T * k)
    _req_rows(o, "o", T * k, H, torch.float32)
    here = _place(hq, stream)
    if here is None:
        with _on(hq, stream):
            return moe_down_w4a4(hq, sh, Wd_q, Wd_s, bd, cnt, off, T, k, o, path)
    if o is None:
        o = torch.empty((T * k, H), dtype=torch.float32, device=hq.device)
    a = _ats(hq, sh, Wd_q, Wd_s, bd, cnt, off, o)
    st = library().moe_down_w4a4(*a[:7], T, H, E, k, I, a[7], path_code(path), here)
    _check(st, "moe_down_w4a4")
    return o if o.shape[0] == T * k else o[:T * k]


# ---------------------------------------------------------------------------
# the backward pass of the block with bf16 weights
# ---------------------------------------------------------------------------
def workspace_bytes_backward(T: int, H: int, E: int, k: int, I: int) -> int:
    return int(library().moe_workspace_bytes_backward(T, H, E, k, I))


def alloc_workspace_backward(T: int, H: int, E: int, k: int, I: int, device=None) -> torch.Tensor:
    n = workspace_bytes_backward(T, H, E, k, I)
    return torch.empty(max(n, 256), dtype=torch.uint8, device=device or "cuda")


def moe_backward(dy, x, Wr, Wgu, bgu, Wd, bd, topk_ids, topk_w, router=True, experts=True, dx=None, dWr=None, dbr=None,
                 dWgu=None, dbgu=None, dWd=None, dbd=None, workspace=None, stream=None):
    """Gradients of moe_forward for the gradient dy of y; topk_ids and topk_w as the forward call left them.  Returns a
    dict of bf16 tensors: dx; dWr and dbr unless router is False; dWgu, dbgu, dWd and dbd unless experts is False
    (frozen weights: their products are not run).  No tokens: the weights' gradients are 0."""
    _dims(topk_ids, "topk_ids", 2)
    k = topk_ids.shape[1]
    _dims(Wr, "Wr", 2)
    E = Wr.shape[0]
    T, H, E = _route_args(x, Wr, None, k, topk_ids, topk_w)
    if topk_w is None:
        raise MoEError("topk_w: needed")
    I = _bf16_experts(Wgu, bgu, Wd, bd, E, H)
    bf16 = torch.bfloat16
    _req(dy, "dy", (T, H), bf16)
    shapes = {"dx": (T, H)}
    if router:
        shapes |= {"dWr": (E, H), "dbr": (E,)}
    if experts:
        shapes |= {"dWgu": (E, H, 2 * I), "dbgu": (E, 2 * I), "dWd": (E, I, H), "dbd": (E, H)}
    grads = {"dx": dx, "dWr": dWr, "dbr": dbr, "dWgu": dWgu, "dbgu": dbgu, "dWd": dWd, "dbd": dbd}
    for name, g in grads.items():
        if g is not None:
            if name not in shapes:
                raise MoEError(f"{name}: given, but not asked for")
            _req(g, name, shapes[name], bf16)
    here = _place(x, stream)
    if here is None:
        with _on(x, stream):
            return moe_backward(dy, x, Wr, Wgu, bgu, Wd, bd, topk_ids, topk_w, router, experts, dx, dWr, dbr, dWgu, dbgu,
                                dWd, dbd, workspace)
    for name, shape in shapes.items():
        if grads[name] is None:
            grads[name] = torch.empty(shape, dtype=bf16, device=x.device)
    if workspace is None:
        workspace = alloc_workspace_backward(T, H, E, k, I, x.device)
    a = _ats(x, dy, Wr, Wgu, bgu, Wd, bd, topk_ids, topk_w, *grads.values(), workspace)
    st = library().moe_backward(a[1], a[0], *a[2:9], T, H, E, k, I, *a[9:17], workspace.numel() * workspace.element_size(),
                                here)
    _check(st, "moe_backward")
    if T == 0:
        for name in shapes:
            grads[name].zero_()
    return {name: grads[name] for name in shapes}


# ---------------------------------------------------------------------------
# measurement probes (not part of the block)
# ---------------------------------------------------------------------------
def probe_mfma_bf16(iters: int, workgroups: int, out=None, stream=None):
    """Enqueue the MFMA rate probe; returns out (float32 [workgroups * 4], each
    2048 * iters when iters <= 8191).  Flops = workgroups * 4 * iters * 8 * 32768."""
    if out is None:
        out = torch.empty(workgroups * 4, dtype=torch.float32, device="cuda")
    _dev(out)
    _check(library().moe_probe_mfma_bf16(iters, workgroups, _ptr(out), _stream(stream)), "moe_probe_mfma_bf16")
    return out


def probe_read(buf, workgroups: int, out=None, stream=None):
    """Enqueue the streaming-read probe over buf (any dtype, contiguous, bytes % 16 == 0);
    returns out (int32 [workgroups * 4] holding uint32 XOR folds)."""
    _dev(buf)
    if out is None:
        out = torch.empty(workgroups * 4, dtype=torch.int32, device=buf.device)
    _dev(out)
    nbytes = buf.numel() * buf.element_size()
    _check(library().moe_probe_read(_ptr(buf), nbytes, workgroups, _ptr(out), _stream(stream)), "moe_probe_read")
    return out


def probe_mfma_dot_bf16(A, B, out=None, stream=None):
    """out[m][n] = A[m] . B[n] through the router's MFMA accumulation (bf16 A [M][K],
    B [16][K]; M % 16 == 0, K % 32 == 0); returns out (float32 [M][16])."""
    _dims(A, "A", 2)
    M, K = A.shape
    _req(A, "A", (M, K), bf16=True)
    _req(B, "B", (16, K), bf16=True)
    _req(out, "out", (M, 16), torch.float32)
    _dev(A, B)
    if out is None:
        out = torch.empty((M, 16), dtype=torch.float32, device=A.device)
    _dev(out)
    _check(library().moe_probe_mfma_dot_bf16(_ptr(A), _ptr(B), M, K, _ptr(out), _stream(stream)),
           "moe_probe_mfma_dot_bf16")
    return out

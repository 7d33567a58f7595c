"""Exact tiled attention (FlashAttention-style) for GB300 / sm_103a.

Thin ctypes binding over ``libfa.so`` (C ABI in ``include/fa.h``): it only
checks tensors, allocates outputs with torch on the current device, and
passes raw pointers plus the current CUDA stream. Every step of the forward
and backward runs in the library's CUDA kernels; there is no fallback path —
if the library is missing or no GPU is present, calls raise.
"""
from __future__ import annotations

import ctypes
import os
import struct

import torch

__all__ = [
    "FAError",
    "lib",
    "lib_path",
    "fwd",
    "bwd",
    "bwd_preprocess",
    "bwd_dkdv",
    "bwd_dq",
    "bwd_dq_d",
    "bwd_fuses_d",
    "bwd_workspace_bytes",
    "last_device_error",
    "debug_checks",
    "softmax_safe",
    "softmax_online",
    "attn_merge",
    "decode_paged",
    "decode_workspace_bytes",
    "fwd_host",
    "fwd_bwd_host",
    "softmax_host",
    "rope_tables",
    "rope_axes",
    "qk_norm_rope",
    "qk_norm_rope_bwd",
    "qk_norm_rope_bwd_workspace_bytes",
    "append_paged",
    "append_paged_q4",
    "decode_paged_q4",
    "decode_q4_splits",
    "extend_paged",
    "extend_paged_q4",
    "extend_workspace_bytes",
    "EXPORTED_SYMBOLS",
]

_HERE = os.path.dirname(os.path.abspath(__file__))
# FA_DEBUG_LIBRARY=1 selects the bounds-checked build (libfa_debug.so, made
# by build.build(debug=True)); it computes the same results.
_LIB_PATH = os.path.join(_HERE, "_lib",
                         "libfa_debug.so" if os.environ.get("FA_DEBUG_LIBRARY") == "1" else "libfa.so")
_lib = None

FA_STATUS = {
    0: "FA_OK",
    1: "FA_ERR_INVALID_ARG",
    2: "FA_ERR_UNSUPPORTED",
    3: "FA_ERR_MISALIGNED",
    4: "FA_ERR_CUDA",
    5: "FA_ERR_TIMEOUT",
    6: "FA_ERR_WORKSPACE",
    7: "FA_ERR_BAD_INDEX",
    8: "FA_ERR_BOUNDS",
}

EXPORTED_SYMBOLS = (
    "fa_fwd",
    "fa_fwd_gqa",
    "fa_bwd_workspace_bytes",
    "fa_bwd",
    "fa_bwd_gqa",
    "fa_bwd_preprocess",
    "fa_bwd_dkdv",
    "fa_bwd_dq",
    "fa_bwd_dq_d",
    "fa_bwd_fuses_d",
    "fa_last_device_error",
    "fa_selftest_wait_limit",
    "fa_status_string",
    "fa_version",
    "fa_bwd_noalloc",
    "fa_softmax_safe",
    "fa_softmax_online",
    "fa_attn_merge",
    "fa_decode_workspace_bytes",
    "fa_decode_paged",
    "fa_fwd_host",
    "fa_fwd_bwd_host",
    "fa_softmax_host",
    "fa_debug_checks",
    "fa_qk_norm_rope",
    "fa_qk_norm_rope_bwd_workspace_bytes",
    "fa_qk_norm_rope_bwd",
    "fa_append_paged",
    "fa_append_paged_q4",
    "fa_decode_q4_splits",
    "fa_decode_paged_q4",
    "fa_qk_norm_rope_axes",
    "fa_qk_norm_rope_axes_bwd",
    "fa_append_paged_axes",
    "fa_append_paged_q4_axes",
    "fa_extend_workspace_bytes",
    "fa_extend_paged",
    "fa_extend_paged_q4",
)


class Tensors(ctypes.Structure):
    """fa_tensors: addresses of one problem's q, k, v, dO, o, lse, dq, dk, dv."""
    _fields_ = [(n, ctypes.c_void_p) for n in ("q", "k", "v", "dO", "o", "lse", "dq", "dk", "dv")]


# Layouts of the argument structs (native alignment), packed for the call:
# building a ctypes structure field by field costs several times as much.
_HEADS, _TOKENS = "Pqqq", "Pqq"  # fa_heads, fa_tokens: address, strides
_NORM_ROPE_ARGS = struct.Struct("@" + 4 * _HEADS + "5P10if")
_NORM_ROPE_GRADS = struct.Struct("@" + 2 * _HEADS + "3PN")
_APPEND_ARGS = struct.Struct("@" + 4 * _TOKENS + "13P12if")
_DECODE_Q4_ARGS = struct.Struct("@10PN8if")
_ROPE_AXES = struct.Struct("@Pi64s")
_EXTEND_ARGS = struct.Struct("@11PN10if")
_ZERO_SKIPPED = 2  # FA_ZERO_SKIPPED


class FAError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {FA_STATUS.get(status, status)}")


def lib_path() -> str:
    return _LIB_PATH


def lib() -> ctypes.CDLL:
    """Load libfa.so (built by ``build.build()``); raises if it is missing."""
    global _lib
    if _lib is None:
        if not os.path.exists(_LIB_PATH):
            raise FAError(-1, f"libfa.so not built at {_LIB_PATH}; run exact_tiled_attention_24_gb300.build.build()")
        L = ctypes.CDLL(_LIB_PATH)
        vp, i, f, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
        L.fa_fwd.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, f, i, vp]
        L.fa_fwd.restype = i
        L.fa_fwd_gqa.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, f, i, vp]
        L.fa_fwd_gqa.restype = i
        L.fa_bwd_workspace_bytes.argtypes = [i, i, i, i]
        L.fa_bwd_workspace_bytes.restype = sz
        L.fa_bwd.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, i, i, i, i, f, i, vp]
        L.fa_bwd.restype = i
        L.fa_bwd_gqa.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, i, i, i, i, i, f, i, vp]
        L.fa_bwd_gqa.restype = i
        L.fa_bwd_preprocess.argtypes = [vp, vp, vp, i, i, i, i, vp]
        L.fa_bwd_preprocess.restype = i
        L.fa_bwd_dkdv.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, f, i, vp]
        L.fa_bwd_dkdv.restype = i
        L.fa_bwd_dq.argtypes = [vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, f, i, vp]
        L.fa_bwd_dq_d.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, f, i, vp]
        L.fa_bwd_dq_d.restype = i
        L.fa_bwd_fuses_d.argtypes = [i, i, i, i, i]
        L.fa_bwd_fuses_d.restype = i
        L.fa_bwd_dq.restype = i
        L.fa_bwd_noalloc.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, f, i, vp]
        L.fa_bwd_noalloc.restype = i
        L.fa_softmax_safe.argtypes = [vp, vp, ctypes.c_longlong, i, vp]
        L.fa_softmax_safe.restype = i
        L.fa_softmax_online.argtypes = [vp, vp, ctypes.c_longlong, i, vp]
        L.fa_softmax_online.restype = i
        L.fa_attn_merge.argtypes = [vp, vp, i, vp, vp, ctypes.c_longlong, i, vp]
        L.fa_attn_merge.restype = i
        L.fa_decode_workspace_bytes.argtypes = [i, i, i, i]
        L.fa_decode_workspace_bytes.restype = sz
        L.fa_decode_paged.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, sz, i, i, i, i, i, i, i, f, i, vp]
        L.fa_decode_paged.restype = i
        tp = ctypes.POINTER(Tensors)
        L.fa_fwd_host.argtypes = [tp, tp, i, i, i, i, i, f, i, i, vp]
        L.fa_fwd_host.restype = i
        L.fa_fwd_bwd_host.argtypes = [tp, tp, vp, sz, i, i, i, i, i, f, i, i, vp]
        L.fa_fwd_bwd_host.restype = i
        L.fa_softmax_host.argtypes = [vp, vp, vp, vp, ctypes.c_longlong, i, i, i, vp]
        L.fa_softmax_host.restype = i
        L.fa_qk_norm_rope.argtypes = [vp, vp]
        L.fa_qk_norm_rope.restype = i
        L.fa_qk_norm_rope_bwd_workspace_bytes.argtypes = [i, i, i]
        L.fa_qk_norm_rope_bwd_workspace_bytes.restype = sz
        L.fa_qk_norm_rope_bwd.argtypes = [vp, vp, vp]
        L.fa_qk_norm_rope_bwd.restype = i
        L.fa_append_paged.argtypes = [vp, vp]
        L.fa_append_paged.restype = i
        L.fa_append_paged_q4.argtypes = [vp, vp]
        L.fa_append_paged_q4.restype = i
        L.fa_decode_q4_splits.argtypes = [i] * 5
        L.fa_decode_q4_splits.restype = i
        L.fa_decode_paged_q4.argtypes = [vp, vp]
        L.fa_decode_paged_q4.restype = i
        L.fa_qk_norm_rope_axes.argtypes = [vp, vp, vp]
        L.fa_qk_norm_rope_axes.restype = i
        L.fa_qk_norm_rope_axes_bwd.argtypes = [vp, vp, vp, vp]
        L.fa_qk_norm_rope_axes_bwd.restype = i
        L.fa_append_paged_axes.argtypes = [vp, vp, vp]
        L.fa_append_paged_axes.restype = i
        L.fa_append_paged_q4_axes.argtypes = [vp, vp, vp]
        L.fa_append_paged_q4_axes.restype = i
        L.fa_extend_workspace_bytes.argtypes = [i] * 7
        L.fa_extend_workspace_bytes.restype = sz
        L.fa_extend_paged.argtypes = [vp, vp]
        L.fa_extend_paged.restype = i
        L.fa_extend_paged_q4.argtypes = [vp, vp]
        L.fa_extend_paged_q4.restype = i
        L.fa_last_device_error.argtypes = [vp]
        L.fa_last_device_error.restype = i
        L.fa_selftest_wait_limit.argtypes = [vp]
        L.fa_selftest_wait_limit.restype = i
        L.fa_status_string.argtypes = [i]
        L.fa_status_string.restype = ctypes.c_char_p
        L.fa_version.argtypes = []
        L.fa_version.restype = ctypes.c_char_p
        L.fa_debug_checks.argtypes = []
        L.fa_debug_checks.restype = i
        _lib = L
    return _lib


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else ctypes.c_void_p(0)


def _stream(device):
    # device: a torch.device. The address behind
    # torch.cuda.current_stream(device).cuda_stream, without the stream object
    # around it (2 us a call).
    index = device.index
    return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device() if index is None else index)


_Tensor = torch.Tensor

# Device type of every tensor the kernels touch. The library launches on the
# current CUDA device, so the tensors must live there as well.
_DEVICE_TYPE = "cuda"


def _on_device(t, name):
    """Raise unless t is a tensor on a device the library can launch on."""
    if not isinstance(t, _Tensor) or (dev := t.device).type != _DEVICE_TYPE:
        raise ValueError(f"{name} must be a {_DEVICE_TYPE.upper()} tensor")
    if _DEVICE_TYPE == "cuda" and dev.index != torch.cuda.current_device():
        raise ValueError(f"{name} is on {dev} but the current device is cuda:"
                         f"{torch.cuda.current_device()}: call under torch.cuda.device({dev})")


def _expect(t, name, shape, dtype, device):
    """Raise unless t is a contiguous `dtype` tensor of exactly `shape` on
    `device`: a buffer the kernels read or write in full, so a smaller one
    would be overrun."""
    if not (isinstance(t, _Tensor) and t.dtype is dtype and t.shape == shape and t.is_contiguous()
            and t.device == device):
        raise ValueError(f"{name}: expected a contiguous {dtype} tensor of shape {tuple(shape)} on {device}")


def _expect_workspace(ws, device):
    """The workspace's size is checked by the library; here its place."""
    if not isinstance(ws, torch.Tensor) or ws.device != device or not ws.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on {device}")


def _check(status, where):
    if status != 0:
        raise FAError(status, where)


def _check_inputs(q, k, v, *rest):
    """q (and o, dO in rest): [B, H, N, d]; k, v: [B, Hkv, N, d] with Hkv dividing H.
    Returns Hkv."""
    if q.dim() != 4 or k.dim() != 4 or v.dim() != 4:
        raise ValueError("expected [B, H, N, d] tensors")
    B, H, N, d = q.shape
    Hkv = k.shape[1]
    _on_device(q, "q")
    for t in (q, k, v) + rest:
        if t.device.type != _DEVICE_TYPE:
            raise ValueError("tensors must be on a CUDA device")
        if t.dtype != torch.bfloat16:
            raise ValueError("tensors must be bfloat16")
        if not t.is_contiguous():
            raise ValueError("tensors must be contiguous")
        if t.device != q.device:
            raise ValueError("tensors must be on one device")
    for t in rest:
        if t.shape != q.shape:
            raise ValueError("o and dO must have q's shape")
    if k.shape != (B, Hkv, N, d) or v.shape != k.shape or Hkv < 1 or H % Hkv:
        raise ValueError("k and v must be [B, Hkv, N, d] with Hkv dividing q's head count")
    return Hkv


def _scale(d, scale):
    return (1.0 / d ** 0.5) if scale is None else float(scale)


def fwd(q, k, v, causal=False, scale=None, out=None, lse=None):
    """o, lse = softmax(scale·q kᵀ [causal]) v and its per-row log-sum-exp.

    k and v may hold fewer heads than q (grouped-query attention): query head
    h then uses K/V head h // (H // Hkv)."""
    Hkv = _check_inputs(q, k, v)
    B, H, N, d = q.shape
    if out is not None:
        _expect(out, "out", q.shape, torch.bfloat16, q.device)
    if lse is not None:
        _expect(lse, "lse", (B, H, N), torch.float32, q.device)
    o = torch.empty_like(q) if out is None else out
    lse_t = torch.empty((B, H, N), dtype=torch.float32, device=q.device) if lse is None else lse
    _check(lib().fa_fwd_gqa(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse_t), B, H, Hkv, N, d,
                            _scale(d, scale), int(bool(causal)), _stream(q.device)), "fa_fwd_gqa")
    return o, lse_t


def bwd_workspace_bytes(B, H, N, d) -> int:
    return int(lib().fa_bwd_workspace_bytes(B, H, N, d))


def bwd(q, k, v, o, lse, do, causal=False, scale=None, workspace=None):
    """dq, dk, dv of o = softmax(scale·q kᵀ [causal]) v for the output gradient do
    (dk, dv shaped like k, v; with grouped-query heads they sum over the group)."""
    Hkv = _check_inputs(q, k, v, o, do)
    B, H, N, d = q.shape
    _expect(lse, "lse", (B, H, N), torch.float32, q.device)
    ws_bytes = bwd_workspace_bytes(B, H, N, d)
    if workspace is None:
        workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=q.device)
    _expect_workspace(workspace, q.device)
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    _check(lib().fa_bwd_gqa(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(do), _ptr(lse), _ptr(dq),
                            _ptr(dk), _ptr(dv), _ptr(workspace), workspace.numel() * workspace.element_size(),
                            B, H, Hkv, N, d, _scale(d, scale), int(bool(causal)), _stream(q.device)),
           "fa_bwd_gqa")
    return dq, dk, dv


def bwd_preprocess(o, do, Dvec):
    """Dvec = rowsum(do * o) (fp32 [B, H, N])."""
    _check_inputs(o, o, o, do)
    B, H, N, d = o.shape
    _expect(Dvec, "Dvec", (B, H, N), torch.float32, o.device)
    _check(lib().fa_bwd_preprocess(_ptr(o), _ptr(do), _ptr(Dvec), B, H, N, d, _stream(o.device)),
           "fa_bwd_preprocess")


def bwd_dkdv(q, k, v, do, lse, Dvec, dk, dv, causal=False, scale=None):
    """dk, dv (bf16, written in place) from the recomputed P and dS."""
    Hkv = _check_inputs(q, k, v, do)
    B, H, N, d = q.shape
    _expect(lse, "lse", (B, H, N), torch.float32, q.device)
    _expect(Dvec, "Dvec", (B, H, N), torch.float32, q.device)
    _expect(dk, "dk", k.shape, torch.bfloat16, q.device)
    _expect(dv, "dv", k.shape, torch.bfloat16, q.device)
    _check(lib().fa_bwd_dkdv(_ptr(q), _ptr(k), _ptr(v), _ptr(do), _ptr(lse), _ptr(Dvec), _ptr(dk),
                             _ptr(dv), B, H, Hkv, N, d, _scale(d, scale), int(bool(causal)),
                             _stream(q.device)), "fa_bwd_dkdv")


def bwd_dq_d(q, k, v, o, do, lse, Dvec, dq, causal=False, scale=None):
    """dq (bf16) and Dvec = rowsum(do * o) (fp32), both written in place, by
    the dQ sweep alone (no preprocess); bwd_dkdv can then read Dvec."""
    Hkv = _check_inputs(q, k, v, o, do)
    B, H, N, d = q.shape
    _expect(lse, "lse", (B, H, N), torch.float32, q.device)
    _expect(Dvec, "Dvec", (B, H, N), torch.float32, q.device)
    _expect(dq, "dq", q.shape, torch.bfloat16, q.device)
    _check(lib().fa_bwd_dq_d(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(do), _ptr(lse), _ptr(Dvec), _ptr(dq),
                             B, H, Hkv, N, d, _scale(d, scale), int(bool(causal)), _stream(q.device)),
           "fa_bwd_dq_d")


def bwd_fuses_d(B, H, Hkv, N, d):
    """True when bwd() runs the dQ sweep with D first and the dK/dV sweep
    after it for these sizes on the current device (see fa_bwd_fuses_d)."""
    return bool(lib().fa_bwd_fuses_d(int(B), int(H), int(Hkv), int(N), int(d)))


def bwd_dq(q, k, v, do, lse, Dvec, dq, causal=False, scale=None):
    """dq (bf16, written in place) from the recomputed dS."""
    Hkv = _check_inputs(q, k, v, do)
    B, H, N, d = q.shape
    _expect(lse, "lse", (B, H, N), torch.float32, q.device)
    _expect(Dvec, "Dvec", (B, H, N), torch.float32, q.device)
    _expect(dq, "dq", q.shape, torch.bfloat16, q.device)
    _check(lib().fa_bwd_dq(_ptr(q), _ptr(k), _ptr(v), _ptr(do), _ptr(lse), _ptr(Dvec), _ptr(dq),
                           B, H, Hkv, N, d, _scale(d, scale), int(bool(causal)), _stream(q.device)),
           "fa_bwd_dq")


def selftest_wait_limit(device=None) -> None:
    """Enqueue the error-path self-test on the current stream: a wait that
    nothing satisfies gives up after its limit, so the next
    last_device_error() returns 5 (FA_ERR_TIMEOUT)."""
    dev = torch.device("cuda" if device is None else device)
    _check(lib().fa_selftest_wait_limit(_stream(dev)), "fa_selftest_wait_limit")


def debug_checks() -> bool:
    """True when the loaded library is the bounds-checked FA_DEBUG build."""
    return bool(lib().fa_debug_checks())


def last_device_error(device=None) -> int:
    """Synchronise the current stream and return (and clear) the device error status."""
    dev = torch.device("cuda" if device is None else device)
    return int(lib().fa_last_device_error(_stream(dev)))


def _softmax(name, x, out):
    if x.device.type != _DEVICE_TYPE or x.dtype != torch.float32 or not x.is_contiguous() or x.dim() < 1:
        raise ValueError("x must be a contiguous float32 CUDA tensor")
    _on_device(x, "x")
    n = x.shape[-1]
    rows = x.numel() // n if n else 0
    if out is not None:
        _expect(out, "out", x.shape, torch.float32, x.device)
    y = torch.empty_like(x) if out is None else out
    _check(getattr(lib(), name)(_ptr(x), _ptr(y), rows, n, _stream(x.device)), name)
    return y


def softmax_safe(x, out=None):
    """Softmax over the last dimension of fp32 x, three passes per row."""
    return _softmax("fa_softmax_safe", x, out)


def softmax_online(x, out=None):
    """Softmax over the last dimension of fp32 x, two passes per row (online)."""
    return _softmax("fa_softmax_online", x, out)


def attn_merge(o_parts, lse_parts, out=None, lse=None):
    """Combine partial attention results: o_parts [S, rows, d] fp32, lse_parts
    [S, rows] fp32 -> (o [rows, d] bf16, lse [rows] fp32)."""
    _on_device(o_parts, "o_parts")
    S, rows, d = o_parts.shape
    if o_parts.dtype != torch.float32 or lse_parts.dtype != torch.float32:
        raise ValueError("o_parts and lse_parts must be float32")
    if lse_parts.shape != (S, rows) or not (o_parts.is_contiguous() and lse_parts.is_contiguous()):
        raise ValueError("lse_parts must be a contiguous [S, rows] tensor beside contiguous o_parts")
    if lse_parts.device != o_parts.device:
        raise ValueError("o_parts and lse_parts must be on one device")
    if out is not None:
        _expect(out, "out", (rows, d), torch.bfloat16, o_parts.device)
    if lse is not None:
        _expect(lse, "lse", (rows,), torch.float32, o_parts.device)
    o = torch.empty((rows, d), dtype=torch.bfloat16, device=o_parts.device) if out is None else out
    lse_t = torch.empty((rows,), dtype=torch.float32, device=o_parts.device) if lse is None else lse
    _check(lib().fa_attn_merge(_ptr(o_parts), _ptr(lse_parts), S, _ptr(o), _ptr(lse_t), rows, d,
                               _stream(o_parts.device)), "fa_attn_merge")
    return o, lse_t


def decode_workspace_bytes(B, H, d, n_splits) -> int:
    return int(lib().fa_decode_workspace_bytes(B, H, d, n_splits))


def decode_paged(q, k_cache, v_cache, block_table, seq_lens, n_splits=1, scale=None, workspace=None,
                 out=None, lse=None):
    """One decode step: q [B, H, d] bf16 against the paged cache k_cache,
    v_cache [num_blocks, Hkv, block_size, d] bf16, with block_table
    [B, max_blocks] int32 and seq_lens [B] int32. Returns (o [B, H, d] bf16,
    lse [B, H] fp32)."""
    B, H, d = q.shape
    num_blocks, Hkv, bs, dk = k_cache.shape
    _on_device(q, "q")
    for t in (q, k_cache, v_cache):
        if t.device != q.device or t.dtype != torch.bfloat16 or not t.is_contiguous():
            raise ValueError("q, k_cache, v_cache must be contiguous bfloat16 CUDA tensors on one device")
    if v_cache.shape != k_cache.shape or dk != d:
        raise ValueError("k_cache and v_cache must be [num_blocks, Hkv, block_size, d]")
    if block_table.dtype != torch.int32 or seq_lens.dtype != torch.int32 or block_table.dim() != 2 \
            or block_table.shape[0] != B or seq_lens.shape != (B,) or not block_table.is_contiguous():
        raise ValueError("block_table [B, max_blocks] and seq_lens [B] must be int32")
    _expect(block_table, "block_table", block_table.shape, torch.int32, q.device)
    _expect(seq_lens, "seq_lens", (B,), torch.int32, q.device)
    ws_bytes = decode_workspace_bytes(B, H, d, n_splits)
    if workspace is None:
        workspace = torch.empty(max(ws_bytes, 16), dtype=torch.uint8, device=q.device)
    _expect_workspace(workspace, q.device)
    if out is not None:
        _expect(out, "out", q.shape, torch.bfloat16, q.device)
    if lse is not None:
        _expect(lse, "lse", (B, H), torch.float32, q.device)
    o = torch.empty_like(q) if out is None else out
    lse_t = torch.empty((B, H), dtype=torch.float32, device=q.device) if lse is None else lse
    _check(lib().fa_decode_paged(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_table), _ptr(seq_lens),
                                 _ptr(o), _ptr(lse_t), _ptr(workspace),
                                 workspace.numel() * workspace.element_size(), B, H, Hkv, d, num_blocks, bs,
                                 block_table.shape[1], _scale(d, scale), n_splits, _stream(q.device)),
           "fa_decode_paged")
    return o, lse_t


_HOST_NAMES = ("q", "k", "v", "dO", "o", "lse", "dq", "dk", "dv")


def _tensors(ts: dict, on_cuda: bool, shapes: dict, names):
    """Check one side's tensors (shape, dtype, contiguity, device kind) and
    pack their addresses into a Tensors struct."""
    st = Tensors()
    for n in names:
        t = ts.get(n)
        if t is None:
            raise ValueError(f"missing tensor {n!r}")
        want_dtype = torch.float32 if n == "lse" else torch.bfloat16
        if tuple(t.shape) != shapes[n] or t.dtype != want_dtype or not t.is_contiguous():
            raise ValueError(f"{n}: expected a contiguous {want_dtype} tensor of shape {shapes[n]}")
        if (t.device.type == _DEVICE_TYPE) != on_cuda or (not on_cuda and t.device.type != "cpu"):
            raise ValueError(f"{n}: expected a {'CUDA' if on_cuda else 'host'} tensor")
        if on_cuda and t.device != ts[names[0]].device:
            raise ValueError(f"{n}: the device tensors must be on one device")
        setattr(st, n, t.data_ptr())
    return st


def _host_shapes(q, k):
    B, H, N, d = q.shape
    Hkv = k.shape[1]
    qs, kvs = (B, H, N, d), (B, Hkv, N, d)
    return {"q": qs, "k": kvs, "v": kvs, "dO": qs, "o": qs, "lse": (B, H, N), "dq": qs, "dk": kvs,
            "dv": kvs}


def fwd_host(host: dict, dev: dict, causal=False, scale=None, n_chunks=0):
    """Forward from host memory: host["q"], ["k"], ["v"] (CPU, ideally
    pinned) are copied into dev["q"], ["k"], ["v"] (CUDA), the forward runs
    there, and dev["o"], ["lse"] are copied back into host["o"], ["lse"], in
    n_chunks pipelined slices (0: the library's default). Asynchronous on the
    current stream: synchronise it before reading host["o"]."""
    names = ("q", "k", "v", "o", "lse")
    q, k = host["q"], host["k"]
    B, H, N, d = q.shape
    Hkv = k.shape[1]
    shapes = _host_shapes(q, k)
    h = _tensors(host, False, shapes, names)
    dv = _tensors(dev, True, shapes, names)
    _on_device(dev["q"], 'dev["q"]')
    _check(lib().fa_fwd_host(ctypes.byref(h), ctypes.byref(dv), B, H, Hkv, N, d, _scale(d, scale),
                             int(bool(causal)), int(n_chunks), _stream(dev["q"].device)), "fa_fwd_host")


def fwd_bwd_host(host: dict, dev: dict, workspace, causal=False, scale=None, n_chunks=0):
    """Forward and backward from host memory: as fwd_host, plus host["dO"]
    in and host["dq"], ["dk"], ["dv"] out; workspace is a CUDA buffer of
    bwd_workspace_bytes(B, H, N, d) bytes."""
    q, k = host["q"], host["k"]
    B, H, N, d = q.shape
    Hkv = k.shape[1]
    shapes = _host_shapes(q, k)
    h = _tensors(host, False, shapes, _HOST_NAMES)
    dv = _tensors(dev, True, shapes, _HOST_NAMES)
    _on_device(dev["q"], 'dev["q"]')
    _expect_workspace(workspace, dev["q"].device)
    _check(lib().fa_fwd_bwd_host(ctypes.byref(h), ctypes.byref(dv), _ptr(workspace),
                                 workspace.numel() * workspace.element_size(), B, H, Hkv, N, d,
                                 _scale(d, scale), int(bool(causal)), int(n_chunks),
                                 _stream(dev["q"].device)), "fa_fwd_bwd_host")


def softmax_host(x_host, y_host, x_dev, y_dev, online=True, n_chunks=0):
    """Row softmax from host memory: x_host (CPU fp32, ideally pinned) is
    copied into x_dev, normalised into y_dev and copied back into y_host, in
    n_chunks pipelined slices of rows (0: the library's default).
    Asynchronous on the current stream: synchronise it before reading y_host."""
    for t, dev_side in ((x_host, False), (y_host, False), (x_dev, True), (y_dev, True)):
        place_ok = t.device == x_dev.device if dev_side else t.device.type == "cpu"
        if not place_ok or t.dtype != torch.float32 or not t.is_contiguous() or t.shape != x_host.shape:
            raise ValueError("x_host, y_host (CPU) and x_dev, y_dev (CUDA) must be contiguous float32 "
                             "tensors of one shape")
    _on_device(x_dev, "x_dev")
    n = x_host.shape[-1]
    rows = x_host.numel() // n if n else 0
    _check(lib().fa_softmax_host(_ptr(x_host), _ptr(y_host), _ptr(x_dev), _ptr(y_dev), rows, n,
                                 int(bool(online)), int(n_chunks), _stream(x_dev.device)), "fa_softmax_host")


# ---------------------------------- norms, rotation, paged appends, 4-bit cache

def rope_tables(n_pos, rot, base=10000.0, device=None):
    """cos, sin [n_pos, rot/2] fp32 of the usual rotary angles, position ·
    base^(-2i/rot), formed in 64 bits (a far position's angle has no correct
    digits left in 32) and rounded once. Make them once and keep them."""
    if n_pos < 1 or rot < 2 or rot % 2:
        raise ValueError("n_pos must be at least 1 and rot even")
    device = torch.device(_DEVICE_TYPE) if device is None else device
    freq = float(base) ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=device) / rot)
    angle = torch.arange(n_pos, dtype=torch.float64, device=device)[:, None] * freq
    return angle.cos().float(), angle.sin().float()


def rope_axes(sections, in_turn=False) -> bytes:
    """The axis of each rotated pair, for the `axes` of qk_norm_rope and the
    appends: sections[a] pairs belong to axis a (up to four axes, rot/2 pairs in
    all), one section after another, or with in_turn dealt 0, 1, 2, 0, 1, 2 ...
    while an axis has pairs left. Any other assignment is a bytes of rot/2 axis
    numbers."""
    left = [int(n) for n in sections]
    if not 1 <= len(left) <= 4 or min(left) < 0 or sum(left) < 1:
        raise ValueError("sections: one to four axes, numbers of pairs")
    if not in_turn:
        return bytes(a for a, n in enumerate(left) for _ in range(n))
    return bytes(a for turn in range(max(left)) for a, n in enumerate(left) if turn < n)


_BF16, _F32, _I32, _U8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8


def _rows(t, name, shape, device, out=False):
    """(address, strides but the last) of t, a bf16 tensor of `shape` on
    `device` whose last dimension is contiguous and whose rows sit on 16-byte
    boundaries (for an output: no two rows overlapping); raises otherwise."""
    if not isinstance(t, _Tensor) or t.shape != shape or t.dtype is not _BF16 or t.device != device:
        raise ValueError(f"{name}: expected a {_BF16} tensor of shape {tuple(shape)} on {device}")
    strides = t.stride()
    if len(strides) == 3:  # the appends' case, without the loops
        a, b, last = strides
        if last == 1 and not (a | b) & 7 and (not out or t.is_contiguous()):
            return t.data_ptr(), a, b
    *lead, last = strides
    odd = 0
    for s in lead:
        odd |= s
    if last != 1 or odd & 7:  # a dimension of one element has no stride to speak of
        lead = [s if n > 1 else 0 for s, n in zip(lead, shape)]
        if last != 1 or any([s & 7 for s in lead]):
            raise ValueError(f"{name}: the last dimension must be contiguous and the other strides multiples of 8")
    if out and not t.is_contiguous():
        need = shape[-1]
        for s, n in sorted((s, n) for s, n in zip(lead, shape) if n > 1):
            if s < need:
                raise ValueError(f"{name}: an output's rows must not overlap")
            need = s * n
    return t.data_ptr(), *lead


def _made(shape, device):
    """A new contiguous bf16 tensor and its address and strides, as _rows gives them."""
    t = torch.empty(shape, dtype=_BF16, device=device)
    if len(shape) == 4:
        _, H, N, d = shape
        return t, (t.data_ptr(), H * N * d, N * d, d)
    _, H, d = shape
    return t, (t.data_ptr(), H * d, d)


def _rope_args(cos, sin, q_weight, k_weight, d, device):
    """Check tables and weights; returns their addresses, and rot, n_pos, weight_fp32."""
    rot = n_pos = w32 = cp = sp = qp = kp = 0
    if cos is not None or sin is not None:
        if not isinstance(cos, torch.Tensor) or cos.dim() != 2 or sin is None:
            raise ValueError("cos and sin go together, [n_pos, rot/2] both")
        n_pos, rot = cos.shape
        rot *= 2
        if n_pos < 1 or rot < 1:
            raise ValueError("cos and sin must not be empty")
        _expect(cos, "cos", cos.shape, _F32, device)
        _expect(sin, "sin", cos.shape, _F32, device)
        cp, sp = cos.data_ptr(), sin.data_ptr()
    if k_weight is not None:
        w32 = int(isinstance(k_weight, torch.Tensor) and k_weight.dtype is _F32)
        _expect(k_weight, "k_weight", (d,), _F32 if w32 else _BF16, device)
        kp = k_weight.data_ptr()
        if q_weight is not None:  # both of one dtype
            _expect(q_weight, "q_weight", (d,), k_weight.dtype, device)
            qp = q_weight.data_ptr()
    return (cp, sp), (qp, kp), rot, n_pos, w32


def _pack_axes(axes, positions, n_axes, rot):
    """The packed fa_rope_axes of checked positions [n_axes, ...]."""
    if type(axes) is not bytes:
        try:
            axes = bytes(list(axes))
        except TypeError:
            raise ValueError("axes: a bytes (or sequence) of axis numbers") from None
    if len(axes) != rot // 2:
        raise ValueError("axes: one axis number for each of the rot/2 pairs")
    return _ROPE_AXES.pack(positions.data_ptr(), n_axes, axes)


def _norm_rope_args(q, k, a, b, cos, sin, positions, q_weight, k_weight, eps, interleaved, names, out, axes):
    """Check qk_norm_rope's arguments; a and b are the tensors beside q and k
    (the outputs, made here if None, or their gradients). Returns a, b, the
    packed fa_norm_rope_args and the packed fa_rope_axes (None without axes)."""
    if not isinstance(q, torch.Tensor) or not isinstance(k, torch.Tensor) or q.dim() != 4 or k.dim() != 4:
        raise ValueError("expected [B, H, N, d] tensors")
    B, H, N, d = qs = q.shape
    Hkv = k.shape[1]
    ks = (B, Hkv, N, d)
    dev = q.device
    _on_device(q, "q")
    if (q_weight is None) != (k_weight is None):
        raise ValueError("q_weight and k_weight go together")
    if cos is None and q_weight is None:
        raise ValueError("neither weights (norm) nor cos and sin (rotation) given")
    tables, weights, rot, n_pos, w32 = _rope_args(cos, sin, q_weight, k_weight, d, dev)
    per_batch = pp = 0
    packed = None
    if axes is not None:
        if not isinstance(positions, torch.Tensor) or positions.dim() < 2 or cos is None:
            raise ValueError("axes need cos, sin and positions [axes, N] or [axes, B, N]")
        per_batch = int(positions.dim() == 3)
        _expect(positions, "positions", (positions.shape[0], B, N) if per_batch else (positions.shape[0], N), _I32, dev)
        packed = _pack_axes(axes, positions, positions.shape[0], rot)
    elif positions is not None:
        per_batch = int(isinstance(positions, torch.Tensor) and positions.dim() == 2)
        _expect(positions, "positions", (B, N) if per_batch else (N,), _I32, dev)
        pp = positions.data_ptr()
    elif rot and n_pos < N:
        raise ValueError("cos and sin must have a row for every token")
    qr, kr = _rows(q, "q", qs, dev), _rows(k, "k", ks, dev)
    a, ar = _made(qs, dev) if a is None else (a, _rows(a, names[0], qs, dev, out))
    b, br = _made(ks, dev) if b is None else (b, _rows(b, names[1], ks, dev, out))
    return a, b, _NORM_ROPE_ARGS.pack(*qr, *kr, *ar, *br, *tables, pp, *weights, B, H, Hkv, N, d, rot, n_pos,
                                      per_batch, w32, 1 if interleaved else 0, eps), packed


def qk_norm_rope(q, k, cos=None, sin=None, positions=None, q_weight=None, k_weight=None, eps=1e-6,
                 interleaved=False, q_out=None, k_out=None, axes=None):
    """Per-head norm (with q_weight, k_weight [d], bf16 or fp32) and position
    rotation (with cos, sin [n_pos, rot/2] fp32) of q [B, H, N, d] and k
    [B, Hkv, N, d], in one pass. Returns (q_out, k_out), contiguous unless
    given: what fwd takes.

    q, k and given outputs may be strided views whose last dimension is
    contiguous, such as those of a packed projection; an output may be its
    input. positions: int32 [N] or [B, N], the token's row of the tables
    (default: token n is at position n). interleaved pairs dimensions
    (2i, 2i + 1), else (i, i + rot/2).

    axes (rope_axes' bytes: the axis of each pair) gives tokens a position on
    each of up to four axes, such as time, height and width: positions are then
    int32 [axes, N] or [axes, B, N], and a pair turns by its own axis's."""
    q_out, k_out, args, packed = _norm_rope_args(q, k, q_out, k_out, cos, sin, positions, q_weight, k_weight, eps,
                                                 interleaved, ("q_out", "k_out"), True, axes)
    if packed is None:
        _check(lib().fa_qk_norm_rope(args, _stream(q.device)), "fa_qk_norm_rope")
    else:
        _check(lib().fa_qk_norm_rope_axes(args, packed, _stream(q.device)), "fa_qk_norm_rope_axes")
    return q_out, k_out


def qk_norm_rope_bwd_workspace_bytes(B, N, d) -> int:
    return int(lib().fa_qk_norm_rope_bwd_workspace_bytes(B, N, d))


def qk_norm_rope_bwd(dq_out, dk_out, q, k, cos=None, sin=None, positions=None, q_weight=None, k_weight=None,
                     eps=1e-6, interleaved=False, dq=None, dk=None, workspace=None, axes=None):
    """Gradient of qk_norm_rope for the output gradients dq_out, dk_out (bwd's
    dq and dk). Returns (dq, dk, dq_weight, dk_weight): dq and dk contiguous
    bf16 unless given (strided views are allowed, as in qk_norm_rope), the
    weight gradients fp32 [d] whatever the weights' type (None without
    weights; q and k are then not read and may be None). axes as in
    qk_norm_rope."""
    if q_weight is None and k_weight is None:
        q, k = dq_out, dk_out
    if dq_out is None or dk_out is None:
        raise ValueError("expected output gradients of both q and k")
    _, _, args, packed = _norm_rope_args(q, k, dq_out, dk_out, cos, sin, positions, q_weight, k_weight, eps,
                                         interleaved, ("dq_out", "dk_out"), False, axes)
    dev = q.device
    dq, dqr = _made(q.shape, dev) if dq is None else (dq, _rows(dq, "dq", q.shape, dev, True))
    dk, dkr = _made(k.shape, dev) if dk is None else (dk, _rows(dk, "dk", k.shape, dev, True))
    dqw = dkw = None
    wp = qp = kp = ws_bytes = 0
    if q_weight is not None:
        B, _, N, d = q.shape
        dqw, dkw = torch.empty((d,), dtype=_F32, device=dev), torch.empty((d,), dtype=_F32, device=dev)
        if workspace is None:
            ws_bytes = lib().fa_qk_norm_rope_bwd_workspace_bytes(B, N, d)
            workspace = torch.empty(ws_bytes, dtype=_U8, device=dev)
        else:
            _expect_workspace(workspace, dev)
            ws_bytes = workspace.numel() * workspace.element_size()
        wp = workspace.data_ptr()
        qp, kp = dqw.data_ptr(), dkw.data_ptr()
    grads = _NORM_ROPE_GRADS.pack(*dqr, *dkr, qp, kp, wp, ws_bytes)
    if packed is None:
        _check(lib().fa_qk_norm_rope_bwd(args, grads, _stream(dev)), "fa_qk_norm_rope_bwd")
    else:
        _check(lib().fa_qk_norm_rope_axes_bwd(args, packed, grads, _stream(dev)), "fa_qk_norm_rope_axes_bwd")
    return dq, dk, dqw, dkw


def _append(entry, k, v, caches, values, block_table, positions, requests, cos, sin, q, q_weight, k_weight, eps,
            interleaved, q_out, rope_positions, axes):
    """Check an append's arguments (the caches' own by the caller) and call it."""
    if not isinstance(k, torch.Tensor) or k.dim() != 3:
        raise ValueError("expected k and v [T, Hkv, d]")
    T, Hkv, d = shape = k.shape
    dev = k.device
    _on_device(k, "k")
    kr, vr = _rows(k, "k", shape, dev), _rows(v, "v", shape, dev)
    H, qr, qor, zero = 0, (0, 0, 0), (0, 0, 0), 0
    if q is not None:
        if not isinstance(q, torch.Tensor) or q.dim() != 3:
            raise ValueError("expected q [T, H, d]")
        H = q.shape[1]
        qr = _rows(q, "q", (T, H, d), dev)
        if (q_weight is None) != (k_weight is None):
            raise ValueError("q_weight and k_weight go together")
        if q_out is None:
            q_out, qor = _made((T, H, d), dev)
            zero = _ZERO_SKIPPED
        else:
            qor = _rows(q_out, "q_out", (T, H, d), dev, True)
    elif q_weight is not None or q_out is not None:
        raise ValueError("q_weight and q_out need q")
    if not isinstance(block_table, torch.Tensor) or block_table.dim() != 2:
        raise ValueError("block_table must be [B, max_blocks] int32")
    B, max_blocks = block_table.shape
    _expect(block_table, "block_table", (B, max_blocks), _I32, dev)
    _expect(positions, "positions", (T,), _I32, dev)
    rp = 0
    if requests is not None:
        _expect(requests, "requests", (T,), _I32, dev)
        rp = requests.data_ptr()
    elif T > B:
        raise ValueError("more tokens than requests: say which request each token belongs to")
    tables, weights, rot, n_pos, w32 = _rope_args(cos, sin, q_weight, k_weight, d, dev)
    packed = None
    if rope_positions is not None:
        if cos is None or not isinstance(rope_positions, _Tensor):
            raise ValueError("rope_positions need cos and sin")
        if axes is None:
            _expect(rope_positions, "rope_positions", (T,), _I32, dev)
            packed = _pack_axes(bytes(rot // 2), rope_positions, 1, rot)
        else:
            n_axes = rope_positions.shape[0] if rope_positions.dim() else 0
            _expect(rope_positions, "rope_positions", (n_axes, T), _I32, dev)
            packed = _pack_axes(axes, rope_positions, n_axes, rot)
    elif axes is not None:
        raise ValueError("axes need rope_positions [axes, T]")
    k_cache = caches[0]
    ks, vs, kv, vv = (caches[1].data_ptr(), caches[3].data_ptr(), *values) if len(caches) == 4 else (0, 0, 0, 0)
    args = _APPEND_ARGS.pack(
        *qr, *kr, *vr, *qor, k_cache.data_ptr(), caches[-1 if len(caches) == 2 else 2].data_ptr(), ks, vs, kv, vv,
        block_table.data_ptr(), positions.data_ptr(), rp, *tables, *weights, T, B, H, Hkv, d, k_cache.shape[0],
        k_cache.shape[2], max_blocks, rot, n_pos, w32 | zero, 1 if interleaved else 0, eps)
    if packed is None:
        _check(getattr(lib(), entry)(args, _stream(dev)), entry)
    else:
        entry += "_axes"
        _check(getattr(lib(), entry)(args, packed, _stream(dev)), entry)
    return q_out


def _expect_cache(t, name, Hkv, last, dtype, device):
    """Check one tensor [num_blocks, Hkv, block_size, last] of a cache."""
    if not isinstance(t, torch.Tensor) or t.dim() != 4:
        raise ValueError(f"{name}: expected a tensor of four dimensions")
    n, _, bs, _ = t.shape
    _expect(t, name, (n, Hkv, bs, last), dtype, device)


def append_paged(k, v, k_cache, v_cache, block_table, positions, requests=None, cos=None, sin=None, q=None,
                 q_weight=None, k_weight=None, eps=1e-6, interleaved=False, q_out=None, rope_positions=None, axes=None):
    """Write new tokens' keys (after norm and rotation, as in qk_norm_rope)
    and values k, v [T, Hkv, d] into the paged cache k_cache, v_cache
    [num_blocks, Hkv, block_size, d] bf16, in place. Token t goes to position
    positions[t] of request requests[t] (int32 [T] both; requests=None: token
    t is request t's), through block_table [B, max_blocks] int32; a negative
    request or position marks padding, which is skipped.

    With q [T, H, d] the tokens' queries get the same norm and rotation;
    returns them ([T, H, d]: decode_paged's q), else None. Rows of skipped
    tokens are zeros in a q_out made here and stay as they were in a given one.
    k, v, q and q_out may be strided views, such as those of a packed
    projection.

    rope_positions turns keys and queries by positions of their own, apart from
    the slots: int32 [T], or with axes (as in qk_norm_rope) [axes, T]."""
    if not isinstance(k, torch.Tensor) or k.dim() != 3:
        raise ValueError("expected k and v [T, Hkv, d]")
    _expect_cache(k_cache, "k_cache", k.shape[1], k.shape[2], _BF16, k.device)
    _expect(v_cache, "v_cache", k_cache.shape, _BF16, k.device)
    return _append("fa_append_paged", k, v, (k_cache, v_cache), None, block_table, positions, requests, cos, sin, q,
                   q_weight, k_weight, eps, interleaved, q_out, rope_positions, axes)


def _expect_q4_cache(k_cache, k_scale, v_cache, v_scale, Hkv, d, device):
    """Check a 4-bit cache's codes and (step, centre) pairs."""
    if not isinstance(k_cache, _Tensor) or k_cache.dim() != 4:
        raise ValueError("k_cache: expected a tensor of four dimensions")
    n, _, bs, _ = k_cache.shape
    codes, pairs = (n, Hkv, bs, d // 2), (n, Hkv, bs, d // 64, 2)
    _expect(k_cache, "k_cache", codes, _U8, device)
    _expect(v_cache, "v_cache", codes, _U8, device)
    _expect(k_scale, "k_scale", pairs, _BF16, device)
    _expect(v_scale, "v_scale", pairs, _BF16, device)


def append_paged_q4(k, v, k_cache, k_scale, v_cache, v_scale, block_table, positions, requests=None, cos=None,
                    sin=None, q=None, q_weight=None, k_weight=None, eps=1e-6, interleaved=False, q_out=None,
                    k_values=None, v_values=None, rope_positions=None, axes=None):
    """append_paged into a cache held in 4 bits: k_cache, v_cache
    [num_blocks, Hkv, block_size, d/2] uint8 codes and k_scale, v_scale
    [num_blocks, Hkv, block_size, d/64, 2] bf16 (step, centre) of each group
    of 64 dimensions (see fa_append_paged_q4). k_values, v_values [T, Hkv, d]
    bf16, contiguous, if given, receive the values that the cache now holds
    (fwd takes them as [B, Hkv, N, d]: transposed and copied)."""
    if not isinstance(k, torch.Tensor) or k.dim() != 3:
        raise ValueError("expected k and v [T, Hkv, d]")
    _expect_q4_cache(k_cache, k_scale, v_cache, v_scale, k.shape[1], k.shape[2], k.device)
    values = (0, 0)
    if k_values is not None or v_values is not None:
        _expect(k_values, "k_values", k.shape, _BF16, k.device)
        _expect(v_values, "v_values", k.shape, _BF16, k.device)
        values = (k_values.data_ptr(), v_values.data_ptr())
    return _append("fa_append_paged_q4", k, v, (k_cache, k_scale, v_cache, v_scale), values, block_table, positions,
                   requests, cos, sin, q, q_weight, k_weight, eps, interleaved, q_out, rope_positions, axes)


def decode_q4_splits(B, H, Hkv, block_size, max_blocks) -> int:
    """The n_splits that decode_paged_q4 takes for n_splits=0."""
    return int(lib().fa_decode_q4_splits(B, H, Hkv, block_size, max_blocks))


def decode_paged_q4(q, k_cache, k_scale, v_cache, v_scale, block_table, seq_lens, n_splits=0, scale=None,
                    workspace=None, out=None, lse=None):
    """decode_paged over a cache held in 4 bits (append_paged_q4's): q
    [B, H, d] bf16, block_table [B, max_blocks] and seq_lens [B] int32.
    n_splits=0 takes decode_q4_splits(...); the workspace is
    decode_workspace_bytes(B, H, d, n_splits) bytes (none for one split).
    Returns (o [B, H, d] bf16, lse [B, H] fp32)."""
    if not isinstance(q, torch.Tensor) or q.dim() != 3:
        raise ValueError("expected q [B, H, d]")
    B, H, d = shape = q.shape
    dev = q.device
    _on_device(q, "q")
    _expect(q, "q", shape, _BF16, dev)
    if not isinstance(k_cache, torch.Tensor) or k_cache.dim() != 4:
        raise ValueError("k_cache and v_cache must be [num_blocks, Hkv, block_size, d/2] uint8")
    num_blocks, Hkv, bs, _ = k_cache.shape
    _expect_q4_cache(k_cache, k_scale, v_cache, v_scale, Hkv, d, dev)
    if not isinstance(block_table, torch.Tensor) or block_table.dim() != 2:
        raise ValueError("block_table must be [B, max_blocks] int32")
    max_blocks = block_table.shape[1]
    _expect(block_table, "block_table", (B, max_blocks), _I32, dev)
    _expect(seq_lens, "seq_lens", (B,), _I32, dev)
    L = lib()
    if n_splits == 0:
        n_splits = L.fa_decode_q4_splits(B, H, Hkv, bs, max_blocks)
    wp = ws_bytes = 0
    if workspace is not None:
        _expect_workspace(workspace, dev)
        wp, ws_bytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    elif n_splits > 1:
        ws_bytes = L.fa_decode_workspace_bytes(B, H, d, n_splits)
        workspace = torch.empty(ws_bytes, dtype=_U8, device=dev)
        wp = workspace.data_ptr()
    if out is None:
        out = torch.empty_like(q)
    else:
        _expect(out, "out", shape, _BF16, dev)
    if lse is None:
        lse = torch.empty((B, H), dtype=_F32, device=dev)
    else:
        _expect(lse, "lse", (B, H), _F32, dev)
    args = _DECODE_Q4_ARGS.pack(
        q.data_ptr(), k_cache.data_ptr(), k_scale.data_ptr(), v_cache.data_ptr(), v_scale.data_ptr(),
        block_table.data_ptr(), seq_lens.data_ptr(), out.data_ptr(), lse.data_ptr(), wp, ws_bytes, B, H, Hkv, d,
        num_blocks, bs, max_blocks, n_splits, _scale(d, scale))
    _check(L.fa_decode_paged_q4(args, _stream(dev)), "fa_decode_paged_q4")
    return out, lse


def extend_workspace_bytes(T, B, H, Hkv, d, block_size, max_blocks) -> int:
    return int(lib().fa_extend_workspace_bytes(T, B, H, Hkv, d, block_size, max_blocks))


def _extend(entry, q, caches, block_table, seq_lens, q_starts, causal, scale, workspace, out, lse):
    """Check a chunk call's arguments (the caches' own by the caller) and call it."""
    T, H, d = shape = q.shape
    dev = q.device
    _on_device(q, "q")
    _expect(q, "q", shape, _BF16, dev)
    if not isinstance(block_table, _Tensor) or block_table.dim() != 2:
        raise ValueError("block_table must be [B, max_blocks] int32")
    B, max_blocks = table_shape = block_table.shape
    _expect(block_table, "block_table", table_shape, _I32, dev)
    _expect(seq_lens, "seq_lens", (B,), _I32, dev)
    _expect(q_starts, "q_starts", (B + 1,), _I32, dev)
    num_blocks, Hkv, bs, _ = caches[0].shape
    L = lib()
    if workspace is None:
        ws_bytes = L.fa_extend_workspace_bytes(T, B, H, Hkv, d, bs, max_blocks)
        workspace = torch.empty(ws_bytes, dtype=_U8, device=dev)
    else:
        _expect_workspace(workspace, dev)
        ws_bytes = workspace.numel() * workspace.element_size()
    zero = out is None and lse is None
    if out is None:
        out = torch.empty_like(q)
    else:
        _expect(out, "out", shape, _BF16, dev)
    if lse is None:
        lse = torch.empty((T, H), dtype=_F32, device=dev)
    else:
        _expect(lse, "lse", (T, H), _F32, dev)
    kc, ks, vc, vs = ((caches[0].data_ptr(), 0, caches[1].data_ptr(), 0) if len(caches) == 2
                      else [t.data_ptr() for t in caches])
    args = _EXTEND_ARGS.pack(
        q.data_ptr(), kc, ks, vc, vs, block_table.data_ptr(), seq_lens.data_ptr(), q_starts.data_ptr(), out.data_ptr(),
        lse.data_ptr(), workspace.data_ptr(), ws_bytes, T, B, H, Hkv, d, num_blocks, bs, max_blocks,
        1 if causal else 0, 1 if zero else 0, _scale(d, scale))
    _check(getattr(L, entry)(args, _stream(dev)), entry)
    return out, lse


def extend_paged(q, k_cache, v_cache, block_table, seq_lens, q_starts, causal=True, scale=None, workspace=None,
                 out=None, lse=None):
    """Attention of chunks of new tokens over a paged cache: q [T, H, d] bf16
    (append_paged's queries), request after request; request b's tokens are
    rows q_starts[b] .. q_starts[b + 1] - 1 (int32 [B + 1]) and the last of its
    seq_lens[b] cached tokens (int32 [B], the new ones included). A token sees
    the keys up to its own position, or with causal=False all of its request's.
    Caches and block_table as in decode_paged; the workspace is
    extend_workspace_bytes(...) bytes. Returns (o [T, H, d] bf16, lse [T, H]
    fp32).

    A request whose two starts are out of order or range, or that begins before
    the end of an earlier one, is taken for empty (and reported by
    last_device_error). Rows of no request (theirs, those before q_starts[0] and
    from q_starts[B] on) are o = 0, lse = -inf where both outputs are made here
    and stay as they were where either is given. The lengths are read on the
    device: a captured call may be replayed with others."""
    if not isinstance(q, torch.Tensor) or q.dim() != 3:
        raise ValueError("expected q [T, H, d]")
    if not isinstance(k_cache, torch.Tensor) or k_cache.dim() != 4:
        raise ValueError("k_cache and v_cache must be [num_blocks, Hkv, block_size, d]")
    _expect_cache(k_cache, "k_cache", k_cache.shape[1], q.shape[2], _BF16, q.device)
    _expect(v_cache, "v_cache", k_cache.shape, _BF16, q.device)
    return _extend("fa_extend_paged", q, (k_cache, v_cache), block_table, seq_lens, q_starts, causal, scale, workspace,
                   out, lse)


def extend_paged_q4(q, k_cache, k_scale, v_cache, v_scale, block_table, seq_lens, q_starts, causal=True, scale=None,
                    workspace=None, out=None, lse=None):
    """extend_paged over a cache held in 4 bits (append_paged_q4's). Keys and
    values are read back in bf16, rounded once: what append_paged_q4 hands out
    as k_values and v_values. (decode_paged_q4 holds them exactly, and keeps 16
    bits of a weight where chunks keep bf16's 8, as fwd does.)"""
    if not isinstance(q, torch.Tensor) or q.dim() != 3:
        raise ValueError("expected q [T, H, d]")
    if not isinstance(k_cache, torch.Tensor) or k_cache.dim() != 4:
        raise ValueError("k_cache and v_cache must be [num_blocks, Hkv, block_size, d/2] uint8")
    _expect_q4_cache(k_cache, k_scale, v_cache, v_scale, k_cache.shape[1], q.shape[2], q.device)
    return _extend("fa_extend_paged_q4", q, (k_cache, k_scale, v_cache, v_scale), block_table, seq_lens, q_starts,
                   causal, scale, workspace, out, lse)

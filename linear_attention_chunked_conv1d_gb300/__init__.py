"""GB300-native chunked gated-delta-rule prefill (GDN / KDA) with a causal conv1d front end.

Thin Python binding of the C ABI in ``include/linattn.h`` (``liblinattn.so``): every function
here only marshals torch CUDA tensors into raw device pointers, sizes and the current CUDA
stream, then calls the C entry point of the same name. All arithmetic runs in the library's
CUDA kernels; there is no CPU or PyTorch fallback, and importing fails loudly when the library
has not been built (``python -m linear_attention_chunked_conv1d_gb300.build``).
"""
from __future__ import annotations

import ctypes
import math
import os

import torch

from .build import LIB_PATH

__all__ = [
    "LinAttnError", "LA_F32", "LA_BF16", "abi_version", "last_error", "device_status",
    "conv1d_silu_prefill", "conv1d_silu_prefill_varlen", "conv1d_silu_l2_prefill",
    "l2norm_heads",
    "prefill_workspace_bytes", "gdn_prefill_batched", "gdn_prefill_varlen",
    "gdn_prefill_varlen_noalloc", "kda_prefill",
    "gated_scan", "gated_scan_backward", "gated_scan_step", "gated_scan_workspace_bytes",
    "gated_scan_saved_bytes", "conv1d_silu_backward", "conv1d_silu_backward_workspace_bytes",
    "w4_matvec", "w4_quantize", "LA_W4_MAX_ROWS",
    "layernorm_rows", "layernorm_rows_backward", "layernorm_rows_backward_workspace_bytes",
    "linear", "linear_saved_bytes", "linear_backward", "linear_backward_workspace_bytes",
    "gated_ffn", "gated_ffn_saved_bytes", "gated_ffn_backward",
    "gated_ffn_backward_workspace_bytes", "LA_ACTIVATIONS",
    "pointer_array", "library_path",
]

LA_OK, LA_ERR_ARG, LA_ERR_COUNT, LA_ERR_UNSUPPORTED, LA_ERR_CUDA = 0, 1, 2, 3, 4
LA_F32, LA_BF16 = 0, 1
LA_DEV_BAD_SEQLENS, LA_DEV_TIMEOUT = 1, 2
LA_W4_MAX_ROWS = 32
# activations of linear and gated_ffn (LA_ACT_*)
LA_ACTIVATIONS = {"none": 0, "relu": 1, "gelu": 2, "gelu_tanh": 3, "silu": 4}
_CODES = {LA_ERR_ARG: "LA_ERR_ARG", LA_ERR_COUNT: "LA_ERR_COUNT",
          LA_ERR_UNSUPPORTED: "LA_ERR_UNSUPPORTED", LA_ERR_CUDA: "LA_ERR_CUDA"}


class LinAttnError(RuntimeError):
    """A linattn call returned a non-zero status; ``code`` holds it."""

    def __init__(self, code: int, msg: str):
        super().__init__(f"{_CODES.get(code, code)}: {msg}")
        self.code = code


_u64, _i64, _i32, _f32, _vp, _sz = (ctypes.c_uint64, ctypes.c_int64, ctypes.c_int,
                                    ctypes.c_float, ctypes.c_void_p, ctypes.c_size_t)

_SIGS = {
    "la_abi_version": ([], ctypes.c_int),
    "la_last_error": ([], ctypes.c_char_p),
    "la_device_status": ([_u64], ctypes.c_int),
    "la_conv1d_silu_prefill": ([_vp, _vp, _vp, _vp, _vp, _i32, _i32, _i32, _i32, _i64, _i64,
                                _i32, _u64], ctypes.c_int),
    "la_conv1d_silu_prefill_varlen": ([_vp, _vp, _vp, _vp, _vp, _vp, _i32, _i32, _i32, _i32,
                                       _i32, _i64, _i64, _i32, _u64], ctypes.c_int),
    "la_l2norm_heads": ([_vp, _i32, _i32, _i32, _i64, _f32, _i32, _u64], ctypes.c_int),
    "la_conv1d_silu_l2_prefill": ([_vp, _vp, _vp, _vp, _vp, _vp, _i32, _i32, _i32, _i32, _i32,
                                   _i32, _i32, _f32, _i64, _i64, _i32, _u64], ctypes.c_int),
    "la_prefill_workspace_bytes": ([_i32, _i32, _i32, _i32, _i32, _i32, _i32], _sz),
    "la_gdn_prefill_batched": ([_vp, _vp, _vp, _vp, _vp, _vp, _vp, _i32, _i32, _i32, _i32, _i32,
                                _i32, _i32, _i64, _i64, _i64, _f32, _i32, _vp, _sz, _u64],
                               ctypes.c_int),
    "la_gdn_prefill_varlen": ([_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i32, _i32, _i32, _i32,
                               _i32, _i32, _i32, _i32, _i64, _i64, _i64, _f32, _i32, _vp, _sz,
                               _u64], ctypes.c_int),
    "la_gdn_prefill_varlen_noalloc": ([_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i32, _i32,
                                       _i32, _i32, _i32, _i32, _i32, _i32, _i64, _i64, _i64,
                                       _f32, _u64], ctypes.c_int),
    "la_kda_prefill": ([_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i32, _i32, _i32, _i32, _i32,
                        _i32, _i32, _i32, _i64, _i64, _i64, _f32, _f32, _i32, _vp, _sz, _u64],
                       ctypes.c_int),
    "la_prefill_front": ([_vp, _vp, _vp, _vp, _vp, _i32, _vp, _vp, _vp, _vp, _i32, _i32, _i32,
                          _i32, _i32, _i32, _i32, _i32, _i64, _f32, _f32, _f32, _vp, _vp, _f32,
                          _i32, _i32, _vp, _sz, _u64], ctypes.c_int),
    "la_gated_rmsnorm": ([_vp, _vp, _vp, _vp, _i32, _i32, _i32, _f32, _i32, _u64], ctypes.c_int),
    "la_gemm_bf16": ([_vp, _vp, _vp, _i32, _i32, _i32, _i64, _i64, _i64, _u64], ctypes.c_int),
    "la_prefill_segmented_workspace_bytes": ([_i32, _i32, _i32], _sz),
    "la_prefill_segmented": ([_vp, _vp, _vp, _vp, _vp, _vp, _vp, _i32, _i32, _i32, _i32, _i32,
                              _i32, _i64, _i64, _i64, _f32, _i32, _i32, _i32, _vp, _sz, _u64],
                             ctypes.c_int),
    "la_rmsnorm_rows": ([_vp, _vp, _vp, _i32, _i32, _i64, _i64, _f32, _u64], ctypes.c_int),
    "la_gate_activations": ([_vp, _i64, _i32, _i32, _i32, _vp, _vp, _u64], ctypes.c_int),
    "la_decode_workspace_bytes": ([_i32, _i32, _i32, _i32, _i32, _i32], _sz),
    "la_decode_step": ([_vp, _vp, _vp, _vp, _vp, _i32, _vp, _vp, _vp, _i32, _i32, _i32, _i32,
                        _i32, _i32, _i64, _f32, _f32, _i32, _i32, _vp, _sz, _u64], ctypes.c_int),
    "la_gated_scan_workspace_bytes": ([_i32, _i32, _i32, _i32], _sz),
    "la_gated_scan_saved_bytes": ([_i32, _i32, _i32, _i32], _sz),
    "la_gated_scan": ([_vp, _vp, _vp, _vp, _vp, _sz, _vp, _i32, _i32, _i32, _i32, _i64, _i64,
                       _i64, _i32, _vp, _sz, _u64], ctypes.c_int),
    "la_gated_scan_backward": ([_vp, _vp, _vp, _sz, _vp, _vp, _vp, _vp, _vp, _vp, _i32, _i32,
                                _i32, _i32, _i64, _i64, _i64, _i64, _i64, _i32, _vp, _sz, _u64],
                               ctypes.c_int),
    "la_gated_scan_step": ([_vp, _vp, _vp, _vp, _vp, _vp, _i32, _vp, _i32, _i32, _i32, _i64, _i64,
                            _i64, _i32, _u64], ctypes.c_int),
    "la_conv1d_silu_backward_workspace_bytes": ([_i32, _i32, _i32, _i32, _i32], _sz),
    "la_conv1d_silu_backward": ([_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i32,
                                 _i32, _i32, _i32, _i32, _i64, _i64, _i64, _i32, _vp, _sz, _u64],
                                ctypes.c_int),
    "la_w4_matvec": ([_vp, _vp, _vp, _vp, _i32, _i32, _i32, _i32, _i64, _i64, _u64],
                     ctypes.c_int),
    "la_w4_quantize": ([_vp, _vp, _vp, _i32, _i32, _i32, _i64, _u64], ctypes.c_int),
    "la_layernorm_rows": ([_vp, _vp, _vp, _vp, _vp, _i32, _i32, _i64, _i64, _f32, _i32, _u64],
                          ctypes.c_int),
    "la_layernorm_rows_backward_workspace_bytes": ([_i32, _i32, _i32], _sz),
    "la_layernorm_rows_backward": ([_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i32, _i32, _i64, _i64,
                                    _i64, _i64, _i32, _vp, _sz, _u64], ctypes.c_int),
    "la_linear_saved_bytes": ([_i32, _i32, _i32], _sz),
    "la_linear": ([_vp, _vp, _vp, _vp, _vp, _vp, _sz, _i32, _i32, _i32, _i64, _i64, _i64, _i64,
                   _i32, _u64], ctypes.c_int),
    "la_linear_backward_workspace_bytes": ([_i32, _i32, _i32, _i32], _sz),
    "la_linear_backward": ([_vp, _vp, _vp, _sz, _vp, _vp, _vp, _vp, _i32, _i32, _i32, _i64, _i64,
                            _i64, _i64, _i64, _i32, _vp, _sz, _u64], ctypes.c_int),
    "la_gated_ffn_saved_bytes": ([_i32, _i32], _sz),
    "la_gated_ffn": ([_vp, _vp, _vp, _vp, _vp, _sz, _i32, _i32, _i32, _i64, _i64, _i64, _i64, _i32,
                      _u64], ctypes.c_int),
    "la_gated_ffn_backward_workspace_bytes": ([_i32, _i32, _i32], _sz),
    "la_gated_ffn_backward": ([_vp, _vp, _vp, _vp, _sz, _vp, _vp, _vp, _vp, _i32, _i32, _i32, _i64,
                               _i64, _i64, _i64, _i64, _i64, _i64, _i32, _vp, _sz, _u64],
                              ctypes.c_int),
}

_lib = None


def library_path() -> str:
    return LIB_PATH


def _load():
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(
                f"linattn CUDA library not built ({LIB_PATH} missing); run "
                "`python -m linear_attention_chunked_conv1d_gb300.build` — there is no fallback")
        lib = ctypes.CDLL(LIB_PATH)
        for name, (args, res) in _SIGS.items():
            fn = getattr(lib, name)
            fn.argtypes = args
            fn.restype = res
        _lib = lib
    return _lib


def _check(rc: int) -> None:
    if rc != LA_OK:
        raise LinAttnError(rc, last_error())


def abi_version() -> int:
    return _load().la_abi_version()


def last_error() -> str:
    return _load().la_last_error().decode()


def _stream(stream) -> int:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def device_status(stream=None) -> int:
    """Synchronise the stream and return (then clear) the device status flags (LA_DEV_*)."""
    return _load().la_device_status(_stream(stream))


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return LA_F32
    if t.dtype == torch.bfloat16:
        return LA_BF16
    raise TypeError(f"activation dtype {t.dtype}: expected float32 or bfloat16")


def _ptr(t) -> int | None:
    return None if t is None else t.data_ptr()


def _row_stride(t: torch.Tensor) -> int:
    return t.stride(0)


def pointer_array(tensors, device=None) -> torch.Tensor:
    """Device array of the data pointers of `tensors` (h-state / conv-state lists), stored as
    int64 (the same 64 bits the C ABI reads as uint64_t)."""
    ptrs = [t.data_ptr() for t in tensors]
    dev = device if device is not None else tensors[0].device
    return torch.tensor(ptrs, dtype=torch.int64, device=dev)


def conv1d_silu_prefill(conv_state, x, w, out, *, t=None, bias=None, max_tokens=None,
                        stream=None) -> None:
    """Causal conv1d + SiLU over one stream, advancing conv_state [K-1][C] in place.

    x, out: [t][stride] (the first C = w.shape[0] channels are used); w [C][K]."""
    t = x.shape[0] if t is None else t
    C, K = w.shape
    _check(_load().la_conv1d_silu_prefill(
        _ptr(conv_state), _ptr(x), _ptr(w), _ptr(bias), _ptr(out), t,
        max_tokens if max_tokens is not None else t, C, K, _row_stride(x), _row_stride(out),
        _dtype_code(x), _stream(stream)))


def conv1d_silu_prefill_varlen(conv_state_ptrs, x, w, out, cu_seqlens, *, bias=None,
                               total_tokens=None, max_tokens=None, stream=None) -> None:
    """conv1d_silu_prefill over B packed streams; conv_state_ptrs is a device uint64 array."""
    B = cu_seqlens.shape[0] - 1
    total = x.shape[0] if total_tokens is None else total_tokens
    C, K = w.shape
    _check(_load().la_conv1d_silu_prefill_varlen(
        _ptr(conv_state_ptrs), _ptr(x), _ptr(w), _ptr(bias), _ptr(out), _ptr(cu_seqlens), B,
        total, max_tokens if max_tokens is not None else total, C, K, _row_stride(x),
        _row_stride(out), _dtype_code(x), _stream(stream)))


def conv1d_silu_l2_prefill(conv_state_ptrs, x, w, out, cu_seqlens=None, *, l2_heads, head_dim,
                           eps=1e-6, bias=None, total_tokens=None, max_tokens=None,
                           stream=None) -> None:
    """Fused conv1d + SiLU + per-head L2 over the first l2_heads*head_dim channels (one pass)."""
    B = 1 if cu_seqlens is None else cu_seqlens.shape[0] - 1
    total = x.shape[0] if total_tokens is None else total_tokens
    C, K = w.shape
    _check(_load().la_conv1d_silu_l2_prefill(
        _ptr(conv_state_ptrs), _ptr(x), _ptr(w), _ptr(bias), _ptr(out), _ptr(cu_seqlens), B,
        total, max_tokens if max_tokens is not None else total, C, K, l2_heads, head_dim,
        float(eps), _row_stride(x), _row_stride(out), _dtype_code(x), _stream(stream)))


def l2norm_heads(x, n_heads, head_dim, *, eps=1e-6, t=None, stream=None) -> None:
    """In-place L2 norm of each (token, head) over the first n_heads*head_dim channels."""
    t = x.shape[0] if t is None else t
    _check(_load().la_l2norm_heads(_ptr(x), t, n_heads, head_dim, _row_stride(x), float(eps),
                                   _dtype_code(x), _stream(stream)))


def prefill_workspace_bytes(B, total_tokens, Hk, Hv, dk, dv, dtype) -> int:
    code = dtype if isinstance(dtype, int) else (LA_BF16 if dtype == torch.bfloat16 else LA_F32)
    return int(_load().la_prefill_workspace_bytes(B, total_tokens, Hk, Hv, dk, dv, code))


def gdn_prefill_batched(h_state_ptrs, q, k, v, g, beta, out, *, B, T, Hk, Hv, dk, dv,
                        scale=None, max_tokens=None, workspace=None, stream=None) -> None:
    """GDN over B equal-length streams of T tokens; states updated through h_state_ptrs."""
    scale = 1.0 / math.sqrt(dk) if scale is None else scale
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(_load().la_gdn_prefill_batched(
        _ptr(h_state_ptrs), _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(out), B, T,
        max_tokens if max_tokens is not None else B * T, Hk, Hv, dk, dv, _row_stride(q),
        _row_stride(k), _row_stride(v), float(scale), _dtype_code(q), _ptr(workspace), ws_bytes,
        _stream(stream)))


def gdn_prefill_varlen(h_state_ptrs, q, k, v, g, beta, out, cu_seqlens, *, max_seqlen, Hk, Hv,
                       dk, dv, total_tokens=None, scale=None, max_tokens=None, workspace=None,
                       stream=None) -> None:
    """GDN over B packed streams of different lengths (cu_seqlens, device int32 [B+1])."""
    B = cu_seqlens.shape[0] - 1
    total = q.shape[0] if total_tokens is None else total_tokens
    scale = 1.0 / math.sqrt(dk) if scale is None else scale
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(_load().la_gdn_prefill_varlen(
        _ptr(h_state_ptrs), _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(out),
        _ptr(cu_seqlens), B, total, max_seqlen,
        max_tokens if max_tokens is not None else total, Hk, Hv, dk, dv, _row_stride(q),
        _row_stride(k), _row_stride(v), float(scale), _dtype_code(q), _ptr(workspace), ws_bytes,
        _stream(stream)))


def gdn_prefill_varlen_noalloc(h_state_ptrs, q, k, v, g, beta, out, cu_seqlens, *, max_seqlen,
                               Hk, Hv, dk, dv, total_tokens=None, scale=None, max_tokens=None,
                               stream=None) -> None:
    """gdn_prefill_varlen without a workspace, for callers that cannot allocate device memory:
    the library's fixed scratch (up to 4096 streams per call) is used instead. Calls that
    overlap on the GPU share that scratch and must be ordered; the first call on a device
    should come before any stream capture there. The entry point is compiled for bf16 q, k, v
    and out only: any other dtype is refused here (the C call has no dtype argument)."""
    for name, t in (("q", q), ("k", k), ("v", v), ("out", out)):
        if t.dtype != torch.bfloat16:
            raise TypeError(f"gdn_prefill_varlen_noalloc takes bf16 tensors; {name} is {t.dtype}")
    B = cu_seqlens.shape[0] - 1
    total = q.shape[0] if total_tokens is None else total_tokens
    scale = 1.0 / math.sqrt(dk) if scale is None else scale
    _check(_load().la_gdn_prefill_varlen_noalloc(
        _ptr(h_state_ptrs), _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(out),
        _ptr(cu_seqlens), B, total, max_seqlen,
        max_tokens if max_tokens is not None else total, Hk, Hv, dk, dv, _row_stride(q),
        _row_stride(k), _row_stride(v), float(scale), _stream(stream)))


def kda_prefill(h_state_ptrs, q, k, v, gate, beta, out, cu_seqlens=None, *, Hk, Hv, dk, dv,
                max_seqlen=None, total_tokens=None, scale=None, pad_fill=0.0, max_tokens=None,
                workspace=None, stream=None) -> None:
    """KDA (per-channel gate [tok][Hv][dk]) over one stream (cu_seqlens None) or B streams."""
    B = 1 if cu_seqlens is None else cu_seqlens.shape[0] - 1
    total = q.shape[0] if total_tokens is None else total_tokens
    max_seqlen = total if max_seqlen is None else max_seqlen
    scale = 1.0 / math.sqrt(dk) if scale is None else scale
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(_load().la_kda_prefill(
        _ptr(h_state_ptrs), _ptr(q), _ptr(k), _ptr(v), _ptr(gate), _ptr(beta), _ptr(out),
        _ptr(cu_seqlens), B, total, max_seqlen,
        max_tokens if max_tokens is not None else total, Hk, Hv, dk, dv, _row_stride(q),
        _row_stride(k), _row_stride(v), float(scale), float(pad_fill), _dtype_code(q),
        _ptr(workspace), ws_bytes, _stream(stream)))


def prefill_front(conv_state_ptrs, h_state_ptrs, x, conv_w, gate, beta, out, cu_seqlens=None, *,
                  B=None, Hk, Hv, dk, dv, kda, conv_bias=None, max_seqlen=None,
                  total_tokens=None, l2_eps=1e-6, scale=None, pad_fill=0.0, max_tokens=None,
                  z=None, norm_w=None, norm_eps=1e-6, workspace=None, stream=None) -> None:
    """conv1d + SiLU + q|k L2 + recurrence of one layer in one launch, from the pre-conv rows
    x [tok][2*Hk*dk + Hv*dv]. cu_seqlens None: B equal streams (B defaults to 1). With z (and
    norm_w [dv]) the output store applies the gated RMSNorm o/rms(o) * norm_w * SiLU(z)."""
    if cu_seqlens is not None:
        B = cu_seqlens.shape[0] - 1
    elif B is None:
        B = 1
    total = x.shape[0] if total_tokens is None else total_tokens
    max_seqlen = (total // B if cu_seqlens is None else total) if max_seqlen is None else max_seqlen
    scale = 1.0 / math.sqrt(dk) if scale is None else scale
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _, K = conv_w.shape
    _check(_load().la_prefill_front(
        _ptr(conv_state_ptrs), _ptr(h_state_ptrs), _ptr(x), _ptr(conv_w), _ptr(conv_bias), K,
        _ptr(gate), _ptr(beta), _ptr(out), _ptr(cu_seqlens), B, total, max_seqlen,
        max_tokens if max_tokens is not None else total, Hk, Hv, dk, dv, _row_stride(x),
        float(l2_eps), float(scale), float(pad_fill), _ptr(z), _ptr(norm_w), float(norm_eps),
        1 if kda else 0, _dtype_code(x), _ptr(workspace), ws_bytes, _stream(stream)))


def decode_workspace_bytes(B, Hk, Hv, dk, dv, dtype) -> int:
    code = dtype if isinstance(dtype, int) else (LA_BF16 if dtype == torch.bfloat16 else LA_F32)
    return int(_load().la_decode_workspace_bytes(B, Hk, Hv, dk, dv, code))


def decode_step(conv_state_ptrs, h_state_ptrs, x, conv_w, gate, beta, out, *, Hk, Hv, dk, dv,
                kda, conv_bias=None, l2_eps=1e-6, scale=None, max_streams=None, workspace=None,
                stream=None) -> None:
    """One decode step: x [B][cd] holds one new token per stream; conv and h states advance
    in place; out [B][Hv][dv]."""
    B = x.shape[0]
    scale = 1.0 / math.sqrt(dk) if scale is None else scale
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _, K = conv_w.shape
    _check(_load().la_decode_step(
        _ptr(conv_state_ptrs), _ptr(h_state_ptrs), _ptr(x), _ptr(conv_w), _ptr(conv_bias), K,
        _ptr(gate), _ptr(beta), _ptr(out), B, max_streams if max_streams is not None else B, Hk,
        Hv, dk, dv, _row_stride(x), float(l2_eps), float(scale), 1 if kda else 0,
        _dtype_code(x), _ptr(workspace), ws_bytes, _stream(stream)))


def gated_rmsnorm(o, z, w, y=None, *, eps=1e-6, stream=None):
    """y = o / sqrt(mean(o^2) + eps) * w * SiLU(z) per row of the last axis; o, z [t][Hv][dv].
    y defaults to o (in place). Returns y."""
    y = o if y is None else y
    t, Hv, dv = o.shape
    _check(_load().la_gated_rmsnorm(_ptr(o), _ptr(z), _ptr(w), _ptr(y), t, Hv, dv, float(eps),
                                    _dtype_code(o), _stream(stream)))
    return y


def gemm_bf16(a, w, c=None, *, stream=None):
    """C = A W^T (bf16, fp32 accumulation on the tensor cores); a [M][K], w [N][K] (a linear
    layer's [out][in] weight); c [M][N] (allocated when None). Returns c."""
    M, K = a.shape
    N = w.shape[0]
    if c is None:
        c = torch.empty(M, N, dtype=torch.bfloat16, device=a.device)
    _check(_load().la_gemm_bf16(_ptr(a), _ptr(w), _ptr(c), M, N, K, _row_stride(a),
                                _row_stride(w), _row_stride(c), _stream(stream)))
    return c


def rmsnorm_rows(x, w, y=None, *, eps=1e-6, stream=None):
    """y = x / sqrt(mean(x^2) + eps) * w per row (bf16); y defaults to a new tensor."""
    rows, width = x.shape
    if y is None:
        y = torch.empty_like(x)
    _check(_load().la_rmsnorm_rows(_ptr(x), _ptr(w), _ptr(y), rows, width, _row_stride(x),
                                   _row_stride(y), float(eps), _stream(stream)))
    return y


def gate_activations(ab, na, g=None, beta=None, *, stream=None):
    """g = -softplus(ab[:, :na]), beta = sigmoid(ab[:, na:]) in fp32 (new tensors by default)."""
    t, width = ab.shape
    nb = width - na
    if g is None:
        g = torch.empty(t, na, dtype=torch.float32, device=ab.device)
    if beta is None:
        beta = torch.empty(t, nb, dtype=torch.float32, device=ab.device)
    _check(_load().la_gate_activations(_ptr(ab), _row_stride(ab), t, na, nb, _ptr(g), _ptr(beta),
                                       _stream(stream)))
    return g, beta


def prefill_segmented_workspace_bytes(total_tokens, Hv, segments) -> int:
    return int(_load().la_prefill_segmented_workspace_bytes(total_tokens, Hv, segments))


def prefill_segmented(h_state_ptrs, q, k, v, gate, beta, out, *, Hk, Hv, dk, dv, kda, segments,
                      total_tokens=None, scale=None, max_tokens=None, workspace=None,
                      stream=None) -> None:
    """The recurrence of ONE long stream with its tokens cut into `segments` pieces that run
    side by side on the tensor cores, then joined (chunk-parallel scan)."""
    total = q.shape[0] if total_tokens is None else total_tokens
    scale = 1.0 / math.sqrt(dk) if scale is None else scale
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(_load().la_prefill_segmented(
        _ptr(h_state_ptrs), _ptr(q), _ptr(k), _ptr(v), _ptr(gate), _ptr(beta), _ptr(out), total,
        max_tokens if max_tokens is not None else total, Hk, Hv, dk, dv, _row_stride(q),
        _row_stride(k), _row_stride(v), float(scale), 1 if kda else 0, int(segments),
        _dtype_code(q), _ptr(workspace), ws_bytes, _stream(stream)))


def _dtype_arg(dtype) -> int:
    return dtype if isinstance(dtype, int) else (LA_BF16 if dtype == torch.bfloat16 else LA_F32)


# The calls below may take no longer than their launch does, so their checks are kept to what costs
# well under a microsecond each: devices are compared by their index.
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _on_gpu(t) -> int:
    """The device index of `t`, which has to be the current one: streams and launches are its own."""
    dev = t.get_device()
    if dev < 0:
        raise ValueError("expected CUDA tensors")
    cur = _current_device()
    if dev != cur:
        raise ValueError(f"tensors on cuda:{dev}, but the current device is cuda:{cur}: use "
                         "torch.cuda.device(...)")
    return dev


def _stream_on(stream, dev) -> int:
    return _current_stream(dev) if stream is None and _current_stream is not None else _stream(stream)


def _matrix(name, t, rows, cols, dtype, dev) -> int:
    """Checks a matrix of dense rows; returns its row stride."""
    if t.dtype != dtype:
        raise TypeError(f"{name} is {t.dtype}, expected {dtype}")
    if t.shape == (rows, cols) and t.get_device() == dev:
        s, inner = t.stride()
        if inner == 1 or cols == 1:
            return s if rows > 1 else cols  # a single row's stride says nothing
    raise ValueError(f"{name}: {tuple(t.shape)} with strides {t.stride()} on device {t.get_device()}, "
                     f"expected {(rows, cols)} with dense rows on device {dev}")


def _on_stream(stream):
    """The context in which what a call allocates belongs to the stream that it runs on."""
    if stream is not None and not isinstance(stream, torch.cuda.Stream):
        handle = _stream(stream)
        # 0 is the default stream; torch would make a new one of it
        stream = torch.cuda.ExternalStream(handle) if handle else torch.cuda.default_stream()
    return torch.cuda.stream(stream)


def _dense(name, t, shape, dtype, dev):
    """The address of a contiguous tensor of this shape."""
    if t.dtype != dtype:
        raise TypeError(f"{name} is {t.dtype}, expected {dtype}")
    if t.shape != shape or not t.is_contiguous() or t.get_device() != dev:
        raise ValueError(f"{name}: {tuple(t.shape)} on device {t.get_device()}, expected a "
                         f"contiguous {tuple(shape)} on device {dev}")
    return t.data_ptr()


def _ptrs(name, t, B, dev):
    """The address of a device array of B pointers (pointer_array), or None."""
    if t is None:
        return None
    if t.dtype != torch.int64 and t.dtype != torch.uint64:
        raise TypeError(f"{name} is {t.dtype}, expected the int64 of pointer_array")
    if t.numel() != B or not t.is_contiguous() or t.get_device() != dev:
        raise ValueError(f"{name}: {t.numel()} pointers on device {t.get_device()}, expected {B} "
                         f"on device {dev}")
    return t.data_ptr()


def _streams(cu_seqlens, B, dev):
    """(address of cu_seqlens or None, number of streams)."""
    if cu_seqlens is None:
        return None, 1 if B is None else B
    n = cu_seqlens.shape[0] - 1
    if B is not None and B != n:
        raise ValueError(f"B = {B}, but cu_seqlens has {n} streams")
    return _dense("cu_seqlens", cu_seqlens, (n + 1,), torch.int32, dev), n


def _room(name, t, dev):
    """(address, bytes) of a workspace or saved buffer, or (None, 0)."""
    if t is None:
        return None, 0
    if not t.is_contiguous() or t.get_device() != dev:
        raise ValueError(f"{name} must be contiguous and on device {dev}")
    return t.data_ptr(), t.numel() * t.element_size()


def gated_scan_workspace_bytes(B, total_tokens, channels, dtype) -> int:
    """Bytes of workspace that gated_scan and gated_scan_backward need."""
    return int(_load().la_gated_scan_workspace_bytes(B, total_tokens, channels, _dtype_arg(dtype)))


def gated_scan_saved_bytes(B, total_tokens, channels, dtype) -> int:
    """Bytes of the buffer that gated_scan fills for gated_scan_backward."""
    return int(_load().la_gated_scan_saved_bytes(B, total_tokens, channels, _dtype_arg(dtype)))


def gated_scan(h_state_ptrs, x, ab, y, cu_seqlens=None, *, B=None, saved=None, max_tokens=None,
               workspace=None, stream=None) -> None:
    """h_t = (1 - sigmoid(a_t)) h_{t-1} + sigmoid(b_t) x_t per channel, y_t = h_t.

    x, y [t][C]; ab [t][2C] holds the gate rows a | b (as gate_activations takes them). Packed
    streams (cu_seqlens, device int32 [B+1]) or, without cu_seqlens, B equal ones. h_state_ptrs:
    pointer_array of B fp32 [C] states, advanced in place, or None (from zero, not kept). saved: a
    buffer of gated_scan_saved_bytes(...) when gated_scan_backward is to follow."""
    dt, dev = x.dtype, x.get_device()
    T, C = x.shape
    (xs, x1), (gs, g1), (ys, y1) = x.stride(), ab.stride(), y.stride()
    if cu_seqlens is not None:
        n = cu_seqlens.shape[0] - 1
    else:
        n = 1 if B is None else B
    # As in gated_scan_step: a scan of a few tokens is as long as its launch.
    if not (dev >= 0 and dev == _current_device() and ab.dtype is dt and y.dtype is dt
            and ab.shape == (T, 2 * C) and y.shape == (T, C) and x1 == g1 == y1 == 1
            and ab.get_device() == dev and y.get_device() == dev
            and (cu_seqlens is None or (cu_seqlens.dtype is torch.int32 and (B is None or B == n)
                                        and cu_seqlens.dim() == 1 and cu_seqlens.is_contiguous()
                                        and cu_seqlens.get_device() == dev))
            and (h_state_ptrs is None or (h_state_ptrs.dtype is torch.int64
                                          and h_state_ptrs.numel() == n
                                          and h_state_ptrs.get_device() == dev
                                          and h_state_ptrs.is_contiguous()))
            and workspace is not None and workspace.is_contiguous()
            and workspace.get_device() == dev
            and (saved is None or (saved.is_contiguous() and saved.get_device() == dev))):
        _on_gpu(x)
        _streams(cu_seqlens, B, dev)
        for name, m, cols in (("x", x, C), ("ab", ab, 2 * C), ("y", y, C)):
            _matrix(name, m, T, cols, dt, dev)
        _ptrs("h_state_ptrs", h_state_ptrs, n, dev)
        _room("saved", saved, dev)
        _room("workspace", workspace, dev)
    if T == 1:  # a single row's stride says nothing
        xs, gs, ys = C, 2 * C, C
    _check(_load().la_gated_scan(
        None if h_state_ptrs is None else h_state_ptrs.data_ptr(), x.data_ptr(), ab.data_ptr(),
        y.data_ptr(), None if saved is None else saved.data_ptr(),
        0 if saved is None else saved.numel() * saved.element_size(),
        None if cu_seqlens is None else cu_seqlens.data_ptr(), n, T,
        T if max_tokens is None else max_tokens, C, xs, gs, ys, _dtype_code(x),
        None if workspace is None else workspace.data_ptr(),
        0 if workspace is None else workspace.numel() * workspace.element_size(),
        _stream_on(stream, dev)))


def gated_scan_backward(x, ab, saved, dy, dx, dab, cu_seqlens=None, *, B=None, dh_final_ptrs=None,
                        dh0_ptrs=None, max_tokens=None, workspace=None, stream=None) -> None:
    """Gradients of gated_scan: dx [t][C] and dab [t][2C] from dy [t][C] and, where given, from the
    gradients of the final states (dh_final_ptrs, B fp32 [C]; None: zero); the gradients of the
    initial states go to dh0_ptrs (B fp32 [C]) where given. x, ab, cu_seqlens and B are those of the
    forward call, saved what it left."""
    dev = _on_gpu(x)
    T, C = x.shape
    cu, B = _streams(cu_seqlens, B, dev)
    sv, sv_bytes = _room("saved", saved, dev)
    ws, ws_bytes = _room("workspace", workspace, dev)
    _check(_load().la_gated_scan_backward(
        x.data_ptr(), ab.data_ptr(), sv, sv_bytes, dy.data_ptr(),
        _ptrs("dh_final_ptrs", dh_final_ptrs, B, dev), dx.data_ptr(), dab.data_ptr(),
        _ptrs("dh0_ptrs", dh0_ptrs, B, dev), cu, B, T, T if max_tokens is None else max_tokens, C,
        _matrix("x", x, T, C, x.dtype, dev), _matrix("ab", ab, T, 2 * C, x.dtype, dev),
        _matrix("dy", dy, T, C, x.dtype, dev), _matrix("dx", dx, T, C, x.dtype, dev),
        _matrix("dab", dab, T, 2 * C, x.dtype, dev), _dtype_code(x), ws, ws_bytes,
        _stream_on(stream, dev)))


def gated_scan_step(h_state_ptrs, x, ab, y, *, conv_state_ptrs=None, conv_w=None, conv_bias=None,
                    max_streams=None, stream=None) -> None:
    """One token for each of B streams: conv1d + SiLU on the carried windows (with conv_w [C][K] and
    conv_state_ptrs to [K-1][C]; without conv_w, x enters as it is), then one step of gated_scan.
    x, y [B][C], ab [B][2C]; both states advance in place."""
    dt, dev = x.dtype, x.get_device()
    B, C = x.shape
    K = 0 if conv_w is None else conv_w.shape[1]
    (xs, x1), (gs, g1), (ys, y1) = x.stride(), ab.stride(), y.stride()
    # A decode step is as long as its launch: one look at everything, and only where something is
    # unusual the checks that say what.
    if not (dev >= 0 and dev == _current_device() and ab.dtype is dt and y.dtype is dt
            and ab.shape == (B, 2 * C) and y.shape == (B, C) and x1 == g1 == y1 == 1
            and ab.get_device() == dev and y.get_device() == dev
            and h_state_ptrs is not None and h_state_ptrs.dtype is torch.int64
            and h_state_ptrs.numel() == B and h_state_ptrs.get_device() == dev
            and h_state_ptrs.is_contiguous()
            and (conv_w is None or (K > 0 and conv_w.dtype is dt and conv_w.shape[0] == C and conv_w.is_contiguous()
                            and conv_w.get_device() == dev
                            and (K == 1 or (conv_state_ptrs is not None
                                            and conv_state_ptrs.dtype is torch.int64
                                            and conv_state_ptrs.numel() == B
                                            and conv_state_ptrs.get_device() == dev
                                            and conv_state_ptrs.is_contiguous()))
                            and (conv_bias is None or (conv_bias.dtype is dt
                                                       and conv_bias.shape == (C,)
                                                       and conv_bias.is_contiguous()
                                                       and conv_bias.get_device() == dev))))):
        _on_gpu(x)
        for name, m, cols in (("x", x, C), ("ab", ab, 2 * C), ("y", y, C)):
            _matrix(name, m, B, cols, dt, dev)
        _ptrs("h_state_ptrs", h_state_ptrs, B, dev)
        _ptrs("conv_state_ptrs", conv_state_ptrs, B, dev)
        if conv_w is not None:
            if K == 0:
                raise ValueError("conv_w has no taps: leave it out for a layer without a convolution")
            _dense("conv_w", conv_w, (C, K), dt, dev)
            if conv_bias is not None:
                _dense("conv_bias", conv_bias, (C,), dt, dev)
    if B == 1:  # a single row's stride says nothing
        xs, gs, ys = C, 2 * C, C
    _check(_load().la_gated_scan_step(
        None if conv_state_ptrs is None else conv_state_ptrs.data_ptr(),
        None if h_state_ptrs is None else h_state_ptrs.data_ptr(), x.data_ptr(), ab.data_ptr(),
        None if conv_w is None else conv_w.data_ptr(),
        None if conv_bias is None else conv_bias.data_ptr(), K, y.data_ptr(), B,
        B if max_streams is None else max_streams, C, xs, gs, ys, _dtype_code(x),
        _stream_on(stream, dev)))


def conv1d_silu_backward_workspace_bytes(B, total_tokens, channels, kernel, dtype) -> int:
    """Bytes of workspace that conv1d_silu_backward needs."""
    return int(_load().la_conv1d_silu_backward_workspace_bytes(B, total_tokens, channels, kernel,
                                                               _dtype_arg(dtype)))


def conv1d_silu_backward(conv_state_ptrs, x, w, dout, dx, dw, cu_seqlens=None, *, B=None, bias=None,
                         dbias=None, dstate_final_ptrs=None, dstate_ptrs=None, max_tokens=None,
                         workspace=None, stream=None) -> None:
    """Gradients of conv1d_silu_prefill[_varlen]: dx [t][C] from dout [t][C], dw [C][K] and dbias [C]
    in fp32, and the gradients of the initial windows (dstate_ptrs, where given).

    conv_state_ptrs: the streams' [K-1][C] windows as they were before the forward call, which
    advances them in place; dstate_final_ptrs: gradients of the windows it left (None: zero)."""
    dev = _on_gpu(x)
    T, C = x.shape
    K = w.shape[1]
    cu, B = _streams(cu_seqlens, B, dev)
    ws, ws_bytes = _room("workspace", workspace, dev)
    _check(_load().la_conv1d_silu_backward(
        _ptrs("conv_state_ptrs", conv_state_ptrs, B, dev), x.data_ptr(),
        _dense("w", w, (C, K), x.dtype, dev),
        None if bias is None else _dense("bias", bias, (C,), x.dtype, dev), dout.data_ptr(),
        _ptrs("dstate_final_ptrs", dstate_final_ptrs, B, dev), dx.data_ptr(),
        _dense("dw", dw, (C, K), torch.float32, dev),
        None if dbias is None else _dense("dbias", dbias, (C,), torch.float32, dev),
        _ptrs("dstate_ptrs", dstate_ptrs, B, dev), cu, B, T, T if max_tokens is None else max_tokens,
        C, K, _matrix("x", x, T, C, x.dtype, dev), _matrix("dout", dout, T, C, x.dtype, dev),
        _matrix("dx", dx, T, C, x.dtype, dev), _dtype_code(x), ws, ws_bytes, _stream_on(stream, dev)))


def w4_quantize(w, q=None, scales=None, *, group=128, stream=None):
    """Lays a bf16 weight w [N][K] out for w4_matvec: (q uint8 [N][K/2], scales bf16 [N][K/group])."""
    dev = _on_gpu(w)
    N, K = w.shape
    if group <= 0 or K % group:
        raise ValueError(f"groups of {group} for {K} inputs")
    with _on_stream(stream):
        if q is None:
            q = torch.empty(N, K // 2, dtype=torch.uint8, device=w.device)
        if scales is None:
            scales = torch.empty(N, K // group, dtype=torch.bfloat16, device=w.device)
    _check(_load().la_w4_quantize(
        w.data_ptr(), _dense("q", q, (N, K // 2), torch.uint8, dev),
        _dense("scales", scales, (N, K // group), torch.bfloat16, dev), N, K, group,
        _matrix("w", w, N, K, torch.bfloat16, dev), _stream_on(stream, dev)))
    return q, scales


def w4_matvec(x, q, scales, y=None, *, stream=None):
    """y = x W^T for 1..LA_W4_MAX_ROWS bf16 rows x [M][K] and a weight that w4_quantize laid out
    (q [N][K/2], scales [N][K/group]); y [M][N] bf16 (allocated when None). Returns y."""
    dev = x.get_device()
    M, K = x.shape
    N, groups = scales.shape
    if groups == 0 or K % groups:
        raise ValueError(f"{groups} scales for each {K} inputs")
    if y is None:
        if stream is None:
            y = torch.empty(M, N, dtype=torch.bfloat16, device=x.device)
        else:
            with _on_stream(stream):
                y = torch.empty(M, N, dtype=torch.bfloat16, device=x.device)
    (xs, x1), (ys, y1) = x.stride(), y.stride()
    if not (dev >= 0 and dev == _current_device() and x.dtype is torch.bfloat16
            and y.dtype is torch.bfloat16 and scales.dtype is torch.bfloat16
            and q.dtype is torch.uint8 and q.shape == (N, K // 2) and y.shape == (M, N)
            and x1 == y1 == 1 and q.get_device() == dev and scales.get_device() == dev
            and y.get_device() == dev and q.is_contiguous() and scales.is_contiguous()):
        _on_gpu(x)  # what is unusual, and whether it is wrong
        _matrix("x", x, M, K, torch.bfloat16, dev)
        _matrix("y", y, M, N, torch.bfloat16, dev)
        _dense("q", q, (N, K // 2), torch.uint8, dev)
        _dense("scales", scales, (N, groups), torch.bfloat16, dev)
    if M == 1:
        xs, ys = K, N
    _check(_load().la_w4_matvec(x.data_ptr(), q.data_ptr(), scales.data_ptr(), y.data_ptr(), M, N, K,
                                K // groups, xs, ys, _stream_on(stream, dev)))
    return y


_BF16, _F32 = torch.bfloat16, torch.float32


def _act_code(act) -> int:
    code = LA_ACTIVATIONS.get(act)
    if code is None:
        raise ValueError(f"activation {act!r}: one of {', '.join(LA_ACTIVATIONS)}")
    return code


def _vector(name, t, n, dtype, dev):
    """The address of a contiguous vector, or None."""
    return None if t is None else _dense(name, t, (n,), dtype, dev)


def _rows_like(shape, dtype, device, stream):
    """A new matrix on the stream of the call, whose rows start on 16 bytes."""
    per = 16 // dtype.itemsize
    ld = (shape[1] + per - 1) // per * per
    if stream is None:
        return torch.empty(shape[0], ld, dtype=dtype, device=device)[:, :shape[1]]
    with _on_stream(stream):
        return torch.empty(shape[0], ld, dtype=dtype, device=device)[:, :shape[1]]


def layernorm_rows(x, w, b=None, y=None, *, stats=None, eps=1e-5, stream=None):
    """y = (x - mean) / sqrt(var + eps) * w + b per row; x, y [rows][width] (fp32 or bf16; width up to
    8192, rows on 16 bytes; y may be x, and defaults to a new tensor), w, b [width]. stats: fp32
    [rows][2] that receives mean and 1 / sqrt(var + eps), when layernorm_rows_backward is to follow.
    Returns y."""
    dev, dt = x.get_device(), x.dtype
    rows, width = x.shape
    if y is None:
        y = _rows_like((rows, width), dt, x.device, stream)
    (xs, x1), (ys, y1) = x.stride(), y.stride()
    # As in gated_scan: one look at everything, and only where something is unusual the checks that say what.
    if not (dev >= 0 and dev == _current_device() and x1 == y1 == 1 and y.shape == (rows, width)
            and y.dtype is dt and y.get_device() == dev and w.dtype is dt and w.shape == (width,)
            and w.is_contiguous() and w.get_device() == dev
            and (b is None or (b.dtype is dt and b.shape == (width,) and b.is_contiguous() and b.get_device() == dev))
            and (stats is None or (stats.dtype is _F32 and stats.shape == (rows, 2)
                                   and stats.is_contiguous() and stats.get_device() == dev))):
        _on_gpu(x)
        xs, ys = _matrix16("x", x, rows, width, dt, dev), _matrix16("y", y, rows, width, dt, dev)
        _dense("w", w, (width,), dt, dev)
        _vector("b", b, width, dt, dev)
        if stats is not None:
            _dense("stats", stats, (rows, 2), torch.float32, dev)
    if rows == 1:  # a single row's stride says nothing
        xs = ys = (width + 7) // 8 * 8
    rc = (_lib or _load()).la_layernorm_rows(
        x.data_ptr(), w.data_ptr(), None if b is None else b.data_ptr(), y.data_ptr(),
        None if stats is None else stats.data_ptr(), rows, width, xs, ys, eps, LA_BF16 if dt is _BF16 else _dtype_code(x),
        _current_stream(dev) if stream is None and _current_stream is not None else _stream(stream))
    if rc:
        _check(rc)
    return y


def _matrix16(name, t, rows, cols, dtype, dev) -> int:
    """_matrix for calls whose rows start on 16 bytes: a single row goes with any stride."""
    s = _matrix(name, t, rows, cols, dtype, dev)
    return s if rows > 1 else (cols + 7) // 8 * 8


def layernorm_rows_backward_workspace_bytes(rows, width, dtype) -> int:
    """Bytes of workspace that layernorm_rows_backward needs."""
    return int(_load().la_layernorm_rows_backward_workspace_bytes(rows, width, _dtype_arg(dtype)))


def layernorm_rows_backward(x, w, stats, dy, dx, dw, db=None, *, dskip=None, workspace=None,
                            stream=None) -> None:
    """Gradients of layernorm_rows: dx [rows][width] (plus dskip [rows][width] where given: a gradient
    that reaches x past the norm; dx may be dy or dskip), dw and db fp32 [width]. x, w and stats are
    those of the forward call."""
    dev, dt = x.get_device(), x.dtype
    rows, width = x.shape
    (xs, x1), (ys, y1), (ds, d1) = x.stride(), dy.stride(), dx.stride()
    ss, s1 = (ds, 1) if dskip is None else dskip.stride()
    f32 = _F32
    # As in gated_scan: one look at everything, and only where something is unusual the checks that say what.
    if not (dev >= 0 and dev == _current_device() and x1 == y1 == d1 == s1 == 1 and dy.dtype is dt and dx.dtype is dt
            and dy.shape == (rows, width) and dx.shape == (rows, width) and dy.get_device() == dev
            and dx.get_device() == dev and w.dtype is dt and w.shape == (width,) and w.is_contiguous()
            and w.get_device() == dev and stats.dtype is f32 and stats.shape == (rows, 2) and stats.is_contiguous()
            and stats.get_device() == dev and dw.dtype is f32 and dw.shape == (width,) and dw.is_contiguous()
            and dw.get_device() == dev
            and (db is None or (db.dtype is f32 and db.shape == (width,) and db.is_contiguous() and db.get_device() == dev))
            and (dskip is None or (dskip.dtype is dt and dskip.shape == (rows, width) and dskip.get_device() == dev))
            and workspace is not None and workspace.is_contiguous() and workspace.get_device() == dev):
        _on_gpu(x)
        xs, ys, ds = (_matrix16(name, t, rows, width, dt, dev) for name, t in (("x", x), ("dy", dy), ("dx", dx)))
        ss = 0 if dskip is None else _matrix16("dskip", dskip, rows, width, dt, dev)
        _dense("w", w, (width,), dt, dev)
        _dense("stats", stats, (rows, 2), f32, dev)
        _dense("dw", dw, (width,), f32, dev)
        _vector("db", db, width, f32, dev)
        _room("workspace", workspace, dev)
    if rows == 1:  # a single row's stride says nothing
        xs = ys = ds = ss = (width + 7) // 8 * 8
    rc = (_lib or _load()).la_layernorm_rows_backward(
        x.data_ptr(), w.data_ptr(), stats.data_ptr(), dy.data_ptr(), None if dskip is None else dskip.data_ptr(),
        dx.data_ptr(), dw.data_ptr(), None if db is None else db.data_ptr(), rows, width, xs, ys, ss, ds, LA_BF16 if dt is _BF16 else _dtype_code(x),
        None if workspace is None else workspace.data_ptr(),
        0 if workspace is None else workspace.numel() * workspace.element_size(),
        _current_stream(dev) if stream is None and _current_stream is not None else _stream(stream))
    if rc:
        _check(rc)


def linear_saved_bytes(rows, outputs, act="none") -> int:
    """Bytes of the buffer that linear fills for linear_backward (0 without an activation)."""
    return int(_load().la_linear_saved_bytes(rows, outputs, _act_code(act)))


def linear(x, w, y=None, *, bias=None, residual=None, act="none", saved=None, stream=None):
    """y = act(x W^T + bias) + residual on the tensor cores (bf16, fp32 accumulation, one rounding).

    x [M][K], w [N][K] (a linear layer's [out][in] weight), bias [N], residual and y [M][N] (y may be
    residual, and defaults to a new tensor); any sizes, rows on 16 bytes. act: one of LA_ACTIVATIONS.
    saved: a buffer of linear_saved_bytes(...) when linear_backward is to follow. Returns y."""
    dev, bf16 = x.get_device(), _BF16
    M, K = x.shape
    N = w.shape[0]
    if y is None:
        y = _rows_like((M, N), bf16, x.device, stream)
    (xs, x1), (ws, w1), (ys, y1) = x.stride(), w.stride(), y.stride()
    rs, r1 = (ys, 1) if residual is None else residual.stride()
    # As in gated_scan: one look at everything, and only where something is unusual the checks that say what.
    if not (dev >= 0 and dev == _current_device() and x.dtype is bf16 and w.dtype is bf16 and y.dtype is bf16
            and w.shape == (N, K) and y.shape == (M, N) and x1 == w1 == y1 == r1 == 1
            and w.get_device() == dev and y.get_device() == dev
            and (residual is None or (residual.dtype is bf16 and residual.shape == (M, N)
                                      and residual.get_device() == dev))
            and (bias is None or (bias.dtype is bf16 and bias.shape == (N,) and bias.is_contiguous()
                                  and bias.get_device() == dev))
            and (saved is None or (saved.is_contiguous() and saved.get_device() == dev))):
        _on_gpu(x)
        xs, ws, ys = (_matrix16("x", x, M, K, bf16, dev), _matrix16("w", w, N, K, bf16, dev),
                      _matrix16("y", y, M, N, bf16, dev))
        rs = 0 if residual is None else _matrix16("residual", residual, M, N, bf16, dev)
        _vector("bias", bias, N, bf16, dev)
        _room("saved", saved, dev)
    if M == 1:  # a single row's stride says nothing
        xs, ys = (K + 7) // 8 * 8, (N + 7) // 8 * 8
        rs = ys
    if N == 1:
        ws = (K + 7) // 8 * 8
    code = LA_ACTIVATIONS.get(act)
    if code is None:
        _act_code(act)  # says what there is
    rc = (_lib or _load()).la_linear(
        x.data_ptr(), w.data_ptr(), None if bias is None else bias.data_ptr(),
        None if residual is None else residual.data_ptr(), y.data_ptr(), None if saved is None else saved.data_ptr(),
        0 if saved is None else saved.numel() * saved.element_size(), M, N, K, xs, ws, rs, ys,
        code,
        _current_stream(dev) if stream is None and _current_stream is not None else _stream(stream))
    if rc:
        _check(rc)
    return y


def linear_backward_workspace_bytes(rows, outputs, inputs, act="none") -> int:
    """Bytes of workspace that linear_backward needs, whichever gradients it is asked for (never 0)."""
    return int(_load().la_linear_backward_workspace_bytes(rows, outputs, inputs, _act_code(act)))


def linear_backward(x, w, saved, dy, dx=None, dw=None, *, dbias=None, act="none", workspace=None,
                    stream=None) -> None:
    """Gradients of linear: dx [M][K], dw [N][K] and dbias [N] (bf16; those that are given) from dy
    [M][N]; the residual's is dy itself. x, w, saved (None without an activation) and act are those of
    the forward call. workspace: a buffer of linear_backward_workspace_bytes(...), which every call needs."""
    dev, bf16 = x.get_device(), _BF16
    M, K = x.shape
    N = w.shape[0]
    (xs, x1), (ws, w1), (ys, y1) = x.stride(), w.stride(), dy.stride()
    ds, d1 = (xs, 1) if dx is None else dx.stride()
    gs, g1 = (ws, 1) if dw is None else dw.stride()
    # As in gated_scan: one look at everything, and only where something is unusual the checks that say what.
    if not (dev >= 0 and dev == _current_device() and x1 == w1 == y1 == d1 == g1 == 1 and x.dtype is bf16
            and w.dtype is bf16 and dy.dtype is bf16 and w.shape == (N, K) and dy.shape == (M, N)
            and w.get_device() == dev and dy.get_device() == dev
            and (dx is None or (dx.dtype is bf16 and dx.shape == (M, K) and dx.get_device() == dev))
            and (dw is None or (dw.dtype is bf16 and dw.shape == (N, K) and dw.get_device() == dev))
            and (dbias is None or (dbias.dtype is bf16 and dbias.shape == (N,) and dbias.is_contiguous()
                                   and dbias.get_device() == dev))
            and (saved is None or (saved.is_contiguous() and saved.get_device() == dev))
            and (workspace is None or (workspace.is_contiguous() and workspace.get_device() == dev))):
        _on_gpu(x)
        xs, ws, ys = (_matrix16("x", x, M, K, bf16, dev), _matrix16("w", w, N, K, bf16, dev),
                      _matrix16("dy", dy, M, N, bf16, dev))
        ds = 0 if dx is None else _matrix16("dx", dx, M, K, bf16, dev)
        gs = 0 if dw is None else _matrix16("dw", dw, N, K, bf16, dev)
        _vector("dbias", dbias, N, bf16, dev)
        _room("saved", saved, dev)
        _room("workspace", workspace, dev)
    if M == 1:  # a single row's stride says nothing
        xs = ds = (K + 7) // 8 * 8
        ys = (N + 7) // 8 * 8
    if N == 1:
        ws = gs = (K + 7) // 8 * 8
    code = LA_ACTIVATIONS.get(act)
    if code is None:
        _act_code(act)  # says what there is
    rc = (_lib or _load()).la_linear_backward(
        x.data_ptr(), w.data_ptr(), None if saved is None else saved.data_ptr(),
        0 if saved is None else saved.numel() * saved.element_size(), dy.data_ptr(), None if dx is None else dx.data_ptr(),
        None if dw is None else dw.data_ptr(), None if dbias is None else dbias.data_ptr(), M, N, K, xs, ws, ys, ds, gs,
        code, None if workspace is None else workspace.data_ptr(),
        0 if workspace is None else workspace.numel() * workspace.element_size(),
        _current_stream(dev) if stream is None and _current_stream is not None else _stream(stream))
    if rc:
        _check(rc)


def gated_ffn_saved_bytes(rows, hidden) -> int:
    """Bytes of the buffer that gated_ffn fills for gated_ffn_backward."""
    return int(_load().la_gated_ffn_saved_bytes(rows, hidden))


def gated_ffn(x, w_gate, w_up, h=None, *, act="silu", saved=None, stream=None):
    """h = act(x Wg^T) * (x Wu^T): both projections, the activation and the product in one kernel.

    x [M][K], w_gate and w_up [F][K] (w[:F] and w[F:] of a packed weight are fine), h [M][F] (a new
    tensor by default): bf16, any sizes, rows on 16 bytes. act: one of LA_ACTIVATIONS. saved: a buffer
    of gated_ffn_saved_bytes(...) when gated_ffn_backward is to follow. The projection back is
    linear(h, w_down, residual=...). Returns h."""
    dev, bf16 = x.get_device(), _BF16
    M, K = x.shape
    F = w_gate.shape[0]
    if h is None:
        h = _rows_like((M, F), bf16, x.device, stream)
    (xs, x1), (gs, g1), (us, u1), (hs, h1) = x.stride(), w_gate.stride(), w_up.stride(), h.stride()
    # As in gated_scan: one look at everything, and only where something is unusual the checks that say what.
    if not (dev >= 0 and dev == _current_device() and x.dtype is bf16 and w_gate.dtype is bf16 and w_up.dtype is bf16
            and h.dtype is bf16 and w_gate.shape == (F, K) and w_up.shape == (F, K) and h.shape == (M, F)
            and x1 == g1 == u1 == h1 == 1 and w_gate.get_device() == dev
            and w_up.get_device() == dev and h.get_device() == dev
            and (saved is None or (saved.is_contiguous() and saved.get_device() == dev))):
        _on_gpu(x)
        xs, hs = _matrix16("x", x, M, K, bf16, dev), _matrix16("h", h, M, F, bf16, dev)
        gs, us = _matrix16("w_gate", w_gate, F, K, bf16, dev), _matrix16("w_up", w_up, F, K, bf16, dev)
        _room("saved", saved, dev)
    if M == 1:  # a single row's stride says nothing
        xs, hs = (K + 7) // 8 * 8, (F + 7) // 8 * 8
    if F == 1:
        gs = us = (K + 7) // 8 * 8
    code = LA_ACTIVATIONS.get(act)
    if code is None:
        _act_code(act)  # says what there is
    rc = (_lib or _load()).la_gated_ffn(
        x.data_ptr(), w_gate.data_ptr(), w_up.data_ptr(), h.data_ptr(), None if saved is None else saved.data_ptr(),
        0 if saved is None else saved.numel() * saved.element_size(), M, F, K, xs, gs, us, hs,
        code,
        _current_stream(dev) if stream is None and _current_stream is not None else _stream(stream))
    if rc:
        _check(rc)
    return h


def gated_ffn_backward_workspace_bytes(rows, hidden, inputs) -> int:
    """Bytes of workspace that gated_ffn_backward needs."""
    return int(_load().la_gated_ffn_backward_workspace_bytes(rows, hidden, inputs))


def gated_ffn_backward(x, w_gate, w_up, saved, dh, dx=None, dw_gate=None, dw_up=None, *, act="silu",
                       workspace=None, stream=None) -> None:
    """Gradients of gated_ffn: dx [M][K] and/or dw_gate and dw_up [F][K] (bf16) from dh [M][F]. x, the
    weights, saved and act are those of the forward call."""
    dev, bf16 = x.get_device(), _BF16
    M, K = x.shape
    F = w_gate.shape[0]
    (xs, x1), (gs, g1), (us, u1), (hs, h1) = x.stride(), w_gate.stride(), w_up.stride(), dh.stride()
    ds, d1 = (xs, 1) if dx is None else dx.stride()
    (dgs, dg1), (dus, du1) = ((gs, 1), (us, 1)) if dw_gate is None or dw_up is None else (dw_gate.stride(), dw_up.stride())
    # As in gated_scan: one look at everything, and only where something is unusual the checks that say what.
    if not (dev >= 0 and dev == _current_device() and x1 == g1 == u1 == h1 == d1 == dg1 == du1 == 1 and x.dtype is bf16
            and w_gate.dtype is bf16 and w_up.dtype is bf16 and dh.dtype is bf16 and w_gate.shape == (F, K)
            and w_up.shape == (F, K) and dh.shape == (M, F) and w_gate.get_device() == dev
            and w_up.get_device() == dev and dh.get_device() == dev
            and (dx is None or (dx.dtype is bf16 and dx.shape == (M, K) and dx.get_device() == dev))
            and ((dw_gate is None and dw_up is None)
                 or (dw_gate is not None and dw_up is not None and dw_gate.dtype is bf16 and dw_up.dtype is bf16
                     and dw_gate.shape == (F, K) and dw_up.shape == (F, K) and dw_gate.get_device() == dev
                     and dw_up.get_device() == dev))
            and saved is not None and saved.is_contiguous() and saved.get_device() == dev
            and workspace is not None and workspace.is_contiguous() and workspace.get_device() == dev):
        _on_gpu(x)
        xs, hs = _matrix16("x", x, M, K, bf16, dev), _matrix16("dh", dh, M, F, bf16, dev)
        gs, us = _matrix16("w_gate", w_gate, F, K, bf16, dev), _matrix16("w_up", w_up, F, K, bf16, dev)
        ds, dgs, dus = (0 if t is None else _matrix16(name, t, r, K, bf16, dev)
                        for name, t, r in (("dx", dx, M), ("dw_gate", dw_gate, F), ("dw_up", dw_up, F)))
        _room("saved", saved, dev)
        _room("workspace", workspace, dev)
    if M == 1:  # a single row's stride says nothing
        xs = ds = (K + 7) // 8 * 8
        hs = (F + 7) // 8 * 8
    if F == 1:
        gs = us = dgs = dus = (K + 7) // 8 * 8
    code = LA_ACTIVATIONS.get(act)
    if code is None:
        _act_code(act)  # says what there is
    rc = (_lib or _load()).la_gated_ffn_backward(
        x.data_ptr(), w_gate.data_ptr(), w_up.data_ptr(), None if saved is None else saved.data_ptr(),
        0 if saved is None else saved.numel() * saved.element_size(), dh.data_ptr(), None if dx is None else dx.data_ptr(),
        None if dw_gate is None else dw_gate.data_ptr(), None if dw_up is None else dw_up.data_ptr(), M, F, K, xs, gs, us, hs,
        ds, dgs, dus, code, None if workspace is None else workspace.data_ptr(),
        0 if workspace is None else workspace.numel() * workspace.element_size(),
        _current_stream(dev) if stream is None and _current_stream is not None else _stream(stream))
    if rc:
        _check(rc)

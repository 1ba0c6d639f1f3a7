"""Thin ctypes binding over libfa.so (include/fa.h).

Argument marshalling only: every step of attention runs in the CUDA kernels
of the library. The functions named like the C ABI (``fa_fwd``, ``fa_fwd_kv``,
``fa_fwd_kv_workspace_bytes``, ``fa_fwd_fp8``, ``fa_fwd_dropout``, ``fa_bwd_dropout``, ``fa_bwd``, ``fa_bwd_workspace_bytes``, ``fa_bwd_kv``,
``fa_bwd_kv_workspace_bytes``,
``fa_status_string``, ``fa_device_status``, ``fa_bwd_noalloc``, ``fa_test_arm_fault``, ``fa_paged_plan``,
``fa_paged_store``, ``fa_fwd_paged``, ``fa_fwd_paged_workspace_bytes``, ``fa_fwd_paged_window``, ``fa_rope_fwd``,
``fa_rope_bwd``, ``fa_rope_bwd_workspace_bytes``, ``fa_paged_positions``, ``fa_paged_rope_store``, ``fa_fwd_window``,
``fa_bwd_window``, ``fa_bwd_window_workspace_bytes``) take either
torch CUDA tensors or raw device addresses (ints). ``attention`` is a
differentiable torch.autograd.Function over the forward and backward calls (``attention_window`` and ``rope`` likewise);
``forward``,
``forward_kv``, ``forward_fp8``, ``forward_dropout``, ``backward``, ``backward_kv`` and
``backward_dropout`` are conveniences that
allocate the outputs with torch, and so do ``forward_window`` and ``backward_window`` (attention in a sliding window) and
``forward_rope`` and ``backward_rope`` (rotation by position, with the norm of each head). ``paged_plan``, ``paged_positions``,
``paged_store``, ``paged_rope_store`` and ``forward_paged`` do the same for serving from a paged key/value cache.

If the library has not been built, or cannot be loaded, every call raises:
there is no fallback implementation.
"""
from __future__ import annotations

import ctypes
import functools
import math
import os
import threading

from . import build as _build

FA_OK = 0
FA_ERR_INVALID_ARG = 1
FA_ERR_UNSUPPORTED = 2
FA_ERR_MISALIGNED = 3
FA_ERR_WORKSPACE = 4
FA_ERR_LAUNCH = 5
FA_ERR_TIMEOUT = 6
FA_ERR_NO_PAGES = 7

EXPORTED = ("fa_fwd", "fa_fwd_kv", "fa_fwd_kv_workspace_bytes", "fa_fwd_fp8", "fa_fwd_dropout", "fa_bwd",
            "fa_bwd_workspace_bytes", "fa_bwd_kv", "fa_bwd_kv_workspace_bytes", "fa_bwd_dropout", "fa_status_string",
            "fa_device_status", "fa_bwd_noalloc", "fa_test_arm_fault", "fa_paged_plan", "fa_paged_store",
            "fa_fwd_paged", "fa_fwd_paged_workspace_bytes", "fa_fwd_paged_window", "fa_rope_fwd", "fa_rope_bwd",
            "fa_rope_bwd_workspace_bytes", "fa_paged_positions", "fa_paged_rope_store", "fa_fwd_window", "fa_bwd_window",
            "fa_bwd_window_workspace_bytes")

_lock = threading.Lock()
_lib = None


class Heads(ctypes.Structure):
    """fa_heads: rows [B, H, N, d] at any strides (in elements)."""

    _fields_ = [("data", ctypes.c_void_p), ("stride_b", ctypes.c_longlong), ("stride_h", ctypes.c_longlong),
                ("stride_n", ctypes.c_longlong)]


class FAError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {status_string(status)} (status {status})")


def lib_path() -> str:
    return _build.LIB


def load(path: str | None = None):
    """Load libfa.so (building it first if it is missing) and declare the signatures."""
    global _lib
    with _lock:
        if _lib is not None and path is None:
            return _lib
        p = path or _build.LIB
        if not os.path.exists(p):
            _build.build()
        lib = ctypes.CDLL(p)
        vp, c_int, c_float, c_size_t = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
        lib.fa_fwd.argtypes = [vp, vp, vp, vp, vp, c_int, c_int, c_int, c_int, c_float, c_int, vp]
        lib.fa_fwd.restype = c_int
        lib.fa_bwd.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, c_int, c_int, c_int, c_int, c_float, c_int, vp,
                               c_size_t, vp]
        lib.fa_bwd.restype = c_int
        lib.fa_fwd_kv.argtypes = [vp, vp, vp, vp, vp, c_int, c_int, c_int, c_int, c_int, c_float, c_int, vp, vp, vp,
                                  c_size_t, vp]
        lib.fa_fwd_kv.restype = c_int
        lib.fa_fwd_fp8.argtypes = [vp, vp, vp, c_float, c_float, c_float, vp, vp, c_int, c_int, c_int, c_int, c_float,
                                   c_int, vp]
        lib.fa_fwd_fp8.restype = c_int
        c_u64, c_u32 = ctypes.c_ulonglong, ctypes.c_uint
        lib.fa_fwd_dropout.argtypes = [vp, vp, vp, vp, vp, c_int, c_int, c_int, c_int, c_float, c_int, c_int, c_u64,
                                       c_u32, vp]
        lib.fa_fwd_dropout.restype = c_int
        lib.fa_bwd_dropout.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, c_int, c_int, c_int, c_int, c_float, c_int,
                                       c_int, c_u64, c_u32, vp, c_size_t, vp]
        lib.fa_bwd_dropout.restype = c_int
        lib.fa_fwd_kv_workspace_bytes.argtypes = [c_int, c_int, c_int, c_int, c_int]
        lib.fa_fwd_kv_workspace_bytes.restype = c_size_t
        lib.fa_bwd_kv.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, c_int, c_int, c_int, c_int, c_int, c_float, c_int,
                                  vp, vp, vp, c_size_t, vp]
        lib.fa_bwd_kv.restype = c_int
        lib.fa_bwd_kv_workspace_bytes.argtypes = [c_int, c_int, c_int, c_int, c_int]
        lib.fa_bwd_kv_workspace_bytes.restype = c_size_t
        lib.fa_bwd_workspace_bytes.argtypes = [c_int, c_int, c_int, c_int]
        lib.fa_bwd_workspace_bytes.restype = c_size_t
        lib.fa_status_string.argtypes = [c_int]
        lib.fa_status_string.restype = ctypes.c_char_p
        lib.fa_device_status.argtypes = [c_int]
        lib.fa_device_status.restype = c_int
        lib.fa_test_arm_fault.argtypes = [c_int]
        lib.fa_test_arm_fault.restype = c_int
        c_i64 = ctypes.c_longlong
        lib.fa_paged_plan.argtypes = [vp, vp, c_int, c_int, vp, c_int, vp, vp, c_int, vp, vp, vp, c_int, vp, vp]
        lib.fa_paged_plan.restype = c_int
        lib.fa_paged_store.argtypes = [vp, vp, c_i64, c_i64, vp, c_int, c_int, c_int, vp, vp, c_int, c_int, c_int,
                                       c_float, c_float, vp]
        lib.fa_paged_store.restype = c_int
        lib.fa_fwd_paged_workspace_bytes.argtypes = [c_int, c_int, c_int, c_int, c_int, c_int]
        lib.fa_fwd_paged_workspace_bytes.restype = c_size_t
        lib.fa_fwd_paged.argtypes = [vp, c_i64, vp, vp, c_int, c_float, c_float, vp, c_int, vp, vp, vp, vp, c_int,
                                     c_int, c_int, c_int, c_int, c_int, c_int, c_int, c_float, c_int, vp, c_size_t, vp]
        lib.fa_fwd_paged.restype = c_int
        lib.fa_fwd_paged_window.argtypes = [vp, c_i64, vp, vp, c_int, c_float, c_float, vp, c_int, vp, vp, vp, vp, c_int,
                                            c_int, c_int, c_int, c_int, c_int, c_int, c_int, c_float, c_int, c_int, vp,
                                            c_size_t, vp]
        lib.fa_fwd_paged_window.restype = c_int
        heads = ctypes.POINTER(Heads)
        lib.fa_rope_fwd.argtypes = [heads, heads, heads, heads, vp, vp, c_int, c_float, vp, c_int, c_int, c_float, vp, c_i64,
                                    c_int, c_int, c_int, c_int, c_int, vp]
        lib.fa_rope_fwd.restype = c_int
        lib.fa_rope_bwd_workspace_bytes.argtypes = [c_int, c_int, c_int]
        lib.fa_rope_bwd_workspace_bytes.restype = c_size_t
        lib.fa_rope_bwd.argtypes = [heads, heads, heads, heads, heads, heads, vp, vp, c_int, c_float, vp, vp, vp, c_int, c_int,
                                    c_float, vp, c_i64, c_int, c_int, c_int, c_int, c_int, vp, c_size_t, vp]
        lib.fa_rope_bwd.restype = c_int
        lib.fa_paged_positions.argtypes = [vp, vp, c_int, vp, c_int, vp]
        lib.fa_paged_positions.restype = c_int
        lib.fa_paged_rope_store.argtypes = [vp, vp, vp, c_i64, c_i64, c_i64, vp, vp, vp, c_int, c_int, c_float, vp, vp, c_int,
                                            c_float, vp, c_i64, c_int, c_int, c_int, c_int, vp, vp, c_int, c_int, c_int,
                                            c_float, c_float, vp]
        lib.fa_paged_rope_store.restype = c_int
        lib.fa_fwd_window.argtypes = [vp, vp, vp, vp, vp, c_int, c_int, c_int, c_int, c_int, c_int, c_float, c_int, c_int, vp,
                                      vp, vp]
        lib.fa_fwd_window.restype = c_int
        lib.fa_bwd_window_workspace_bytes.argtypes = [c_int] * 8
        lib.fa_bwd_window_workspace_bytes.restype = c_size_t
        lib.fa_bwd_window.argtypes = [vp] * 9 + [c_int] * 6 + [c_float, c_int, c_int, vp, vp, vp, c_size_t, vp]
        lib.fa_bwd_window.restype = c_int
        if path is None:
            _lib = lib
        return lib


def _addr(x) -> int | None:
    if x is None:
        return None
    if isinstance(x, int):
        return x
    return int(x.data_ptr())


def _stream(stream) -> int | None:
    if stream is None:
        import torch

        return int(torch.cuda.current_stream().cuda_stream)
    if isinstance(stream, int):
        return stream
    return int(stream.cuda_stream)


def status_string(status: int) -> str:
    return load().fa_status_string(int(status)).decode()


fa_status_string = status_string


def fa_fwd(q, k, v, o, lse, B: int, H: int, N: int, d: int, scale: float, causal: bool, stream=None) -> int:
    return int(load().fa_fwd(_addr(q), _addr(k), _addr(v), _addr(o), _addr(lse), B, H, N, d, float(scale),
                             int(bool(causal)), _stream(stream)))


def fa_fwd_kv_workspace_bytes(B: int, H: int, Nq: int, Nk: int, d: int) -> int:
    return int(load().fa_fwd_kv_workspace_bytes(B, H, Nq, Nk, d))


def fa_fwd_kv(q, k, v, o, lse, B: int, H: int, Nq: int, Nk: int, d: int, scale: float, causal: bool,
              seqlens_q=None, seqlens_k=None, workspace=None, workspace_bytes: int = 0, stream=None) -> int:
    return int(load().fa_fwd_kv(_addr(q), _addr(k), _addr(v), _addr(o), _addr(lse), B, H, Nq, Nk, d, float(scale),
                                int(bool(causal)), _addr(seqlens_q), _addr(seqlens_k), _addr(workspace),
                                int(workspace_bytes), _stream(stream)))


def fa_fwd_fp8(q, k, v, descale_q: float, descale_k: float, descale_v: float, o, lse, B: int, H: int, N: int, d: int,
               scale: float, causal: bool, stream=None) -> int:
    return int(load().fa_fwd_fp8(_addr(q), _addr(k), _addr(v), float(descale_q), float(descale_k), float(descale_v),
                                 _addr(o), _addr(lse), B, H, N, d, float(scale), int(bool(causal)), _stream(stream)))


def fa_fwd_dropout(q, k, v, o, lse, B: int, H: int, N: int, d: int, scale: float, causal: bool, p256: int, seed: int,
                   offset: int = 0, stream=None) -> int:
    return int(load().fa_fwd_dropout(_addr(q), _addr(k), _addr(v), _addr(o), _addr(lse), B, H, N, d, float(scale),
                                     int(bool(causal)), int(p256), int(seed), int(offset), _stream(stream)))


def fa_bwd_dropout(q, k, v, o, lse, dO, dq, dk, dv, B: int, H: int, N: int, d: int, scale: float, causal: bool,
                   p256: int, seed: int, offset: int, workspace, workspace_bytes: int, stream=None) -> int:
    return int(load().fa_bwd_dropout(_addr(q), _addr(k), _addr(v), _addr(o), _addr(lse), _addr(dO), _addr(dq),
                                     _addr(dk), _addr(dv), B, H, N, d, float(scale), int(bool(causal)), int(p256),
                                     int(seed), int(offset), _addr(workspace), int(workspace_bytes), _stream(stream)))


def fa_bwd_workspace_bytes(B: int, H: int, N: int, d: int) -> int:
    return int(load().fa_bwd_workspace_bytes(B, H, N, d))


def fa_bwd(q, k, v, o, lse, dO, dq, dk, dv, B: int, H: int, N: int, d: int, scale: float, causal: bool,
           workspace, workspace_bytes: int, stream=None) -> int:
    return int(load().fa_bwd(_addr(q), _addr(k), _addr(v), _addr(o), _addr(lse), _addr(dO), _addr(dq), _addr(dk),
                             _addr(dv), B, H, N, d, float(scale), int(bool(causal)), _addr(workspace),
                             int(workspace_bytes), _stream(stream)))


def fa_bwd_kv_workspace_bytes(B: int, H: int, Nq: int, Nk: int, d: int) -> int:
    return int(load().fa_bwd_kv_workspace_bytes(B, H, Nq, Nk, d))


def fa_bwd_kv(q, k, v, o, lse, dO, dq, dk, dv, B: int, H: int, Nq: int, Nk: int, d: int, scale: float, causal: bool,
              seqlens_q, seqlens_k, workspace, workspace_bytes: int, stream=None) -> int:
    return int(load().fa_bwd_kv(_addr(q), _addr(k), _addr(v), _addr(o), _addr(lse), _addr(dO), _addr(dq), _addr(dk),
                                _addr(dv), B, H, Nq, Nk, d, float(scale), int(bool(causal)), _addr(seqlens_q),
                                _addr(seqlens_k), _addr(workspace), int(workspace_bytes), _stream(stream)))


def fa_device_status(reset: bool = True) -> int:
    return int(load().fa_device_status(int(bool(reset))))


def fa_test_arm_fault(kind: int) -> int:
    """Test hook: arm a one-shot fault for the next forward launch (1: withhold the first query
    tile, so the kernels' bounded wait runs out and fa_device_status reports FA_ERR_TIMEOUT)."""
    return int(load().fa_test_arm_fault(int(kind)))


def _lens(x, B: int):
    """A per-sequence length tensor as the library takes it: int32, [B], contiguous, on the GPU."""
    if x is None:
        return None
    import torch

    if x.dtype != torch.int32 or tuple(x.shape) != (B,) or not x.is_contiguous() or not x.is_cuda:
        raise ValueError("sequence lengths must be a contiguous int32 CUDA tensor of shape [B]")
    return x


def _shape(q):
    if q.dim() != 4:
        raise ValueError("expected [B, H, N, d] tensors")
    return tuple(int(s) for s in q.shape)


def _bf16(*ts):
    """The 16-bit entry points read raw device memory: bf16, contiguous, on the GPU."""
    import torch

    for t in ts:
        if t.dtype != torch.bfloat16 or not t.is_contiguous() or not t.is_cuda:
            raise ValueError("expected contiguous bf16 CUDA tensors")


_refused_fn = None


def _once(backward):
    """Decorator of a backward method: gradients that it makes under create_graph stand in the graph behind everything they were made of
    (its arguments and saved tensors, so also where the loss is linear in the outputs), and differentiating them raises."""
    global _refused_fn
    import torch

    if _refused_fn is None:
        class _Refused(torch.autograd.Function):
            @staticmethod
            def forward(ctx, n, *tensors):
                return tensors[:n]

            @staticmethod
            def backward(ctx, *_):
                raise RuntimeError("second derivatives of attention, attention_window and rope are not implemented")

        _refused_fn = _Refused

    @functools.wraps(backward)
    def once(ctx, *grads):
        with torch.no_grad():
            r = backward(ctx, *grads)
        return _refused_fn.apply(len(r), *r, *grads, *ctx.saved_tensors) if torch.is_grad_enabled() else r

    return once


_attention_fn = None


def _gradient(x):
    """A gradient as the attention kernels read it: bf16, contiguous and 16-byte aligned (a contiguous view may begin anywhere)."""
    import torch

    x = x.to(torch.bfloat16).contiguous()
    return x if x.data_ptr() % 16 == 0 else x.clone()


def attention(q, k, v, causal: bool = False, scale: float | None = None, dropout_p256: int = 0, seed: int = 0,
              offset: int = 0):
    """Differentiable attention o = softmax(scale q k^T [causal]) v (with dropout of probability
    dropout_p256 / 256 after the softmax if given) for q, k, v of shape [B, H, N, d], bf16: a
    torch.autograd.Function whose forward runs fa_fwd (fa_fwd_dropout) and whose backward runs fa_bwd
    (fa_bwd_dropout, the same mask made again from seed and offset). Gradients of the gradients are refused."""
    global _attention_fn
    if _attention_fn is None:
        import torch

        class _Attention(torch.autograd.Function):
            @staticmethod
            def forward(ctx, q, k, v, causal, scale, p256, seed, offset):
                if p256:
                    o, lse = forward_dropout(q, k, v, p256, seed, offset, causal=causal, scale=scale)
                else:
                    o, lse = forward(q, k, v, causal=causal, scale=scale)
                ctx.save_for_backward(q, k, v, o, lse)
                ctx.args = (causal, scale, p256, seed, offset)
                return o

            @staticmethod
            @_once
            def backward(ctx, dO):
                q, k, v, o, lse = ctx.saved_tensors
                causal, scale, p256, seed, offset = ctx.args
                dO = _gradient(dO)
                if p256:
                    dq, dk, dv = backward_dropout(q, k, v, o, lse, dO, p256, seed, offset, causal=causal, scale=scale)
                else:
                    dq, dk, dv = backward(q, k, v, o, lse, dO, causal=causal, scale=scale)
                return dq, dk, dv, None, None, None, None, None

        _attention_fn = _Attention
    _bf16(q, k, v)
    scale = 1.0 / math.sqrt(int(q.shape[-1])) if scale is None else scale
    return _attention_fn.apply(q, k, v, bool(causal), float(scale), int(dropout_p256), int(seed), int(offset))


def forward(q, k, v, causal: bool = False, scale: float | None = None, stream=None):
    """Allocate o (bf16) and lse (fp32) with torch and run fa_fwd. Returns (o, lse)."""
    import torch

    _bf16(q, k, v)
    B, H, N, d = _shape(q)
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    o = torch.empty_like(q)
    lse = torch.empty((B, H, N), dtype=torch.float32, device=q.device)
    st = fa_fwd(q, k, v, o, lse, B, H, N, d, scale, causal, stream)
    if st != FA_OK:
        raise FAError(st, "fa_fwd")
    return o, lse


def forward_fp8(q8, k8, v8, descale_q: float, descale_k: float, descale_v: float, causal: bool = False,
                scale: float | None = None, stream=None):
    """8-bit forward: q8, k8, v8 are [B, H, N, 128] tensors of E4M3 codes (uint8 or float8_e4m3fn) with
    per-tensor dequantisation factors; allocate o (bf16) and lse (fp32) and run fa_fwd_fp8. Returns (o, lse)."""
    import torch

    B, H, N, d = _shape(q8)
    for x in (q8, k8, v8):
        if x.element_size() != 1 or not x.is_contiguous():
            raise ValueError("expected contiguous one-byte E4M3 tensors")
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    o = torch.empty((B, H, N, d), dtype=torch.bfloat16, device=q8.device)
    lse = torch.empty((B, H, N), dtype=torch.float32, device=q8.device)
    st = fa_fwd_fp8(q8, k8, v8, descale_q, descale_k, descale_v, o, lse, B, H, N, d, scale, causal, stream)
    if st != FA_OK:
        raise FAError(st, "fa_fwd_fp8")
    return o, lse


def forward_dropout(q, k, v, p256: int, seed: int, offset: int = 0, causal: bool = False, scale: float | None = None,
                    stream=None):
    """Forward with dropout probability p256 / 256 (Philox mask of seed, offset). Returns (o, lse)."""
    import torch

    _bf16(q, k, v)
    B, H, N, d = _shape(q)
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    o = torch.empty_like(q)
    lse = torch.empty((B, H, N), dtype=torch.float32, device=q.device)
    st = fa_fwd_dropout(q, k, v, o, lse, B, H, N, d, scale, causal, p256, seed, offset, stream)
    if st != FA_OK:
        raise FAError(st, "fa_fwd_dropout")
    return o, lse


def backward_dropout(q, k, v, o, lse, dO, p256: int, seed: int, offset: int = 0, causal: bool = False,
                     scale: float | None = None, stream=None):
    """Backward of forward_dropout with the same (p256, seed, offset). Returns (dq, dk, dv)."""
    import torch

    _bf16(q, k, v, o, dO)
    B, H, N, d = _shape(q)
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    need = fa_bwd_workspace_bytes(B, H, N, d)
    ws = torch.empty(need, dtype=torch.uint8, device=q.device)
    st = fa_bwd_dropout(q, k, v, o, lse, dO, dq, dk, dv, B, H, N, d, scale, causal, p256, seed, offset, ws, need,
                        stream)
    if st != FA_OK:
        raise FAError(st, "fa_bwd_dropout")
    return dq, dk, dv


def forward_kv(q, k, v, causal: bool = False, scale: float | None = None, split: bool = True, seqlens_q=None,
               seqlens_k=None, stream=None):
    """Nq query rows against Nk keys: allocate o, lse (and, with ``split``, the key-range
    workspace fa_fwd_kv_workspace_bytes asks for) with torch and run fa_fwd_kv. ``seqlens_q`` /
    ``seqlens_k`` are optional int32 [B] device tensors (padding masks). Returns (o, lse)."""
    import torch

    _bf16(q, k, v)
    B, H, Nq, d = _shape(q)
    Nk = int(k.shape[2])
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    o = torch.empty_like(q)
    lse = torch.empty((B, H, Nq), dtype=torch.float32, device=q.device)
    need = fa_fwd_kv_workspace_bytes(B, H, Nq, Nk, d) if split else 0
    ws = torch.empty(need, dtype=torch.uint8, device=q.device) if need else None
    st = fa_fwd_kv(q, k, v, o, lse, B, H, Nq, Nk, d, scale, causal, _lens(seqlens_q, B), _lens(seqlens_k, B), ws,
                   need, stream)
    if st != FA_OK:
        raise FAError(st, "fa_fwd_kv")
    return o, lse


def backward(q, k, v, o, lse, dO, causal: bool = False, scale: float | None = None, workspace=None, stream=None):
    """Allocate dq, dk, dv (and the workspace if none is given) and run fa_bwd."""
    import torch

    _bf16(q, k, v, o, dO)
    B, H, N, d = _shape(q)
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    need = fa_bwd_workspace_bytes(B, H, N, d)
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    st = fa_bwd(q, k, v, o, lse, dO, dq, dk, dv, B, H, N, d, scale, causal, workspace,
                workspace.numel() * workspace.element_size(), stream)
    if st != FA_OK:
        raise FAError(st, "fa_bwd")
    return dq, dk, dv


def backward_kv(q, k, v, o, lse, dO, causal: bool = False, scale: float | None = None, seqlens_q=None,
                seqlens_k=None, stream=None):
    """Nq query rows against Nk keys: allocate dq, dk, dv and the workspace with torch and run fa_bwd_kv
    (``seqlens_q`` / ``seqlens_k`` as in forward_kv)."""
    import torch

    _bf16(q, k, v, o, dO)
    B, H, Nq, d = _shape(q)
    Nk = int(k.shape[2])
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    need = fa_bwd_kv_workspace_bytes(B, H, Nq, Nk, d)
    ws = torch.empty(need, dtype=torch.uint8, device=q.device)
    st = fa_bwd_kv(q, k, v, o, lse, dO, dq, dk, dv, B, H, Nq, Nk, d, scale, causal, _lens(seqlens_q, B),
                   _lens(seqlens_k, B), ws, need, stream)
    if st != FA_OK:
        raise FAError(st, "fa_bwd_kv")
    return dq, dk, dv


# Largest scratch fa_bwd_noalloc holds per device (FA_BWD_NOALLOC_MAX_SCRATCH_BYTES in include/fa.h).
FA_BWD_NOALLOC_MAX_SCRATCH_BYTES = 32 << 20


def fa_bwd_noalloc(q, k, v, o, lse, dO, dq, dk, dv, B: int, H: int, N: int, d: int, scale: float, causal: bool,
                   stream=None) -> int:
    """fa_bwd without a workspace, for callers that cannot allocate device memory.

    The library keeps the scratch in a fixed device array of
    FA_BWD_NOALLOC_MAX_SCRATCH_BYTES; larger shapes return FA_ERR_WORKSPACE.
    The first call on a device looks up that array's address, so make it
    before any stream capture; calls that may overlap on one device race on
    the shared array.
    """
    lib = load()
    fn = lib.fa_bwd_noalloc
    if fn.argtypes is None:
        vp, c_int, c_float = ctypes.c_void_p, ctypes.c_int, ctypes.c_float
        fn.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, c_int, c_int, c_int, c_int, c_float, c_int, vp]
        fn.restype = c_int
    return int(fn(_addr(q), _addr(k), _addr(v), _addr(o), _addr(lse), _addr(dO), _addr(dq), _addr(dk), _addr(dv),
                  B, H, N, d, float(scale), int(bool(causal)), _stream(stream)))


# ---------------------------------------------------------------- paged key/value cache
def fa_paged_plan(ctx_lens, new_lens, R: int, page_size: int, free_pages, n_free: int, free_head, block_table,
                  max_pages: int, query_start, seq_lens, slots, T: int, pages_taken, stream=None) -> int:
    return load().fa_paged_plan(_addr(ctx_lens), _addr(new_lens), R, page_size, _addr(free_pages), n_free,
                                _addr(free_head), _addr(block_table), max_pages, _addr(query_start), _addr(seq_lens),
                                _addr(slots), T, _addr(pages_taken), _stream(stream))


def fa_paged_store(k, v, k_stride: int, v_stride: int, slots, T: int, Hkv: int, d: int, k_cache, v_cache,
                   num_pages: int, page_size: int, fp8: bool, descale_k: float, descale_v: float, stream=None) -> int:
    return load().fa_paged_store(_addr(k), _addr(v), k_stride, v_stride, _addr(slots), T, Hkv, d, _addr(k_cache),
                                 _addr(v_cache), num_pages, page_size, int(bool(fp8)), descale_k, descale_v,
                                 _stream(stream))


def fa_fwd_paged_workspace_bytes(T: int, R: int, Hq: int, Hkv: int, d: int, max_new: int) -> int:
    return int(load().fa_fwd_paged_workspace_bytes(T, R, Hq, Hkv, d, max_new))


def fa_fwd_paged(q, q_stride: int, k_cache, v_cache, fp8: bool, descale_k: float, descale_v: float, block_table,
                 max_pages: int, query_start, seq_lens, o, lse, T: int, R: int, Hq: int, Hkv: int, d: int,
                 num_pages: int, page_size: int, max_new: int, scale: float, causal: bool, workspace,
                 workspace_bytes: int, stream=None) -> int:
    return load().fa_fwd_paged(_addr(q), q_stride, _addr(k_cache), _addr(v_cache), int(bool(fp8)), descale_k,
                               descale_v, _addr(block_table), max_pages, _addr(query_start), _addr(seq_lens), _addr(o),
                               _addr(lse), T, R, Hq, Hkv, d, num_pages, page_size, max_new, scale, int(bool(causal)),
                               _addr(workspace), workspace_bytes, _stream(stream))


def fa_fwd_paged_window(q, q_stride: int, k_cache, v_cache, fp8: bool, descale_k: float, descale_v: float, block_table,
                        max_pages: int, query_start, seq_lens, o, lse, T: int, R: int, Hq: int, Hkv: int, d: int,
                        num_pages: int, page_size: int, max_new: int, scale: float, window: int, sinks: int, workspace,
                        workspace_bytes: int, stream=None) -> int:
    return load().fa_fwd_paged_window(_addr(q), q_stride, _addr(k_cache), _addr(v_cache), int(bool(fp8)), descale_k,
                                      descale_v, _addr(block_table), max_pages, _addr(query_start), _addr(seq_lens),
                                      _addr(o), _addr(lse), T, R, Hq, Hkv, d, num_pages, page_size, max_new, scale, window,
                                      sinks, _addr(workspace), workspace_bytes, _stream(stream))


_torch_module = None


def _paged():
    """The module that checks torch tensors and makes the calls (built and loaded on first use)."""
    global _torch_module
    if _torch_module is None:
        import importlib.machinery
        import importlib.util

        lib = load()
        with _lock:
            path = _build.build_torch_module()
        loader = importlib.machinery.ExtensionFileLoader("_fa_torch", path)
        module = importlib.util.module_from_spec(importlib.util.spec_from_file_location("_fa_torch", path, loader=loader))
        loader.exec_module(module)
        module.bind(*(ctypes.cast(f, ctypes.c_void_p).value for f in (
            lib.fa_paged_plan, lib.fa_paged_store, lib.fa_fwd_paged_workspace_bytes, lib.fa_fwd_paged, lib.fa_rope_fwd,
            lib.fa_rope_bwd_workspace_bytes, lib.fa_rope_bwd, lib.fa_paged_positions, lib.fa_paged_rope_store,
            lib.fa_fwd_paged_window, lib.fa_fwd_window, lib.fa_bwd_window_workspace_bytes, lib.fa_bwd_window)))
        _torch_module = module
    return _torch_module


def _on(stream, x):
    """The context of a call on ``stream`` (a torch.cuda.Stream or a handle) of the device of tensor ``x``: the tensors it
    allocates are that stream's. Handle 0 is the default stream (an ExternalStream of 0 would be a new stream)."""
    import torch

    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream, device=x.device) if stream else torch.cuda.default_stream(x.device)
    elif stream.device != x.device:
        raise ValueError(f"the stream must belong to {x.device}")
    return torch.cuda.stream(stream)


def paged_plan(ctx_lens, new_lens, block_table, free_pages, page_size: int, num_tokens: int, free_head=None, out=None,
               stream=None):
    """Plan a step of R requests: pages for their new tokens out of ``free_pages`` (from entry ``free_head`` on, an
    int32 [1] tensor) into ``block_table`` [R, max_pages] (in place), and where each of the ``num_tokens`` packed
    rows goes. All tensors int32 on the GPU. Returns (query_start [R + 1], seq_lens [R], slots [num_tokens],
    pages_taken [1]); ``out``: the four tensors to write them into, none of them an input's memory."""
    if stream is not None:
        with _on(stream, ctx_lens):
            return paged_plan(ctx_lens, new_lens, block_table, free_pages, page_size, num_tokens, free_head, out)
    r = (_torch_module or _paged()).plan(ctx_lens, new_lens, block_table, free_pages, page_size, num_tokens, free_head,
                                         None if out is None else tuple(out))
    if type(r) is int:
        raise FAError(r, "fa_paged_plan")
    return r


def paged_store(k, v, slots, k_cache, v_cache, descale_k: float = 1.0, descale_v: float = 1.0, stream=None) -> None:
    """Store the new tokens' k, v ([T, Hkv, d] bf16, slices of a projection's output allowed) into the caches
    [num_pages, Hkv, page_size, d] (bf16, or E4M3 codes of value / descale) at ``slots`` [T] (int32; negative:
    nowhere)."""
    if stream is not None:
        with _on(stream, k_cache):
            return paged_store(k, v, slots, k_cache, v_cache, descale_k, descale_v)
    r = (_torch_module or _paged()).store(k, v, slots, k_cache, v_cache, descale_k, descale_v)
    if r is not None:
        raise FAError(r, "fa_paged_store")


def forward_paged(q, k_cache, v_cache, block_table, query_start, seq_lens, max_new: int | None = None,
                  causal: bool = True, scale: float | None = None, descale_k: float = 1.0, descale_v: float = 1.0,
                  out=None, lse=None, workspace=None, stream=None, window: int | None = None, sinks: int = 0):
    """Attention of the packed new tokens q [T, Hq, d] (bf16) over the paged caches, which hold their keys and values
    already (paged_store): request r has rows query_start[r] .. query_start[r + 1] - 1, seq_lens[r] keys and the pages
    of block_table[r]. ``max_new``: the most new tokens a request has, if known. Only speed depends on it, but much: without
    it every request may have all T, so a batch of single tokens should say 1. The table's width stands for the longest
    request there may be: one much wider than the step's lengths costs a second launch or two. ``out`` and ``lse`` are
    written in place if given, rows of no request left as they are (zeros in the ones allocated here). ``window`` (causal
    calls): a token sees only the last ``window`` keys up to its own, and the first ``sinks`` of its request; pages of which
    no token sees a key are not read, and their table entries not followed. No gradients: a
    cache is not trained through. Returns (o [T, Hq, d], lse [T, Hq])."""
    if stream is not None:
        with _on(stream, k_cache):
            return forward_paged(q, k_cache, v_cache, block_table, query_start, seq_lens, max_new, causal, scale,
                                 descale_k, descale_v, out, lse, workspace, None, window, sinks)
    r = (_torch_module or _paged()).forward(q, k_cache, v_cache, block_table, query_start, seq_lens, max_new, causal,
                                            scale, descale_k, descale_v, out, lse, workspace, window, sinks)
    if type(r) is int:
        raise FAError(r, "fa_fwd_paged" if window is None else "fa_fwd_paged_window")
    return r


def paged_positions(query_start, seq_lens, num_tokens: int, out=None, stream=None):
    """Positions [num_tokens] (int32) of a step's packed tokens from paged_plan's query_start and seq_lens: new token i of
    the n of request r stands at seq_lens[r] - n + i; rows of no request get -1. Once per step, for all layers. ``out``:
    the tensor to write them into."""
    if stream is not None:
        with _on(stream, seq_lens):
            return paged_positions(query_start, seq_lens, num_tokens, out)
    r = (_torch_module or _paged()).positions(query_start, seq_lens, num_tokens, out)
    if type(r) is int:
        raise FAError(r, "fa_paged_positions")
    return r


def paged_rope_store(q, k, v, slots, positions, freqs, k_cache, v_cache, interleaved: bool = False, factor: float = 1.0,
                     q_weight=None, k_weight=None, eps: float = 1e-6, descale_k: float = 1.0, descale_v: float = 1.0, out=None,
                     stream=None):
    """A serving step's tokens into a layer, in one launch: q [T, Hq, d] normed (with weights) and rotated as in
    forward_rope, keys the same and values as they are into the paged caches, as paged_store does. ``positions`` [T] int32
    (paged_positions). Rows whose slot is negative are left out: nothing of them is stored, and their rows of the result
    stay as they are (zeros where it is allocated here). ``out``: where q goes, q itself allowed. Returns the rotated q."""
    if stream is not None:
        with _on(stream, k_cache):
            return paged_rope_store(q, k, v, slots, positions, freqs, k_cache, v_cache, interleaved, factor, q_weight, k_weight,
                                    eps, descale_k, descale_v, out)
    r = (_torch_module or _paged()).rope_store(q, k, v, slots, positions, freqs, k_cache, v_cache, interleaved, factor,
                                               q_weight, k_weight, eps, descale_k, descale_v, out)
    if type(r) is int:
        raise FAError(r, "fa_paged_rope_store")
    return r


# ---------------------------------------------------------------- rotation by position
def _heads(x, stride_b=None, stride_h=None, stride_n=None):
    """fa_heads of a torch tensor [B, H, N, d], or of an address with its strides; NULL for None."""
    if x is None:
        return None
    if isinstance(x, Heads):
        return ctypes.byref(x)
    if isinstance(x, int):
        return ctypes.byref(Heads(x, stride_b, stride_h, stride_n))
    return ctypes.byref(Heads(int(x.data_ptr()), x.stride(0), x.stride(1), x.stride(2)))


def fa_rope_fwd(q, k, q_out, k_out, q_weight, k_weight, weights_fp32: bool, eps: float, freqs, rotary: int, interleaved: bool,
                factor: float, positions, positions_stride: int, B: int, Hq: int, Hk: int, N: int, d: int, stream=None) -> int:
    """q, k, q_out, k_out: torch tensors [B, H, N, d] at any strides, or Heads."""
    return load().fa_rope_fwd(_heads(q), _heads(k), _heads(q_out), _heads(k_out), _addr(q_weight), _addr(k_weight),
                              int(bool(weights_fp32)), eps, _addr(freqs), rotary, int(bool(interleaved)), factor,
                              _addr(positions), positions_stride, B, Hq, Hk, N, d, _stream(stream))


def fa_rope_bwd_workspace_bytes(Hq: int, Hk: int, d: int) -> int:
    return int(load().fa_rope_bwd_workspace_bytes(Hq, Hk, d))


def fa_rope_bwd(dq_out, dk_out, q, k, dq, dk, q_weight, k_weight, weights_fp32: bool, eps: float, dq_weight, dk_weight, freqs,
                rotary: int, interleaved: bool, factor: float, positions, positions_stride: int, B: int, Hq: int, Hk: int,
                N: int, d: int, workspace, workspace_bytes: int, stream=None) -> int:
    """dq_out, dk_out, q, k, dq, dk: torch tensors [B, H, N, d] at any strides, or Heads."""
    return load().fa_rope_bwd(_heads(dq_out), _heads(dk_out), _heads(q), _heads(k), _heads(dq), _heads(dk), _addr(q_weight),
                              _addr(k_weight), int(bool(weights_fp32)), eps, _addr(dq_weight), _addr(dk_weight), _addr(freqs),
                              rotary, int(bool(interleaved)), factor, _addr(positions), positions_stride, B, Hq, Hk, N, d,
                              _addr(workspace), workspace_bytes, _stream(stream))


def fa_paged_positions(query_start, seq_lens, R: int, positions, T: int, stream=None) -> int:
    return load().fa_paged_positions(_addr(query_start), _addr(seq_lens), R, _addr(positions), T, _stream(stream))


def fa_paged_rope_store(q, k, v, q_stride: int, k_stride: int, v_stride: int, slots, positions, freqs, rotary: int,
                        interleaved: bool, factor: float, q_weight, k_weight, weights_fp32: bool, eps: float, q_out,
                        q_out_stride: int, T: int, Hq: int, Hkv: int, d: int, k_cache, v_cache, num_pages: int, page_size: int,
                        fp8: bool, descale_k: float, descale_v: float, stream=None) -> int:
    return load().fa_paged_rope_store(_addr(q), _addr(k), _addr(v), q_stride, k_stride, v_stride, _addr(slots),
                                      _addr(positions), _addr(freqs), rotary, int(bool(interleaved)), factor, _addr(q_weight),
                                      _addr(k_weight), int(bool(weights_fp32)), eps, _addr(q_out), q_out_stride, T, Hq, Hkv, d,
                                      _addr(k_cache), _addr(v_cache), num_pages, page_size, int(bool(fp8)), descale_k,
                                      descale_v, _stream(stream))


def rope_frequencies(rotary: int, base: float = 10000.0, linear: float = 1.0, base_stretch: float = 1.0, ramp=None,
                     device="cuda"):
    """Angles a position (radians, fp64 [rotary / 2]) of a head's pairs, freqs[i] = base^(-2 i / rotary), and for texts longer
    than a model was trained on one of
      linear: all of them divided by this (positions squeezed into the old range);
      base_stretch: the base times base_stretch^(rotary / (rotary - 2)): the lowest frequency is divided by it, the highest
          stays;
      ramp (stretch, length, slow, fast): a pair that turns at least ``fast`` times within ``length`` positions stays, one that
          turns at most ``slow`` times is divided by ``stretch``, in between a straight mixture by the turns."""
    import torch

    if rotary < 2 or rotary % 2 or not (base > 0 and linear > 0 and base_stretch > 0):
        raise ValueError("rotary must be even, base, linear and base_stretch positive")
    if base_stretch != 1.0:
        if rotary == 2:
            raise ValueError("base_stretch needs more than one pair")
        base = base * base_stretch ** (rotary / (rotary - 2))
    f = base ** (-torch.arange(0, rotary, 2, dtype=torch.float64) / rotary) / linear
    if ramp is not None:
        stretch, length, slow, fast = ramp
        if not (stretch > 0 and length > 0 and fast > slow):
            raise ValueError("ramp is (stretch, length, slow, fast), stretch and length positive, fast above slow")
        keep = ((f * (length / (2 * math.pi)) - slow) / (fast - slow)).clamp(0.0, 1.0)
        f = f * keep + f / stretch * (1 - keep)
    return f.to(device)


def forward_rope(q, k, freqs, positions=None, interleaved: bool = False, factor: float = 1.0, q_weight=None, k_weight=None,
                 eps: float = 1e-6, out=None, stream=None):
    """Rotate q [B, Hq, N, d] and k [B, Hk, N, d] (bf16, any strides with contiguous rows: slices of a projection's output are
    read as they are; k may be None) by their positions (int32 [N] or [B, N]; None: 0 .. N - 1): the pairs of the first
    2 * len(freqs) elements of each head turn by position * freqs (fp64, rope_frequencies), pairs being neighbours
    (``interleaved``) or halves apart, times ``factor``. With q_weight, k_weight ([d], bf16 or fp32) each head is first normed,
    x * weight / sqrt(mean(x^2) + eps), in the same pass. Returns (q_out, k_out), contiguous as attention takes them, or the
    tensors of ``out`` (which may be q and k themselves)."""
    if stream is not None:
        with _on(stream, q):
            return forward_rope(q, k, freqs, positions, interleaved, factor, q_weight, k_weight, eps, out)
    r = (_torch_module or _paged()).rope(q, k, freqs, positions, interleaved, factor, q_weight, k_weight, eps,
                                         None if out is None else tuple(out))
    if type(r) is int:
        raise FAError(r, "fa_rope_fwd")
    return r


def backward_rope(dq_out, dk_out, freqs, positions=None, interleaved: bool = False, factor: float = 1.0, q=None, k=None,
                  q_weight=None, k_weight=None, eps: float = 1e-6, stream=None):
    """Gradients of forward_rope given those of its results (any strides with contiguous rows): (dq, dk, dq_weight, dk_weight).
    With norms it needs the forward's q and k; without them the last two are None. dq and dk are [B, H, N, d] laid out
    token by token, the weights' gradients fp32. Repeated calls give identical bits."""
    if stream is not None:
        with _on(stream, dq_out):
            return backward_rope(dq_out, dk_out, freqs, positions, interleaved, factor, q, k, q_weight, k_weight, eps)
    r = (_torch_module or _paged()).rope_backward(dq_out, dk_out, freqs, positions, interleaved, factor, q, k, q_weight,
                                                  k_weight, eps)
    if type(r) is int:
        raise FAError(r, "fa_rope_bwd")
    return r


def _rows_contiguous(x):
    """A gradient as the kernels read it: bf16, the elements of a row contiguous, rows 16-byte aligned."""
    import torch

    x = x.to(torch.bfloat16)
    ok = x.stride(-1) == 1 and all(s % 8 == 0 for s, n in zip(x.stride()[:-1], x.shape[:-1]) if n > 1) and x.data_ptr() % 16 == 0
    return x if ok else _gradient(x)


_rope_fn = None


def rope(q, k, freqs, positions=None, interleaved: bool = False, factor: float = 1.0, q_weight=None, k_weight=None,
         eps: float = 1e-6):
    """Differentiable forward_rope: a torch.autograd.Function over forward_rope and backward_rope, with gradients of q, k and
    the weights (gradients of those are refused). Returns (q_out, k_out); k may be None. (As with any function of torch's: before a backward pass is captured
    into a CUDA graph, results of eager calls on the same leaves have to be gone.)"""
    global _rope_fn
    if _rope_fn is None:
        import torch

        class _Rope(torch.autograd.Function):
            @staticmethod
            def forward(ctx, q, k, q_weight, k_weight, freqs, positions, interleaved, factor, eps):
                q_out, k_out = forward_rope(q, k, freqs, positions, interleaved, factor, q_weight, k_weight, eps)
                keep = q_weight is not None  # without norms the gradient does not look at the inputs
                ctx.save_for_backward(q if keep else None, k if keep else None, q_weight, k_weight, freqs, positions)
                ctx.args = (interleaved, factor, eps, k is not None)
                return q_out, k_out

            @staticmethod
            @_once
            def backward(ctx, dq_out, dk_out):
                q, k, q_weight, k_weight, freqs, positions = ctx.saved_tensors
                interleaved, factor, eps, has_k = ctx.args
                dq, dk, dwq, dwk = backward_rope(_rows_contiguous(dq_out), _rows_contiguous(dk_out) if has_k else None, freqs,
                                                 positions, interleaved, factor, q, k, q_weight, k_weight, eps)
                dwq, dwk = (None if g is None else g.to(w.dtype) for g, w in ((dwq, q_weight), (dwk, k_weight)))
                return dq, dk, dwq, dwk, None, None, None, None, None

        _rope_fn = _Rope
    return _rope_fn.apply(q, k, q_weight, k_weight, freqs, positions, bool(interleaved), float(factor), float(eps))


# ---------------------------------------------------------------- attention in a sliding window
def fa_fwd_window(q, k, v, o, lse, B: int, Hq: int, Hkv: int, Nq: int, Nk: int, d: int, scale: float, window: int, sinks: int,
                  seqlens_q=None, seqlens_k=None, stream=None) -> int:
    return load().fa_fwd_window(_addr(q), _addr(k), _addr(v), _addr(o), _addr(lse), B, Hq, Hkv, Nq, Nk, d, scale, window, sinks,
                                _addr(seqlens_q), _addr(seqlens_k), _stream(stream))


def fa_bwd_window_workspace_bytes(B: int, Hq: int, Hkv: int, Nq: int, Nk: int, d: int, window: int, sinks: int) -> int:
    return int(load().fa_bwd_window_workspace_bytes(B, Hq, Hkv, Nq, Nk, d, window, sinks))


def fa_bwd_window(q, k, v, o, lse, dO, dq, dk, dv, B: int, Hq: int, Hkv: int, Nq: int, Nk: int, d: int, scale: float,
                  window: int, sinks: int, seqlens_q, seqlens_k, workspace, workspace_bytes: int, stream=None) -> int:
    return load().fa_bwd_window(_addr(q), _addr(k), _addr(v), _addr(o), _addr(lse), _addr(dO), _addr(dq), _addr(dk), _addr(dv),
                                B, Hq, Hkv, Nq, Nk, d, scale, window, sinks, _addr(seqlens_q), _addr(seqlens_k),
                                _addr(workspace), workspace_bytes, _stream(stream))


def forward_window(q, k, v, window: int, sinks: int = 0, scale: float | None = None, seqlens_q=None, seqlens_k=None,
                   stream=None):
    """Causal attention of q [B, Hq, Nq, d] over k, v [B, Hkv, Nk, d] (bf16; Hq a multiple of Hkv; the queries are the last Nq
    positions) in which a row sees the last ``window`` keys up to its own position, and the first ``sinks`` of the sequence:
    allocate o (bf16) and lse (fp32) with torch and run fa_fwd_window. ``seqlens_q`` / ``seqlens_k``: padding lengths, as in
    forward_kv. On the device of q, on its current stream or ``stream``. Returns (o, lse)."""
    if stream is not None:
        with _on(stream, q):
            return forward_window(q, k, v, window, sinks, scale, seqlens_q, seqlens_k)
    r = (_torch_module or _paged()).window(q, k, v, window, sinks, scale, seqlens_q, seqlens_k)
    if type(r) is int:
        raise FAError(r, "fa_fwd_window")
    return r


def backward_window(q, k, v, o, lse, dO, window: int, sinks: int = 0, scale: float | None = None, seqlens_q=None,
                    seqlens_k=None, workspace=None, stream=None):
    """Gradients of forward_window: allocate dq, dk, dv (and the workspace if none is given) and run fa_bwd_window."""
    if stream is not None:
        with _on(stream, q):
            return backward_window(q, k, v, o, lse, dO, window, sinks, scale, seqlens_q, seqlens_k, workspace)
    r = (_torch_module or _paged()).window_backward(q, k, v, o, lse, dO, window, sinks, scale, seqlens_q, seqlens_k, workspace)
    if type(r) is int:
        raise FAError(r, "fa_bwd_window")
    return r


_window_fn = None


def attention_window(q, k, v, window: int, sinks: int = 0, scale: float | None = None, seqlens_q=None, seqlens_k=None):
    """Differentiable forward_window: a torch.autograd.Function over forward_window and backward_window (gradients of the
    gradients are refused). Returns o. (Captured into a CUDA graph as rope is.)"""
    global _window_fn
    if _window_fn is None:
        import torch

        class _Window(torch.autograd.Function):
            @staticmethod
            def forward(ctx, q, k, v, seqlens_q, seqlens_k, args):
                o, lse = forward_window(q, k, v, *args, seqlens_q, seqlens_k)
                ctx.save_for_backward(q, k, v, o, lse, seqlens_q, seqlens_k)
                ctx.args = args
                return o

            @staticmethod
            @_once
            def backward(ctx, dO):
                q, k, v, o, lse, seqlens_q, seqlens_k = ctx.saved_tensors
                return (*backward_window(q, k, v, o, lse, _gradient(dO), *ctx.args, seqlens_q, seqlens_k), None, None, None)

        _window_fn = _Window
    scale = 1.0 / math.sqrt(int(q.shape[-1])) if scale is None else scale
    return _window_fn.apply(q, k, v, seqlens_q, seqlens_k, (int(window), int(sinks), float(scale)))

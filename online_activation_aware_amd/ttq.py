"""Thin ctypes binding of libttq (include/ttq.h).

Argument marshalling only: every step of the path runs in the HIP kernels of
libttq.so.  Tensors must be device (HIP) tensors; PyTorch supplies memory and
the current stream.  There is no CPU fallback: if the library is missing or a
call fails, an exception is raised.
"""
from __future__ import annotations

import ctypes
import functools
import inspect
import os
from typing import Optional

import torch

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libttq.so")

TTQ_OK, TTQ_ERR_INVALID, TTQ_ERR_UNSUPPORTED, TTQ_ERR_DEVICE = 0, 1, 2, 3
TTQ_F32, TTQ_BF16 = 0, 1

EXPORTS = ("ttq_stats", "ttq_stats_p", "ttq_awq_scales", "ttq_quantize_groups", "ttq_qgemm", "ttq_qgemm_batched",
           "ttq_lowrank_add", "ttq_lowrank_factors", "ttq_lowrank_factors_workspace_bytes",
           "ttq_workspace_bytes", "ttq_linear", "ttq_linear_shared", "ttq_linear_shared_workspace_bytes",
           "ttq_linear_noalloc", "ttq_moe_route", "ttq_moe", "ttq_moe_workspace_bytes", "ttq_adapters_add",
           "ttq_adapters_workspace_bytes", "ttq_qgemm_adapters", "ttq_qgemm_adapters_workspace_bytes",
           "ttq_quantize_rows", "ttq_gemm_i8", "ttq_gemm_i8_workspace_bytes", "ttq_qgemm_i8",
           "ttq_qgemm_i8_workspace_bytes", "ttq_moe_sort", "ttq_moe_sort_workspace_bytes", "ttq_moe_gather",
           "ttq_moe_combine", "ttq_moe_combine_grad", "ttq_moe_i8", "ttq_moe_i8_workspace_bytes",
           "ttq_status_str", "ttq_last_error")


class TTQError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(message)
        self.status = status


class LinearArgs(ctypes.Structure):
    _fields_ = [
        ("X", ctypes.c_void_p), ("xt", ctypes.c_int), ("T", ctypes.c_int64),
        ("K", ctypes.c_int64), ("ldx", ctypes.c_int64),
        ("W", ctypes.c_void_p), ("wt", ctypes.c_int), ("M", ctypes.c_int64),
        ("ldw", ctypes.c_int64),
        ("alpha", ctypes.c_float), ("lambda_rel", ctypes.c_float), ("p", ctypes.c_float),
        ("bits", ctypes.c_int), ("group", ctypes.c_int),
        ("B", ctypes.c_void_p), ("A", ctypes.c_void_p), ("rank", ctypes.c_int),
        ("Y", ctypes.c_void_p), ("yt", ctypes.c_int), ("ldy", ctypes.c_int64),
        ("ssq", ctypes.c_void_p), ("s", ctypes.c_void_p), ("codes", ctypes.c_void_p),
        ("scale_f16", ctypes.c_void_p), ("zero_f16", ctypes.c_void_p),
        ("stage_events", ctypes.c_void_p),
    ]


class ExpertState(ctypes.Structure):
    _fields_ = [("s", ctypes.c_void_p), ("s_stride", ctypes.c_int64), ("codes", ctypes.c_void_p),
                ("scale_f16", ctypes.c_void_p), ("zero_f16", ctypes.c_void_p)]


class MoeArgs(ctypes.Structure):
    _fields_ = [
        ("X", ctypes.c_void_p), ("xt", ctypes.c_int), ("T", ctypes.c_int64), ("K", ctypes.c_int64),
        ("ldx", ctypes.c_int64), ("ids", ctypes.c_void_p), ("w", ctypes.c_void_p), ("topk", ctypes.c_int64),
        ("E", ctypes.c_int64), ("I", ctypes.c_int64), ("M", ctypes.c_int64),
        ("gate_up", ExpertState), ("down", ExpertState),
        ("bits", ctypes.c_int), ("group", ctypes.c_int), ("act", ctypes.c_int),
        ("Y", ctypes.c_void_p), ("yt", ctypes.c_int), ("ldy", ctypes.c_int64),
    ]


class AdaptersArgs(ctypes.Structure):
    _fields_ = [("A", ctypes.c_void_p), ("B", ctypes.c_void_p), ("dt", ctypes.c_int), ("n", ctypes.c_int64),
                ("rank", ctypes.c_int), ("ranks", ctypes.c_void_p), ("scale", ctypes.c_void_p),
                ("ids", ctypes.c_void_p)]


class ExpertI8(ctypes.Structure):
    _fields_ = [("s", ctypes.c_void_p), ("s_stride", ctypes.c_int64), ("codes", ctypes.c_void_p),
                ("scale", ctypes.c_void_p)]


class MoeI8Args(ctypes.Structure):
    _fields_ = [
        ("X", ctypes.c_void_p), ("xt", ctypes.c_int), ("T", ctypes.c_int64), ("K", ctypes.c_int64),
        ("ldx", ctypes.c_int64), ("ids", ctypes.c_void_p), ("w", ctypes.c_void_p), ("topk", ctypes.c_int64),
        ("E", ctypes.c_int64), ("I", ctypes.c_int64), ("M", ctypes.c_int64),
        ("gate_up", ExpertI8), ("down", ExpertI8), ("act", ctypes.c_int),
        ("Y", ctypes.c_void_p), ("yt", ctypes.c_int), ("ldy", ctypes.c_int64),
    ]


_lib_handle = None


def lib() -> ctypes.CDLL:
    """Load libttq.so (once) and declare the C signatures."""
    global _lib_handle
    if _lib_handle is not None:
        return _lib_handle
    if not os.path.exists(_LIB_PATH):
        raise RuntimeError(f"{_LIB_PATH} is not built: run `python -m online_activation_aware_amd.build`")
    L = ctypes.CDLL(_LIB_PATH)
    vp, i32, i64, f32, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t
    sig = {
        "ttq_stats": [vp, i32, i64, i64, i64, vp, i32, vp, sz, vp],
        "ttq_stats_p": [vp, i32, i64, i64, i64, f32, vp, i32, vp, sz, vp],
        "ttq_awq_scales": [vp, i64, i64, f32, f32, f32, vp, vp],
        "ttq_quantize_groups": [vp, i32, i64, i64, i64, vp, i32, i32, vp, vp, i32, vp, vp, vp, vp],
        "ttq_qgemm": [vp, i32, i64, i64, i64, vp, vp, vp, vp, i64, i32, i32, vp, i32, i64, vp, sz, vp],
        "ttq_lowrank_add": [vp, i32, i64, i64, i64, vp, vp, i64, i32, vp, i32, i64, vp, sz, vp],
        "ttq_qgemm_batched": [vp, i32, i64, i64, i64, i64, i64, vp, i64, vp, i64, vp, vp, i64, i64, i32, i32, vp,
                              i32, i64, i64, vp],
        "ttq_workspace_bytes": [i64, i64, i64, i32, i32, i32],
        "ttq_lowrank_factors": [vp, i32, i64, i64, i64, vp, vp, i32, i32, i32, vp, vp, vp, sz, vp],
        "ttq_lowrank_factors_workspace_bytes": [i64, i64, i32],
        "ttq_linear": [ctypes.POINTER(LinearArgs), vp, sz, vp],
        "ttq_linear_noalloc": [ctypes.POINTER(LinearArgs), vp],
        "ttq_linear_shared": [ctypes.POINTER(LinearArgs), i32, vp, sz, vp],
        "ttq_linear_shared_workspace_bytes": [ctypes.POINTER(LinearArgs), i32],
        "ttq_moe_route": [vp, i32, i64, i64, i64, i32, i32, i32, vp, vp, vp],
        "ttq_moe": [ctypes.POINTER(MoeArgs), vp, sz, vp],
        "ttq_moe_workspace_bytes": [i64, i64, i64, i64, i64, i64, i32, i32],
        "ttq_adapters_add": [vp, i32, i64, i64, i64, ctypes.POINTER(AdaptersArgs), i64, vp, i64, vp, i32, i64, vp, sz,
                             vp],
        "ttq_adapters_workspace_bytes": [i64, i64, i64, i32],
        "ttq_qgemm_adapters": [vp, i32, i64, i64, i64, vp, vp, vp, vp, i64, i32, i32, ctypes.POINTER(AdaptersArgs),
                               vp, i32, i64, vp, sz, vp],
        "ttq_qgemm_adapters_workspace_bytes": [i64, i64, i64, i32, i32, i32],
        "ttq_quantize_rows": [vp, i32, i64, i64, i64, vp, i32, vp, i64, vp, vp],
        "ttq_gemm_i8": [vp, vp, i64, i64, i64, vp, vp, i64, i64, vp, i32, i64, vp, sz, vp],
        "ttq_gemm_i8_workspace_bytes": [i64, i64, i64],
        "ttq_qgemm_i8": [vp, i32, i64, i64, i64, vp, vp, vp, i64, i64, vp, i32, i64, vp, sz, vp],
        "ttq_qgemm_i8_workspace_bytes": [i64, i64, i64],
        "ttq_moe_sort": [vp, i64, i64, i64, vp, vp, vp, vp, sz, vp],
        "ttq_moe_sort_workspace_bytes": [i64, i64, i64],
        "ttq_moe_gather": [vp, i32, i64, i64, i64, vp, i64, vp, i64, i64, vp],
        "ttq_moe_combine": [vp, i32, i64, i64, vp, vp, i64, i64, i64, vp, i32, i64, vp],
        "ttq_moe_combine_grad": [vp, i32, i64, i64, i64, vp, i32, i64, i64, vp, vp, i64, vp, i64, vp, vp],
        "ttq_moe_i8": [ctypes.POINTER(MoeI8Args), vp, sz, vp],
        "ttq_moe_i8_workspace_bytes": [i64, i64, i64, i64, i64, i64],
        "ttq_status_str": [i32],
        "ttq_last_error": [],
    }
    for name, argtypes in sig.items():
        fn = getattr(L, name)
        fn.argtypes = argtypes
        fn.restype = ctypes.c_int
    L.ttq_workspace_bytes.restype = ctypes.c_size_t
    L.ttq_lowrank_factors_workspace_bytes.restype = ctypes.c_size_t
    L.ttq_linear_shared_workspace_bytes.restype = ctypes.c_size_t
    for name in ("ttq_moe_workspace_bytes", "ttq_adapters_workspace_bytes", "ttq_qgemm_adapters_workspace_bytes",
                 "ttq_gemm_i8_workspace_bytes", "ttq_qgemm_i8_workspace_bytes", "ttq_moe_sort_workspace_bytes",
                 "ttq_moe_i8_workspace_bytes"):
        getattr(L, name).restype = ctypes.c_size_t
    L.ttq_status_str.restype = ctypes.c_char_p
    L.ttq_last_error.restype = ctypes.c_char_p
    _lib_handle = L
    return L


# ------------------------------------------------------------------ helpers

def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return TTQ_F32
    if t.dtype == torch.bfloat16:
        return TTQ_BF16
    raise TypeError(f"unsupported dtype {t.dtype} (float32 or bfloat16)")


def _dev(t: Optional[torch.Tensor], name: str):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a device tensor")
    return t.data_ptr()


def _ld(t: torch.Tensor, name: str) -> int:
    if t.dim() != 2 or t.stride(1) != 1:
        raise ValueError(f"{name} must be 2-D with unit stride in its last dimension")
    return t.stride(0)


def _stream(stream) -> Optional[int]:
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else stream


def _torch_stream(stream) -> torch.cuda.Stream:
    """The launch stream as a torch stream (a raw hipStream_t handle is
    wrapped as an external stream)."""
    if stream is None:
        return torch.cuda.current_stream()
    if isinstance(stream, torch.cuda.Stream):
        return stream
    return torch.cuda.ExternalStream(int(stream))


def _on_launch_stream(fn):
    """Run a call with its launch stream as torch's current stream, so that
    every tensor the binding allocates for it (outputs, default workspaces)
    belongs to the stream the kernels run on: the caching allocator then
    cannot hand such memory to other work before those kernels are done."""
    sig = inspect.signature(fn)

    @functools.wraps(fn)
    def call(*args, **kwargs):
        bound = sig.bind(*args, **kwargs)
        ts = _torch_stream(bound.arguments.get("stream"))
        bound.arguments["stream"] = ts
        with torch.cuda.stream(ts):
            return fn(*bound.args, **bound.kwargs)
    return call


def _check(status: int) -> None:
    if status != TTQ_OK:
        L = lib()
        raise TTQError(status, f"{L.ttq_status_str(status).decode()}: {L.ttq_last_error().decode()}")


def _ws(ws: Optional[torch.Tensor], device) -> tuple:
    if ws is None:
        return None, 0
    if ws.dtype != torch.uint8:
        raise TypeError("workspace must be a uint8 tensor")
    return _dev(ws, "ws"), ws.numel()


# ------------------------------------------------------------------ calls

def ttq_workspace_bytes(T: int, K: int, M: int, bits: int, group: int, rank: int = 0) -> int:
    return int(lib().ttq_workspace_bytes(T, K, M, bits, group, rank))


def workspace(T: int, K: int, M: int, bits: int, group: int, rank: int = 0, device="cuda") -> torch.Tensor:
    """Allocate a workspace tensor of ttq_workspace_bytes() bytes."""
    n = ttq_workspace_bytes(T, K, M, bits, group, rank)
    if n == 0:
        raise ValueError("no call accepts these sizes")
    return torch.empty(n, dtype=torch.uint8, device=device)


@_on_launch_stream
def ttq_stats(X: torch.Tensor, ssq: torch.Tensor, accumulate: bool = False,
              ws: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    if ssq.dtype != torch.float64:
        raise TypeError("ssq must be float64")
    T, K = X.shape
    wp, wn = _ws(ws, X.device)
    _check(lib().ttq_stats(_dev(X, "X"), _dtype_code(X), T, K, _ld(X, "X"), _dev(ssq, "ssq"),
                           int(bool(accumulate)), wp, wn, _stream(stream)))
    return ssq


@_on_launch_stream
def ttq_stats_p(X: torch.Tensor, p: float, msum: torch.Tensor, accumulate: bool = False,
                ws: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    if msum.dtype != torch.float64:
        raise TypeError("msum must be float64")
    T, K = X.shape
    wp, wn = _ws(ws, X.device)
    _check(lib().ttq_stats_p(_dev(X, "X"), _dtype_code(X), T, K, _ld(X, "X"), p, _dev(msum, "msum"),
                             int(bool(accumulate)), wp, wn, _stream(stream)))
    return msum


@_on_launch_stream
def ttq_awq_scales(ssq: torch.Tensor, n_tokens: int, alpha: float, lambda_rel: float,
                   p: float = 2.0, s: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    K = ssq.numel()
    if s is None:
        s = torch.empty(K, dtype=torch.float32, device=ssq.device)
    _check(lib().ttq_awq_scales(_dev(ssq, "ssq"), n_tokens, K, alpha, lambda_rel, p, _dev(s, "s"),
                                _stream(stream)))
    return s


@_on_launch_stream
def ttq_quantize_groups(W: torch.Tensor, s: Optional[torch.Tensor], bits: int, group: int,
                        B: Optional[torch.Tensor] = None, A: Optional[torch.Tensor] = None,
                        codes: Optional[torch.Tensor] = None, scale_f16: Optional[torch.Tensor] = None,
                        zero_f16: Optional[torch.Tensor] = None, stream=None):
    M, K = W.shape
    rank = 0 if B is None else B.shape[1]
    dev = W.device
    if codes is None:
        codes = torch.empty((M, K * bits // 32), dtype=torch.int32, device=dev)
    if scale_f16 is None:
        scale_f16 = torch.empty((M, K // group), dtype=torch.float16, device=dev)
    if zero_f16 is None:
        zero_f16 = torch.empty((M, K // group), dtype=torch.float16, device=dev)
    _check(lib().ttq_quantize_groups(_dev(W, "W"), _dtype_code(W), M, K, _ld(W, "W"), _dev(s, "s"),
                                     bits, group, _dev(B, "B"), _dev(A, "A"), rank, _dev(codes, "codes"),
                                     _dev(scale_f16, "scale_f16"), _dev(zero_f16, "zero_f16"),
                                     _stream(stream)))
    return codes, scale_f16, zero_f16


@_on_launch_stream
def ttq_qgemm(X: torch.Tensor, s: torch.Tensor, codes: torch.Tensor, scale_f16: torch.Tensor,
              zero_f16: torch.Tensor, M: int, bits: int, group: int, Y: Optional[torch.Tensor] = None,
              y_dtype=torch.float32, ws: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    T, K = X.shape
    if Y is None:
        Y = torch.empty((T, M), dtype=y_dtype, device=X.device)
    wp, wn = _ws(ws, X.device)
    _check(lib().ttq_qgemm(_dev(X, "X"), _dtype_code(X), T, K, _ld(X, "X"), _dev(s, "s"),
                           _dev(codes, "codes"), _dev(scale_f16, "scale_f16"), _dev(zero_f16, "zero_f16"),
                           M, bits, group, _dev(Y, "Y"), _dtype_code(Y), _ld(Y, "Y"), wp, wn,
                           _stream(stream)))
    return Y


@_on_launch_stream
def ttq_qgemm_batched(X: torch.Tensor, s: torch.Tensor, codes: torch.Tensor, scale_f16: torch.Tensor,
                      zero_f16: torch.Tensor, M: int, bits: int, group: int, Y: Optional[torch.Tensor] = None,
                      y_dtype=torch.float32, stream=None) -> torch.Tensor:
    """One decode step of P prompts: X [P][T][K], s [P][K], codes [P][M][.],
    scale_f16 / zero_f16 [P][M][K/group]; returns Y [P][T][M]."""
    P, T, K = X.shape
    if Y is None:
        Y = torch.empty((P, T, M), dtype=y_dtype, device=X.device)
    for name, t in (("s", s), ("codes", codes), ("scale_f16", scale_f16), ("zero_f16", zero_f16)):
        if t.shape[0] != P or not t.is_contiguous():
            raise ValueError(f"{name}: expected a contiguous [P][...] tensor")
    if X.stride(2) != 1 or Y.stride(2) != 1:
        raise ValueError("X and Y rows must be contiguous")
    if scale_f16.stride(0) != zero_f16.stride(0):
        raise ValueError("scale_f16 and zero_f16 must have the same prompt stride")
    _check(lib().ttq_qgemm_batched(_dev(X, "X"), _dtype_code(X), P, T, K, X.stride(1), X.stride(0),
                                   _dev(s, "s"), s.stride(0), _dev(codes, "codes"), codes.stride(0),
                                   _dev(scale_f16, "scale_f16"), _dev(zero_f16, "zero_f16"), scale_f16.stride(0),
                                   M, bits, group, _dev(Y, "Y"), _dtype_code(Y), Y.stride(1), Y.stride(0),
                                   _stream(stream)))
    return Y


@_on_launch_stream
def ttq_lowrank_add(X: torch.Tensor, A: torch.Tensor, B: torch.Tensor, Y: torch.Tensor,
                    ws: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    T, K = X.shape
    M, rank = B.shape
    wp, wn = _ws(ws, X.device)
    _check(lib().ttq_lowrank_add(_dev(X, "X"), _dtype_code(X), T, K, _ld(X, "X"), _dev(A, "A"),
                                 _dev(B, "B"), M, rank, _dev(Y, "Y"), _dtype_code(Y), _ld(Y, "Y"),
                                 wp, wn, _stream(stream)))
    return Y


@_on_launch_stream
def ttq_lowrank_factors(W: torch.Tensor, s: torch.Tensor, omega: torch.Tensor, rank: int, q: int,
                        B: Optional[torch.Tensor] = None, A: Optional[torch.Tensor] = None,
                        ws: Optional[torch.Tensor] = None, stream=None):
    """Per-prompt factors of W diag(s): returns (B [M][rank], A [rank][K])."""
    M, K = W.shape
    l = omega.shape[0]
    if omega.shape != (l, K) or omega.dtype != torch.float32:
        raise ValueError("omega must be float32 [l][K]")
    if B is None:
        B = torch.empty((M, rank), dtype=torch.float32, device=W.device)
    if A is None:
        A = torch.empty((rank, K), dtype=torch.float32, device=W.device)
    if ws is None:
        n = lib().ttq_lowrank_factors_workspace_bytes(M, K, l)
        if n == 0:
            raise ValueError("no factorization accepts these sizes")
        ws = torch.empty(n, dtype=torch.uint8, device=W.device)
    _check(lib().ttq_lowrank_factors(_dev(W, "W"), _dtype_code(W), M, K, _ld(W, "W"), _dev(s, "s"),
                                     _dev(omega, "omega"), l, q, rank, _dev(B, "B"), _dev(A, "A"),
                                     ws.data_ptr(), ws.numel() * ws.element_size(), _stream(stream)))
    return B, A


@_on_launch_stream
def ttq_linear(X: torch.Tensor, W: torch.Tensor, bits: int, group: int, alpha: float,
               lambda_rel: float, p: float = 2.0, B: Optional[torch.Tensor] = None,
               A: Optional[torch.Tensor] = None, Y: Optional[torch.Tensor] = None,
               y_dtype=torch.float32, ws: Optional[torch.Tensor] = None, state: Optional[dict] = None,
               stream=None, stage_events=None) -> torch.Tensor:
    """One call for the whole layer.  ``state`` may hold preallocated output
    tensors ``ssq``, ``s``, ``codes``, ``scale_f16``, ``zero_f16`` that receive
    the prompt's quantization state (for later decode-step ttq_qgemm calls).
    ``stage_events``: optional StageEvents, recorded at the stage boundaries."""
    T, K = X.shape
    M = W.shape[0]
    rank = 0 if B is None else B.shape[1]
    if Y is None:
        Y = torch.empty((T, M), dtype=y_dtype, device=X.device)
    if ws is None:
        ws = workspace(T, K, M, bits, group, rank, device=X.device)
    st = state or {}
    a = LinearArgs(
        X=_dev(X, "X"), xt=_dtype_code(X), T=T, K=K, ldx=_ld(X, "X"),
        W=_dev(W, "W"), wt=_dtype_code(W), M=M, ldw=_ld(W, "W"),
        alpha=alpha, lambda_rel=lambda_rel, p=p, bits=bits, group=group,
        B=_dev(B, "B"), A=_dev(A, "A"), rank=rank,
        Y=_dev(Y, "Y"), yt=_dtype_code(Y), ldy=_ld(Y, "Y"),
        ssq=_dev(st.get("ssq"), "ssq"), s=_dev(st.get("s"), "s"), codes=_dev(st.get("codes"), "codes"),
        scale_f16=_dev(st.get("scale_f16"), "scale_f16"), zero_f16=_dev(st.get("zero_f16"), "zero_f16"),
        stage_events=None if stage_events is None else ctypes.cast(stage_events.handles, ctypes.c_void_p),
    )
    wp, wn = _ws(ws, X.device)
    _check(lib().ttq_linear(ctypes.byref(a), wp, wn, _stream(stream)))
    return Y


@_on_launch_stream
def ttq_linear_noalloc(X: torch.Tensor, W: torch.Tensor, bits: int, group: int, alpha: float,
                       lambda_rel: float, Y: torch.Tensor, p: float = 2.0, B: Optional[torch.Tensor] = None,
                       A: Optional[torch.Tensor] = None, state: Optional[dict] = None,
                       stream=None) -> torch.Tensor:
    """ttq_linear with the library's own scratch array as the workspace (the
    call allocates nothing; Y and the optional state tensors come from the
    caller)."""
    T, K = X.shape
    M = W.shape[0]
    st = state or {}
    a = LinearArgs(
        X=_dev(X, "X"), xt=_dtype_code(X), T=T, K=K, ldx=_ld(X, "X"),
        W=_dev(W, "W"), wt=_dtype_code(W), M=M, ldw=_ld(W, "W"),
        alpha=alpha, lambda_rel=lambda_rel, p=p, bits=bits, group=group,
        B=_dev(B, "B"), A=_dev(A, "A"), rank=0 if B is None else B.shape[1],
        Y=_dev(Y, "Y"), yt=_dtype_code(Y), ldy=_ld(Y, "Y"),
        ssq=_dev(st.get("ssq"), "ssq"), s=_dev(st.get("s"), "s"), codes=_dev(st.get("codes"), "codes"),
        scale_f16=_dev(st.get("scale_f16"), "scale_f16"), zero_f16=_dev(st.get("zero_f16"), "zero_f16"),
        stage_events=None)
    _check(lib().ttq_linear_noalloc(ctypes.byref(a), _stream(stream)))
    return Y


@_on_launch_stream
def ttq_linear_shared(X: torch.Tensor, layers: list, alpha: float, lambda_rel: float, p: float = 2.0,
                      ws: Optional[torch.Tensor] = None, stream=None) -> list:
    """Several layers on the same X with one statistics pass.  ``layers``:
    dicts with ``W``, ``bits``, ``group`` and optionally ``B``, ``A``, ``Y``,
    ``y_dtype``, ``state`` (only the first layer's state may hold ``ssq``).
    Returns the layers' outputs Y."""
    T, K = X.shape
    arr = (LinearArgs * len(layers))()
    outs = []
    for i, ly in enumerate(layers):
        W = ly["W"]
        M = W.shape[0]
        B, A = ly.get("B"), ly.get("A")
        Y = ly.get("Y")
        if Y is None:
            Y = torch.empty((T, M), dtype=ly.get("y_dtype", torch.float32), device=X.device)
        outs.append(Y)
        st = ly.get("state") or {}
        arr[i] = LinearArgs(
            X=_dev(X, "X"), xt=_dtype_code(X), T=T, K=K, ldx=_ld(X, "X"),
            W=_dev(W, "W"), wt=_dtype_code(W), M=M, ldw=_ld(W, "W"),
            alpha=alpha, lambda_rel=lambda_rel, p=p, bits=ly["bits"], group=ly["group"],
            B=_dev(B, "B"), A=_dev(A, "A"), rank=0 if B is None else B.shape[1],
            Y=_dev(Y, "Y"), yt=_dtype_code(Y), ldy=_ld(Y, "Y"),
            ssq=_dev(st.get("ssq"), "ssq"), s=_dev(st.get("s"), "s"), codes=_dev(st.get("codes"), "codes"),
            scale_f16=_dev(st.get("scale_f16"), "scale_f16"), zero_f16=_dev(st.get("zero_f16"), "zero_f16"),
            stage_events=None)
    if ws is None:
        n = lib().ttq_linear_shared_workspace_bytes(arr, len(layers))
        if n == 0:
            raise ValueError("no call accepts these sizes")
        ws = torch.empty(n, dtype=torch.uint8, device=X.device)
    wp, wn = _ws(ws, X.device)
    _check(lib().ttq_linear_shared(arr, len(layers), wp, wn, _stream(stream)))
    return outs


# ------------------------------------------------------------------ weights chosen per token

TTQ_SCORES = {"softmax": 0, "sigmoid": 1}
TTQ_ACTS = {"silu": 0, "gelu": 1}


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _current_stream(index: int) -> int:
    """The device's current stream as a handle (the direct accessor, where
    torch has it, costs a thirtieth of making a stream object)."""
    return _raw_stream(index) if _raw_stream is not None else torch.cuda.current_stream(index).cuda_stream


def _on_tensor_device(fn):
    """Run a call on its first tensor's device and on ``stream`` (default:
    that device's current stream); what the call allocates belongs to that
    stream."""
    names = list(inspect.signature(fn).parameters)
    first, at = names[0], names.index("stream")

    @functools.wraps(fn)
    def call(*args, stream=None, **kwargs):
        if len(args) == at + 1:           # the stream in its place
            args, stream = args[:at], args[at]
        if args:
            X = args[0]
        elif first in kwargs:
            X = kwargs[first]
        else:
            raise TypeError(f"{fn.__name__}() missing its first argument, {first!r}")
        if not isinstance(X, torch.Tensor) or not X.is_cuda:
            raise TypeError(f"{first} must be a device tensor")
        index = X.get_device()
        if stream is None and index == _current_device():
            return fn(*args, stream=_current_stream(index), **kwargs)
        with torch.cuda.device(index):
            ts = _torch_stream(stream)
            with torch.cuda.stream(ts):
                return fn(*args, stream=ts.cuda_stream, **kwargs)
    return call


def _dense(t: torch.Tensor, name: str, dtype: torch.dtype, shape: tuple, device: int) -> int:
    """The address of a dense tensor of this dtype and shape on this device."""
    try:
        if t.dtype is dtype and t.shape == shape and t.get_device() == device and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    if not isinstance(t, torch.Tensor) or t.dtype is not dtype:
        raise TypeError(f"{name} must be a {dtype} tensor")
    if t.get_device() != device:
        raise ValueError(f"{name} must be on device {device}")
    if t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous {list(shape)} (got {list(t.shape)})")
    return t.data_ptr()


_CODES = {torch.float32: TTQ_F32, torch.bfloat16: TTQ_BF16}


def _code(t: torch.Tensor) -> int:
    c = _CODES.get(t.dtype)
    return c if c is not None else _dtype_code(t)


def _row_stride(t: torch.Tensor, name: str) -> int:
    """Row stride of a matrix; that of a single row does not matter."""
    st = t.stride()
    if len(st) != 2 or st[1] != 1 and t.shape[1] > 1:
        raise ValueError(f"{name} must be 2-D with unit stride in its last dimension")
    return st[0] if t.shape[0] > 1 else t.shape[1]


def _output(Y: Optional[torch.Tensor], shape: tuple, y_dtype, X: torch.Tensor, name: str = "Y") -> torch.Tensor:
    if Y is None:
        return X.new_empty(shape, dtype=y_dtype)
    if Y.get_device() != X.get_device() or Y.shape != shape:
        raise ValueError(f"{name} must be {list(shape)} on {X.device}")
    return Y


def _scratch(ws: Optional[torch.Tensor], n: int, X: torch.Tensor) -> tuple:
    """(address, bytes, tensor) of the workspace, allocated where none is given."""
    if ws is None:
        if n == 0:
            raise ValueError("no call accepts these sizes")
        ws = X.new_empty(n, dtype=torch.uint8)
    elif ws.get_device() != X.get_device() or not ws.is_contiguous():
        raise ValueError(f"ws must be contiguous on {X.device}")
    return _ws(ws, X.device) + (ws,)


def _bytes_tensor(n: int, device) -> torch.Tensor:
    if n == 0:
        raise ValueError("no call accepts these sizes")
    return torch.empty(n, dtype=torch.uint8, device=device)


@_on_tensor_device
def ttq_moe_route(logits: torch.Tensor, topk: int, score: str = "softmax", renormalize: bool = False,
                  ids: Optional[torch.Tensor] = None, w: Optional[torch.Tensor] = None, stream=None):
    """Each token's topk experts (int32 [T][topk], -1 where none is left) and
    their weights (float32 [T][topk]) from its logits [T][E]."""
    if score not in TTQ_SCORES:
        raise ValueError(f"score must be one of {sorted(TTQ_SCORES)}")
    ld = _row_stride(logits, "logits")
    T, E = logits.shape
    dev = logits.get_device()
    k = topk if 0 <= topk <= E else 0     # others are refused below, with nothing allocated for them
    if ids is None:
        ids = logits.new_empty((T, k), dtype=torch.int32)
        ip = ids.data_ptr()
    else:
        ip = _dense(ids, "ids", torch.int32, (T, topk), dev)
    if w is None:
        w = logits.new_empty((T, k), dtype=torch.float32)
        wp = w.data_ptr()
    else:
        wp = _dense(w, "w", torch.float32, (T, topk), dev)
    _check(lib().ttq_moe_route(logits.data_ptr(), _code(logits), T, E, ld, topk, TTQ_SCORES[score],
                               int(bool(renormalize)), ip, wp, stream))
    return ids, w


def ttq_moe_workspace_bytes(T: int, topk: int, K: int, I: int, M: int, E: int, bits: int, group: int) -> int:
    return int(lib().ttq_moe_workspace_bytes(T, topk, K, I, M, E, bits, group))


def moe_workspace(T: int, topk: int, K: int, I: int, M: int, E: int, bits: int, group: int,
                  device="cuda") -> torch.Tensor:
    """Allocate a workspace tensor of ttq_moe_workspace_bytes() bytes."""
    return _bytes_tensor(ttq_moe_workspace_bytes(T, topk, K, I, M, E, bits, group), device)


def _expert_state(name: str, q: dict, E: int, rows: int, K: int, bits: int, group: int, dev) -> ExpertState:
    s = q["s"]
    per = isinstance(s, torch.Tensor) and s.dim() == 2
    return ExpertState(       # in the order of its fields
        _dense(s, name + " s", torch.float32, (E, K) if per else (K,), dev), K if per else 0,
        _dense(q["codes"], name + " codes", torch.int32, (E, rows, K * bits // 32), dev),
        _dense(q["scale_f16"], name + " scale_f16", torch.float16, (E, rows, K // group), dev),
        _dense(q["zero_f16"], name + " zero_f16", torch.float16, (E, rows, K // group), dev))


@_on_tensor_device
def ttq_moe(X: torch.Tensor, ids: torch.Tensor, w: torch.Tensor, gate_up: dict, down: dict, bits: int, group: int,
            act: str = "silu", Y: Optional[torch.Tensor] = None, y_dtype=torch.float32,
            ws: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """A gated mixture-of-experts layer on quantized experts: X [T][K], ids
    and w [T][topk] (ttq_moe_route); gate_up and down: dicts of ``codes``
    [E][rows][.], ``scale_f16`` / ``zero_f16`` [E][rows][K/group] and ``s``
    ([K], or [E][K] for scales per expert), with 2 I rows of K channels (gate
    first) and M rows of I channels.  Returns Y [T][M]."""
    if act not in TTQ_ACTS:
        raise ValueError(f"act must be one of {sorted(TTQ_ACTS)}")
    ldx = _row_stride(X, "X")
    T, K = X.shape
    dev = X.get_device()
    if ids.dim() != 2 or gate_up["codes"].dim() != 3 or down["codes"].dim() != 3:
        raise ValueError("ids must be [T][topk] and codes [E][rows][words]")
    topk = ids.shape[1]
    E, rows2, _ = gate_up["codes"].shape
    M, I = down["codes"].shape[1], rows2 // 2
    if rows2 % 2 or bits <= 0 or group <= 0:
        raise ValueError("gate_up must have an even number of rows; bits and group must be positive")
    Y = _output(Y, (T, M), y_dtype, X)
    wp, wn, ws = _scratch(ws, 0 if ws is not None else lib().ttq_moe_workspace_bytes(T, topk, K, I, M, E, bits, group),
                          X)
    a = MoeArgs(              # in the order of its fields
        X.data_ptr(), _code(X), T, K, ldx, _dense(ids, "ids", torch.int32, (T, topk), dev),
        _dense(w, "w", torch.float32, (T, topk), dev), topk, E, I, M,
        _expert_state("gate_up", gate_up, E, rows2, K, bits, group, dev),
        _expert_state("down", down, E, M, I, bits, group, dev), bits, group, TTQ_ACTS[act], Y.data_ptr(), _code(Y),
        _row_stride(Y, "Y"))
    _check(lib().ttq_moe(ctypes.byref(a), wp, wn, stream))
    return Y


def ttq_adapters_workspace_bytes(T: int, K: int, M: int, rank: int) -> int:
    return int(lib().ttq_adapters_workspace_bytes(T, K, M, rank))


def adapters_workspace(T: int, K: int, M: int, rank: int, device="cuda") -> torch.Tensor:
    """Allocate a workspace tensor of ttq_adapters_workspace_bytes() bytes."""
    return _bytes_tensor(ttq_adapters_workspace_bytes(T, K, M, rank), device)


def _adapters(A, B, ids, ranks, scale, T: int, K: int, M: Optional[int], dev) -> AdaptersArgs:
    if A.dim() != 3 or B.dim() != 3:
        raise ValueError("A must be [n][rank][K] and B [n][M][rank]")
    n, rank, _ = A.shape
    dt = _code(A)
    return AdaptersArgs(      # in the order of its fields
        _dense(A, "A", A.dtype, (n, rank, K), dev),
        _dense(B, "B", A.dtype, (n, B.shape[1] if M is None else M, rank), dev), dt, n, rank,
        None if ranks is None else _dense(ranks, "ranks", torch.int32, (n,), dev),
        None if scale is None else _dense(scale, "scale", torch.float32, (n,), dev),
        _dense(ids, "ids", torch.int32, (T,), dev))


@_on_tensor_device
def ttq_adapters_add(X: torch.Tensor, A: torch.Tensor, B: torch.Tensor, ids: torch.Tensor,
                     C: Optional[torch.Tensor] = None, ranks: Optional[torch.Tensor] = None,
                     scale: Optional[torch.Tensor] = None, Y: Optional[torch.Tensor] = None, y_dtype=None,
                     ws: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Y[t] = C[t] + scale[a] B[a] (A[a] X[t]), a = ids[t] (outside [0, n):
    none): A [n][rank][K], B [n][M][rank], ranks int32 [n] (rows of A in use),
    scale float32 [n].  C (default zeros) has Y's dtype; Y=C works in place."""
    ldx = _row_stride(X, "X")
    T, K = X.shape
    dev = X.get_device()
    ad = _adapters(A, B, ids, ranks, scale, T, K, None, dev)
    M = B.shape[1]
    if y_dtype is None:
        y_dtype = torch.float32 if C is None else C.dtype
    Y = _output(Y, (T, M), y_dtype, X)
    cp, ldc = None, 0
    if C is not None:
        _output(C, (T, M), C.dtype, X, "C")
        if C.dtype != Y.dtype:
            raise TypeError("C must have Y's dtype")
        cp, ldc = C.data_ptr(), _row_stride(C, "C")
    wp, wn, ws = _scratch(ws, 0 if ws is not None else lib().ttq_adapters_workspace_bytes(T, K, M, ad.rank), X)
    _check(lib().ttq_adapters_add(X.data_ptr(), _code(X), T, K, ldx, ctypes.byref(ad), M, cp, ldc, Y.data_ptr(),
                                  _code(Y), _row_stride(Y, "Y"), wp, wn, stream))
    return Y


def ttq_qgemm_adapters_workspace_bytes(T: int, K: int, M: int, bits: int, group: int, rank: int) -> int:
    return int(lib().ttq_qgemm_adapters_workspace_bytes(T, K, M, bits, group, rank))


def qgemm_adapters_workspace(T: int, K: int, M: int, bits: int, group: int, rank: int, device="cuda") -> torch.Tensor:
    """Allocate a workspace tensor of ttq_qgemm_adapters_workspace_bytes() bytes."""
    return _bytes_tensor(ttq_qgemm_adapters_workspace_bytes(T, K, M, bits, group, rank), device)


@_on_tensor_device
def ttq_qgemm_adapters(X: torch.Tensor, s: torch.Tensor, codes: torch.Tensor, scale_f16: torch.Tensor,
                       zero_f16: torch.Tensor, M: int, bits: int, group: int, A: torch.Tensor, B: torch.Tensor,
                       ids: torch.Tensor, ranks: Optional[torch.Tensor] = None,
                       scale: Optional[torch.Tensor] = None, Y: Optional[torch.Tensor] = None,
                       y_dtype=torch.float32, ws: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """ttq_qgemm on one shared quantized state plus each token's adapter (see
    ttq_adapters_add); Y is rounded once."""
    ldx = _row_stride(X, "X")
    T, K = X.shape
    dev = X.get_device()
    if bits <= 0 or group <= 0:
        raise ValueError("bits and group must be positive")
    ad = _adapters(A, B, ids, ranks, scale, T, K, M, dev)
    Y = _output(Y, (T, M), y_dtype, X)
    wp, wn, ws = _scratch(
        ws, 0 if ws is not None else lib().ttq_qgemm_adapters_workspace_bytes(T, K, M, bits, group, ad.rank), X)
    _check(lib().ttq_qgemm_adapters(
        X.data_ptr(), _code(X), T, K, ldx, _dense(s, "s", torch.float32, (K,), dev),
        _dense(codes, "codes", torch.int32, (M, K * bits // 32), dev),
        _dense(scale_f16, "scale_f16", torch.float16, (M, K // group), dev),
        _dense(zero_f16, "zero_f16", torch.float16, (M, K // group), dev), M, bits, group, ctypes.byref(ad),
        Y.data_ptr(), _code(Y), _row_stride(Y, "Y"), wp, wn, stream))
    return Y


# ------------------------------------------------------------------ 8-bit integers, sorted tokens

def _rows8(codes: torch.Tensor, name: str, dev: int) -> int:
    """Row stride of a matrix of 8-bit codes."""
    try:
        st, shape = codes.stride(), codes.shape
        if codes.dtype is torch.int8 and codes.get_device() == dev and len(st) == 2 and st[1] == 1:
            return st[0] if shape[0] > 1 else shape[1]
    except AttributeError:
        pass
    if not isinstance(codes, torch.Tensor) or codes.dtype is not torch.int8:
        raise TypeError(f"{name} must be a torch.int8 tensor")
    if codes.get_device() != dev:
        raise ValueError(f"{name} must be on device {dev}")
    return _row_stride(codes, name)


def _on(t: torch.Tensor, name: str, dev: int) -> torch.Tensor:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a device tensor")
    if t.get_device() != dev:
        raise ValueError(f"{name} must be on device {dev}")
    return t


def _wide_stride(t: torch.Tensor, name: str) -> int:
    """Row stride of a matrix whose rows need not be whole 16-byte pieces
    long; that of a single row does not matter."""
    st, (rows, row) = t.stride(), t.shape if t.dim() == 2 else (0, 0)
    if len(st) != 2 or st[1] != 1 and row > 1:
        raise ValueError(f"{name} must be 2-D with unit stride in its last dimension")
    return st[0] if rows > 1 else -(-row // 8) * 8


def _new_rows(rows: int, row: int, like: torch.Tensor) -> torch.Tensor:
    """A matrix of `like`'s dtype whose rows begin at whole 16-byte pieces
    (dense where their length allows it)."""
    n = 16 // like.element_size()
    return like.new_empty((rows, -(-row // n) * n))[:, :row]


@_on_tensor_device
def ttq_quantize_rows(X: torch.Tensor, s: Optional[torch.Tensor] = None, divide: bool = False,
                      codes: Optional[torch.Tensor] = None, scale: Optional[torch.Tensor] = None, stream=None):
    """Rows of X [R][K] (times s [K], or with divide=True by it) in 8 bits:
    codes int8 [R][K] and scale float32 [R]."""
    ldx = _row_stride(X, "X")
    R, K = X.shape
    dev = X.get_device()
    codes = _output(codes, (R, K), torch.int8, X, "codes")
    ldc = _rows8(codes, "codes", dev)
    if scale is None:
        scale = X.new_empty((R,), dtype=torch.float32)
    _check(lib().ttq_quantize_rows(X.data_ptr(), _code(X), R, K, ldx,
                                   None if s is None else _dense(s, "s", torch.float32, (K,), dev), int(bool(divide)),
                                   codes.data_ptr(), ldc, _dense(scale, "scale", torch.float32, (R,), dev), stream))
    return codes, scale


def ttq_gemm_i8_workspace_bytes(T: int, K: int, M: int) -> int:
    return int(lib().ttq_gemm_i8_workspace_bytes(T, K, M))


def gemm_i8_workspace(T: int, K: int, M: int, device="cuda") -> torch.Tensor:
    """Allocate a workspace tensor of ttq_gemm_i8_workspace_bytes() bytes."""
    return _bytes_tensor(ttq_gemm_i8_workspace_bytes(T, K, M), device)


@_on_tensor_device
def ttq_gemm_i8(X: torch.Tensor, x_scale: torch.Tensor, W: torch.Tensor, w_scale: torch.Tensor,
                Y: Optional[torch.Tensor] = None, y_dtype=torch.float32, ws: Optional[torch.Tensor] = None,
                stream=None) -> torch.Tensor:
    """Product of 8-bit rows (ttq_quantize_rows): Y[t][o] = x_scale[t]
    w_scale[o] sum_j X[t][j] W[o][j], X int8 [T][K], W int8 [M][K]."""
    dev = X.get_device()
    ldx, ldw = _rows8(X, "X", dev), _rows8(W, "W", dev)
    T, K = X.shape
    M = W.shape[0]
    if W.shape[1] != K:
        raise ValueError(f"W must be [M][{K}] (got {list(W.shape)})")
    if Y is None:
        Y, ldy = X.new_empty((T, M), dtype=y_dtype), M
    else:
        ldy = _row_stride(_output(Y, (T, M), None, X), "Y")
    L = lib()
    wp, wn, ws = _scratch(ws, 0 if ws is not None else L.ttq_gemm_i8_workspace_bytes(T, K, M), X)
    _check(L.ttq_gemm_i8(X.data_ptr(), _dense(x_scale, "x_scale", torch.float32, (T,), dev), T, K, ldx, W.data_ptr(),
                         _dense(w_scale, "w_scale", torch.float32, (M,), dev), M, ldw, Y.data_ptr(), _code(Y), ldy,
                         wp, wn, stream))
    return Y


def ttq_qgemm_i8_workspace_bytes(T: int, K: int, M: int) -> int:
    return int(lib().ttq_qgemm_i8_workspace_bytes(T, K, M))


def qgemm_i8_workspace(T: int, K: int, M: int, device="cuda") -> torch.Tensor:
    """Allocate a workspace tensor of ttq_qgemm_i8_workspace_bytes() bytes."""
    return _bytes_tensor(ttq_qgemm_i8_workspace_bytes(T, K, M), device)


@_on_tensor_device
def ttq_qgemm_i8(X: torch.Tensor, s: Optional[torch.Tensor], W: torch.Tensor, w_scale: torch.Tensor,
                 Y: Optional[torch.Tensor] = None, y_dtype=torch.float32, ws: Optional[torch.Tensor] = None,
                 stream=None) -> torch.Tensor:
    """The projection W_hat (X / s) in 8-bit integers: X [T][K] is quantized
    per token (ttq_quantize_rows with divide=True), W int8 [M][K] and w_scale
    [M] are the weight times s in 8 bits."""
    dev = X.get_device()
    ldx, ldw = _row_stride(X, "X"), _rows8(W, "W", dev)
    T, K = X.shape
    M = W.shape[0]
    if W.shape[1] != K:
        raise ValueError(f"W must be [M][{K}] (got {list(W.shape)})")
    if Y is None:
        Y, ldy = X.new_empty((T, M), dtype=y_dtype), M
    else:
        ldy = _row_stride(_output(Y, (T, M), None, X), "Y")
    L = lib()
    wp, wn, ws = _scratch(ws, 0 if ws is not None else L.ttq_qgemm_i8_workspace_bytes(T, K, M), X)
    _check(L.ttq_qgemm_i8(X.data_ptr(), _code(X), T, K, ldx,
                          None if s is None else _dense(s, "s", torch.float32, (K,), dev), W.data_ptr(),
                          _dense(w_scale, "w_scale", torch.float32, (M,), dev), M, ldw, Y.data_ptr(), _code(Y), ldy,
                          wp, wn, stream))
    return Y


def ttq_moe_sort_workspace_bytes(T: int, topk: int, E: int) -> int:
    return int(lib().ttq_moe_sort_workspace_bytes(T, topk, E))


def moe_sort_workspace(T: int, topk: int, E: int, device="cuda") -> torch.Tensor:
    """Allocate a workspace tensor of ttq_moe_sort_workspace_bytes() bytes."""
    return torch.empty(ttq_moe_sort_workspace_bytes(T, topk, E), dtype=torch.uint8, device=device)


@_on_tensor_device
def ttq_moe_sort(ids: torch.Tensor, E: int, offsets: Optional[torch.Tensor] = None,
                 order: Optional[torch.Tensor] = None, pos: Optional[torch.Tensor] = None,
                 ws: Optional[torch.Tensor] = None, stream=None):
    """The slots of ids (int32 [T][topk]) sorted by expert, stably: offsets
    [E + 1] (each expert's rows), order [T * topk] (each row's slot, -1 behind
    the last) and pos [T][topk] (each slot's row, -1 without an expert)."""
    if ids.dim() != 2:
        raise ValueError("ids must be [T][topk]")
    T, topk = ids.shape
    dev = ids.get_device()
    ip = _dense(ids, "ids", torch.int32, (T, topk), dev)
    n = E + 1 if 0 <= E <= 1024 else 0       # others are refused below
    L = lib()
    if offsets is None:
        offsets = ids.new_empty((n,))
        fp = offsets.data_ptr()
    else:
        fp = _dense(offsets, "offsets", torch.int32, (n,), dev)
    if order is None:
        order = ids.new_empty((T * topk,))
        op = order.data_ptr()
    else:
        op = _dense(order, "order", torch.int32, (T * topk,), dev)
    if pos is None:
        pos = ids.new_empty((T, topk))
        pp = pos.data_ptr()
    else:
        pp = _dense(pos, "pos", torch.int32, (T, topk), dev)
    if ws is None:
        need = L.ttq_moe_sort_workspace_bytes(T, topk, E)
        ws = ids.new_empty((need,), dtype=torch.uint8) if need else None
    wp, wn = (None, 0) if ws is None else _scratch(ws, 0, ids)[:2]
    _check(L.ttq_moe_sort(ip, T, topk, E, fp, op, pp, wp, wn, stream))
    return offsets, order, pos


@_on_tensor_device
def ttq_moe_gather(X: torch.Tensor, pos: torch.Tensor, R: Optional[torch.Tensor] = None,
                   stream=None) -> torch.Tensor:
    """R[pos[t][j]] = X[t]: the tokens' rows in their experts' order (pos from
    ttq_moe_sort).  R [rows][K] has X's dtype (default: new, a row for each
    slot, its row stride K rounded up to 16 bytes); rows that no slot names
    are left as they were."""
    ldx = _wide_stride(X, "X")
    T, K = X.shape
    if pos.dim() != 2:
        raise ValueError("pos must be [T][topk]")
    topk = pos.shape[1]
    if R is None:
        R = _new_rows(T * topk, K, X)
    elif _on(R, "R", X.get_device()).dtype != X.dtype or R.dim() != 2 or R.shape[1] != K:
        raise ValueError(f"R must be [rows][{K}] of X's dtype")
    _check(lib().ttq_moe_gather(X.data_ptr(), _code(X), T, K, ldx,
                                _dense(pos, "pos", torch.int32, (T, topk), X.get_device()), topk, R.data_ptr(),
                                R.shape[0], _wide_stride(R, "R"), stream))
    return R


@_on_tensor_device
def ttq_moe_combine(R: torch.Tensor, pos: torch.Tensor, w: Optional[torch.Tensor] = None,
                    Y: Optional[torch.Tensor] = None, y_dtype=None, stream=None) -> torch.Tensor:
    """Y[t] = sum_j w[t][j] R[pos[t][j]] (w None: ones, the gradient of
    ttq_moe_gather); a slot without a row adds nothing.  Y: R's dtype unless
    given."""
    ldr = _wide_stride(R, "R")
    rows, M = R.shape
    if pos.dim() != 2:
        raise ValueError("pos must be [T][topk]")
    T, topk = pos.shape
    dev = R.get_device()
    if Y is None:
        Y = R.new_empty((T, M), dtype=R.dtype if y_dtype is None else y_dtype)
        ldy = M
    else:
        ldy = _row_stride(_output(Y, (T, M), None, R), "Y")
    _check(lib().ttq_moe_combine(R.data_ptr(), _code(R), rows, ldr, _dense(pos, "pos", torch.int32, (T, topk), dev),
                                 None if w is None else _dense(w, "w", torch.float32, (T, topk), dev), T, topk, M,
                                 Y.data_ptr(), _code(Y), ldy, stream))
    return Y


@_on_tensor_device
def ttq_moe_combine_grad(dY: torch.Tensor, R: torch.Tensor, pos: torch.Tensor, w: Optional[torch.Tensor] = None,
                         dR: Optional[torch.Tensor] = None, dw: Optional[torch.Tensor] = None, stream=None):
    """The gradient of ttq_moe_combine: (dR [rows][M], dw [T][topk]) from dY
    [T][M].  dR (default: new, its row stride M rounded up to 16 bytes) keeps
    the rows that no slot names."""
    lddy, ldr = _wide_stride(dY, "dY"), _wide_stride(R, "R")
    T, M = dY.shape
    dev = dY.get_device()
    if _on(R, "R", dev).shape[1] != M or pos.dim() != 2:
        raise ValueError(f"R must be [rows][{M}] and pos [T][topk]")
    topk = pos.shape[1]
    rt = _code(R)
    dR = _new_rows(R.shape[0], M, R) if dR is None else _output(dR, R.shape, R.dtype, dY, "dR")
    if dR.dtype is not R.dtype:
        raise TypeError("dR must have R's dtype")
    if dw is None:
        dw = dY.new_empty((T, topk), dtype=torch.float32)
        dwp = dw.data_ptr()
    else:
        dwp = _dense(dw, "dw", torch.float32, (T, topk), dev)
    _check(lib().ttq_moe_combine_grad(dY.data_ptr(), _code(dY), T, M, lddy, R.data_ptr(), rt, R.shape[0], ldr,
                                      _dense(pos, "pos", torch.int32, (T, topk), dev),
                                      None if w is None else _dense(w, "w", torch.float32, (T, topk), dev), topk,
                                      dR.data_ptr(), _wide_stride(dR, "dR"), dwp, stream))
    return dR, dw


def ttq_moe_i8_workspace_bytes(T: int, topk: int, K: int, I: int, M: int, E: int) -> int:
    return int(lib().ttq_moe_i8_workspace_bytes(T, topk, K, I, M, E))


def moe_i8_workspace(T: int, topk: int, K: int, I: int, M: int, E: int, device="cuda") -> torch.Tensor:
    """Allocate a workspace tensor of ttq_moe_i8_workspace_bytes() bytes."""
    return _bytes_tensor(ttq_moe_i8_workspace_bytes(T, topk, K, I, M, E), device)


def _expert_i8(name: str, q: dict, E: int, rows: int, K: int, dev) -> ExpertI8:
    s = q["s"]
    per = isinstance(s, torch.Tensor) and s.dim() == 2
    return ExpertI8(          # in the order of its fields
        _dense(s, name + " s", torch.float32, (E, K) if per else (K,), dev), K if per else 0,
        _dense(q["codes"], name + " codes", torch.int8, (E, rows, K), dev),
        _dense(q["scale"], name + " scale", torch.float32, (E, rows), dev))


@_on_tensor_device
def ttq_moe_i8(X: torch.Tensor, ids: torch.Tensor, w: torch.Tensor, gate_up: dict, down: dict, act: str = "silu",
               Y: Optional[torch.Tensor] = None, y_dtype=torch.float32, ws: Optional[torch.Tensor] = None,
               stream=None) -> torch.Tensor:
    """A gated mixture-of-experts layer in 8-bit integers, long prompts too
    (T topk up to 2^24, T K below 2^31): X [T][K], ids and w [T][topk]
    (ttq_moe_route); gate_up and down: dicts of ``codes`` int8 [E][rows][K],
    ``scale`` [E][rows] and ``s`` ([K], or [E][K] for scales per expert), with
    2 I rows of K channels (gate first) and M rows of I channels.  Returns Y
    [T][M]."""
    if act not in TTQ_ACTS:
        raise ValueError(f"act must be one of {sorted(TTQ_ACTS)}")
    ldx = _row_stride(X, "X")
    T, K = X.shape
    dev = X.get_device()
    if ids.dim() != 2 or gate_up["codes"].dim() != 3 or down["codes"].dim() != 3:
        raise ValueError("ids must be [T][topk] and codes [E][rows][channels]")
    topk = ids.shape[1]
    E, rows2, _ = gate_up["codes"].shape
    M, I = down["codes"].shape[1], rows2 // 2
    if rows2 % 2:
        raise ValueError("gate_up must have an even number of rows")
    Y = _output(Y, (T, M), y_dtype, X)
    wp, wn, ws = _scratch(ws, 0 if ws is not None else lib().ttq_moe_i8_workspace_bytes(T, topk, K, I, M, E), X)
    a = MoeI8Args(            # in the order of its fields
        X.data_ptr(), _code(X), T, K, ldx, _dense(ids, "ids", torch.int32, (T, topk), dev),
        _dense(w, "w", torch.float32, (T, topk), dev), topk, E, I, M, _expert_i8("gate_up", gate_up, E, rows2, K, dev),
        _expert_i8("down", down, E, M, I, dev), TTQ_ACTS[act], Y.data_ptr(), _code(Y), _row_stride(Y, "Y"))
    _check(lib().ttq_moe_i8(ctypes.byref(a), wp, wn, stream))
    return Y


TTQ_LINEAR_STAGE_EVENTS = 8
LINEAR_STAGES = ("stats", "quantize", "projection", "lowrank")

_hip_handle = None


def _hip() -> ctypes.CDLL:
    """The HIP runtime already loaded by torch (same soname, one runtime)."""
    global _hip_handle
    if _hip_handle is None:
        h = ctypes.CDLL("libamdhip64.so.7")
        h.hipEventCreate.argtypes = [ctypes.c_void_p]
        h.hipEventDestroy.argtypes = [ctypes.c_void_p]
        h.hipEventSynchronize.argtypes = [ctypes.c_void_p]
        h.hipEventElapsedTime.argtypes = [ctypes.POINTER(ctypes.c_float), ctypes.c_void_p, ctypes.c_void_p]
        _hip_handle = h
    return _hip_handle


class StageEvents:
    """TTQ_LINEAR_STAGE_EVENTS timing events for ttq_linear(stage_events=...):
    a (start, stop) pair per stage, stamped by the stage's own kernels."""

    def __init__(self):
        h = _hip()
        self.handles = (ctypes.c_void_p * TTQ_LINEAR_STAGE_EVENTS)()
        for i in range(TTQ_LINEAR_STAGE_EVENTS):
            ev = ctypes.c_void_p()
            if h.hipEventCreate(ctypes.byref(ev)) != 0:
                raise RuntimeError("hipEventCreate failed")
            self.handles[i] = ev

    def stage_ms(self) -> dict:
        """Milliseconds per stage (waits for the last event)."""
        h = _hip()
        if h.hipEventSynchronize(self.handles[-1]) != 0:
            raise RuntimeError("hipEventSynchronize failed")
        out = {}
        for i, name in enumerate(LINEAR_STAGES):
            ms = ctypes.c_float()
            if h.hipEventElapsedTime(ctypes.byref(ms), self.handles[2 * i], self.handles[2 * i + 1]) != 0:
                raise RuntimeError("hipEventElapsedTime failed")
            out[name] = ms.value
        return out

    def __del__(self):
        try:
            h = _hip()
            for ev in self.handles:
                if ev:
                    h.hipEventDestroy(ev)
        except Exception:
            pass


def linear_state(T: int, K: int, M: int, bits: int, group: int, device="cuda") -> dict:
    """Preallocated tensors for the quantization state ttq_linear can fill."""
    return {
        "ssq": torch.empty(K, dtype=torch.float64, device=device),
        "s": torch.empty(K, dtype=torch.float32, device=device),
        "codes": torch.empty((M, K * bits // 32), dtype=torch.int32, device=device),
        "scale_f16": torch.empty((M, K // group), dtype=torch.float16, device=device),
        "zero_f16": torch.empty((M, K // group), dtype=torch.float16, device=device),
    }

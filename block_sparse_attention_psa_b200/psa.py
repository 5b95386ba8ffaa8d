"""Thin Python binding of the C ABI in ``include/psa.h`` (``libpsa.so``).

Argument marshalling only: every step runs in the library's CUDA kernels.
Each function has the name of the C entry point it calls.  Tensors are
PyTorch CUDA tensors (PyTorch is used for device memory and streams); the
call is issued with the device of its main tensor current, on that device's
``torch.cuda.current_stream()`` unless a stream is given.
A non-zero status raises :class:`PSAError`.  There is no fallback: if the
library is missing, :func:`lib` raises.

The serving calls, whose kernels may take less time than reading their
arguments in Python, go through ``_call.so`` (``csrc/call.cpp``) where it is
built: it makes the same call for arguments that are plainly right, and leaves
all others, and every error, to the functions here.
"""

from __future__ import annotations

import ctypes
import functools
import os

import torch

from . import build

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libpsa.so")

PSA_OK = 0
PSA_ERR_ARG = 1
PSA_ERR_SHAPE = 2
PSA_ERR_UNSUPPORTED = 3
PSA_ERR_CAPACITY = 4
PSA_ERR_CUDA = 5
PSA_ERR_TIMEOUT = 6
PSA_ERR_CSR = 7
PSA_ERR_DEVICE = 8
PSA_ERR_LENGTH = 9

PSA_BF16 = 0
PSA_FP16 = 1

EXPORTS = ("psa_status_string", "psa_version", "psa_workspace_size", "psa_route_capacity", "psa_pool",
           "psa_route_topk", "psa_route_thresh", "psa_attn", "psa_dense", "psa_read_status",
           "psa_attn_noalloc", "psa_route_thresh_prob", "psa_test_stall_next_attn",
           "psa_read_fixup_count", "psa_hyd_stat", "psa_attn_hyd", "psa_attn_bwd", "psa_decode_workspace_size",
           "psa_decode", "psa_key_weight_workspace_size", "psa_key_weight", "psa_cache_evict_workspace_size",
           "psa_cache_evict", "psa_test_stall_next_serve")

_lib = None


class PSAError(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        super().__init__(f"{fn}: status {status}: {status_text(status)}")


def _declare(L: ctypes.CDLL) -> None:
    P, I, Z, F = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t, ctypes.c_float
    sig = {
        "psa_status_string": (ctypes.c_char_p, [I]),
        "psa_version": (I, []),
        "psa_workspace_size": (Z, [I, I, I, I]),
        "psa_route_capacity": (Z, [I, I, I, I]),
        "psa_pool": (I, [P, P, P, I, I, I, I, I, P, P, P, P]),
        "psa_route_topk": (I, [P, P, I, I, I, I, F, I, P, P, Z, P, P, P, Z, P]),
        "psa_route_thresh": (I, [P, P, I, I, I, I, F, I, I, P, P, Z, P, P, P, Z, P]),
        "psa_route_thresh_prob": (I, [P, P, I, I, I, I, F, I, I, P, P, Z, P, P, P, Z, P]),
        "psa_attn": (I, [P, P, P, P, P, P, P, Z, P, I, I, I, I, I, I, P, P, P, Z, P]),
        "psa_dense": (I, [P, P, P, I, I, I, I, I, P, P, P, Z, P]),
        "psa_read_status": (I, [P, ctypes.POINTER(I), P]),
        "psa_read_fixup_count": (I, [P, ctypes.POINTER(I), ctypes.POINTER(I), P]),
        "psa_hyd_stat": (I, [P, P, P, P, I, I, I, I, P, P, Z, P]),
        "psa_attn_bwd": (I, [P, P, P, P, P, P, P, Z, I, I, I, I, I, I, P, P, P, P, P, P, P, Z, P]),
        "psa_attn_hyd": (I, [P, P, P, P, P, P, P, P, Z, P, I, I, I, I, I, I, P, P, P, Z, P]),
        "psa_decode_workspace_size": (Z, [I] * 8),
        "psa_decode": (I, [P] * 7 + [I] * 9 + [P, P, P, Z, P]),
        "psa_key_weight_workspace_size": (Z, [I] * 7),
        "psa_key_weight": (I, [P] * 5 + [I] * 9 + [P, P, Z, P]),
        "psa_cache_evict_workspace_size": (Z, [I] * 4),
        "psa_cache_evict": (I, [P] * 5 + [I] * 8 + [P] * 7 + [Z, P]),
        "psa_test_stall_next_attn": (I, [I]),
        "psa_test_stall_next_serve": (I, [I]),
        "psa_attn_noalloc": (I, [P, P, P, P, P, P, P, Z, P, I, I, I, I, I, I, P, P, P, P]),
    }
    for name, (res, args) in sig.items():
        fn = getattr(L, name)
        fn.restype = res
        fn.argtypes = args


def _load_native():
    """The module ``_call`` if it is there and built for this PyTorch and Python
    (it reads tensors by their layout), else None: the same calls, some 10 us
    slower on the host."""
    try:
        from . import _call
    except ImportError:
        return None
    return _call if getattr(_call, "built_for", None) == build.built_for() else None


def __getattr__(name):
    if name == "_native":   # loaded with the library, not on import
        lib()
        return globals()[name]
    raise AttributeError(f"module {__name__!r} has no attribute {name!r}")


def lib() -> ctypes.CDLL:
    """The loaded library (raises if it has not been built), and with it ``_call.so``."""
    global _lib, _native
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing; build it with "
                               "`python -m block_sparse_attention_psa_b200.build`")
        L = ctypes.CDLL(LIB_PATH)
        _declare(L)
        _native = _load_native()
        if _native is not None:
            _native.bind(*(ctypes.cast(f, ctypes.c_void_p).value for f in (
                L.psa_decode, L.psa_decode_workspace_size, L.psa_key_weight, L.psa_key_weight_workspace_size,
                L.psa_cache_evict, L.psa_cache_evict_workspace_size)))
        _lib = L
    return _lib


def status_text(status: int) -> str:
    return lib().psa_status_string(int(status)).decode()


def _check(fn: str, status: int) -> None:
    if status != PSA_OK:
        raise PSAError(fn, status)


def _ptr(t):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("tensor must live on a CUDA device")
    if not t.is_contiguous():
        raise ValueError("tensor must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream, like):
    """The caller's stream, else the current stream of the problem's device."""
    s = stream if stream is not None else torch.cuda.current_stream(like.device)
    return ctypes.c_void_p(s.cuda_stream)


def _call(fn: str, like, *args) -> None:
    """Call the C entry point with the device of ``like`` (the problem's main
    tensor) current: the library launches on the current device and sizes its
    TMA descriptors and scratch for it, so the tensors' device must be the
    current one (the library itself refuses a mismatch with PSA_ERR_DEVICE)."""
    with torch.cuda.device(like.device):
        status = getattr(lib(), fn)(*args)
    _check(fn, status)


def _shape(q):
    if q.dim() != 4 or q.dtype != torch.bfloat16:
        raise ValueError("q, k, v must be bf16 [B, H, N, d]")
    return tuple(int(x) for x in q.shape)


def _expect(name, t, like=None, shape=None, dtype=None, min_numel=None):
    """The C ABI takes plain pointers sized from the problem's dimensions, so
    every tensor is checked against them here, before any pointer is passed:
    a smaller or differently typed buffer would be read or written past its
    end on the device."""
    if t is None:
        return
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if min_numel is not None and t.numel() < min_numel:
        raise ValueError(f"{name} needs at least {min_numel} elements, has {t.numel()}")
    if like is not None and t.device != like.device:
        raise ValueError(f"{name} is on {t.device}, the problem on {like.device}")


def _expect_qkv(q, k, v):
    B, H, N, d = _shape(q)
    _expect("k", k, q, (B, H, N, d), torch.bfloat16)
    _expect("v", v, q, (B, H, N, d), torch.bfloat16)
    return B, H, N, d


def _expect_ws(ws, q, B, H, N, d):
    _expect("ws", ws, q, dtype=torch.uint8, min_numel=psa_workspace_size(B, H, N, d))


def _expect_route_out(out, q, BH, M):
    row_ptr, col_idx, nnz, row_max = out
    _expect("row_ptr", row_ptr, q, dtype=torch.int32, min_numel=BH * M + 1)
    _expect("col_idx", col_idx, q, dtype=torch.int32, min_numel=1)
    _expect("nnz", nnz, q, dtype=torch.int32, min_numel=1)
    _expect("row_max", row_max, q, dtype=torch.float32, min_numel=BH * M)


def psa_workspace_size(B: int, H: int, N: int, d: int) -> int:
    return int(lib().psa_workspace_size(B, H, N, d))


def psa_route_capacity(B: int, H: int, M: int, causal: bool) -> int:
    return int(lib().psa_route_capacity(B, H, M, int(causal)))


def workspace(B: int, H: int, N: int, d: int, device=None) -> torch.Tensor:
    """A device workspace of psa_workspace_size bytes (256-byte aligned)."""
    n = psa_workspace_size(B, H, N, d)
    if n == 0:
        raise PSAError("psa_workspace_size", PSA_ERR_ARG)
    return torch.empty(n, dtype=torch.uint8, device=device or "cuda")


def psa_pool(q, k, v, block_size: int = 64, out=None, stream=None):
    """Returns (qbar, kbar, vsum) float32 [B, H, M, d]."""
    B, H, N, d = _expect_qkv(q, k, v)
    M = N // block_size if block_size > 0 else 0
    if out is None:
        out = tuple(torch.empty(B, H, M, d, dtype=torch.float32, device=q.device) for _ in range(3))
    qbar, kbar, vsum = out
    for name, t in (("qbar", qbar), ("kbar", kbar), ("vsum", vsum)):
        _expect(name, t, q, (B, H, M, d), torch.float32)
    _call("psa_pool", q, _ptr(q), _ptr(k), _ptr(v), B, H, N, d, block_size,
          _ptr(qbar), _ptr(kbar), _ptr(vsum), _stream(stream, q))
    return qbar, kbar, vsum


def _expect_stats(qbar, kbar):
    if qbar.dim() != 4 or qbar.dtype != torch.float32:
        raise ValueError("qbar, kbar must be float32 [B, H, M, d]")
    _expect("kbar", kbar, qbar, tuple(qbar.shape), torch.float32)
    return tuple(int(x) for x in qbar.shape)


def _route_out(B, H, M, causal, capacity, device):
    cap = capacity if capacity is not None else psa_route_capacity(B, H, M, causal)
    return (torch.empty(B * H * M + 1, dtype=torch.int32, device=device),
            torch.empty(max(cap, 1), dtype=torch.int32, device=device),
            torch.empty(1, dtype=torch.int32, device=device),
            torch.empty(B * H * M, dtype=torch.float32, device=device))


def psa_route_topk(qbar, kbar, density: float, causal: bool = False, capacity: int | None = None,
                   out=None, ws=None, stream=None):
    """Returns (row_ptr, col_idx, nnz, row_max): device int32 tensors (nnz has
    one element) and the float32 row maxima of the block scores (``out`` may
    give row_max as None to skip it)."""
    B, H, M, d = _expect_stats(qbar, kbar)
    if ws is None:
        ws = workspace(B, H, M * 64, d, qbar.device)
    if out is None:
        out = _route_out(B, H, M, causal, capacity, qbar.device)
    _expect_ws(ws, qbar, B, H, M * 64, d)
    _expect_route_out(out, qbar, B * H, M)
    row_ptr, col_idx, nnz, row_max = out
    _call("psa_route_topk", qbar, _ptr(qbar), _ptr(kbar), B, H, M, d, float(density), int(causal),
          _ptr(row_ptr), _ptr(col_idx), col_idx.numel(), _ptr(nnz), _ptr(row_max), _ptr(ws), ws.numel(),
          _stream(stream, qbar))
    return row_ptr, col_idx, nnz, row_max


def psa_route_thresh(qbar, kbar, alpha: float, causal: bool = False, keep_first: bool = False,
                     ws=None, capacity: int | None = None, out=None, stream=None):
    """Returns (row_ptr, col_idx, nnz, row_max); nnz > col_idx.numel() means truncated."""
    B, H, M, d = _expect_stats(qbar, kbar)
    if ws is None:
        ws = workspace(B, H, M * 64, d, qbar.device)
    if out is None:
        out = _route_out(B, H, M, causal, capacity, qbar.device)
    _expect_ws(ws, qbar, B, H, M * 64, d)
    _expect_route_out(out, qbar, B * H, M)
    row_ptr, col_idx, nnz, row_max = out
    _call("psa_route_thresh", qbar, _ptr(qbar), _ptr(kbar), B, H, M, d, float(alpha), int(causal),
          int(keep_first), _ptr(row_ptr), _ptr(col_idx), col_idx.numel(), _ptr(nnz), _ptr(row_max), _ptr(ws),
          ws.numel(), _stream(stream, qbar))
    return row_ptr, col_idx, nnz, row_max


def psa_route_thresh_prob(qbar, kbar, alpha: float, causal: bool = False, keep_first: bool = False,
                          ws=None, capacity: int | None = None, out=None, stream=None):
    """Threshold routing in the probability domain: keep J iff
    s_IJ >= max_J s_IJ + ln(alpha).  Returns (row_ptr, col_idx, nnz, row_max)."""
    B, H, M, d = _expect_stats(qbar, kbar)
    if ws is None:
        ws = workspace(B, H, M * 64, d, qbar.device)
    if out is None:
        out = _route_out(B, H, M, causal, capacity, qbar.device)
    _expect_ws(ws, qbar, B, H, M * 64, d)
    _expect_route_out(out, qbar, B * H, M)
    row_ptr, col_idx, nnz, row_max = out
    _call("psa_route_thresh_prob", qbar, _ptr(qbar), _ptr(kbar), B, H, M, d, float(alpha), int(causal),
          int(keep_first), _ptr(row_ptr), _ptr(col_idx), col_idx.numel(), _ptr(nnz), _ptr(row_max), _ptr(ws),
          ws.numel(), _stream(stream, qbar))
    return row_ptr, col_idx, nnz, row_max


def _expect_attn_inputs(q, kbar, vsum, row_ptr, col_idx, row_max, B, H, M, d):
    _expect("kbar", kbar, q, (B, H, M, d), torch.float32)
    _expect("vsum", vsum, q, (B, H, M, d), torch.float32)
    _expect("row_ptr", row_ptr, q, dtype=torch.int32, min_numel=B * H * M + 1)
    _expect("col_idx", col_idx, q, dtype=torch.int32, min_numel=1)
    _expect("row_max", row_max, q, dtype=torch.float32, min_numel=B * H * M)


def psa_attn(q, k, v, kbar, vsum, row_ptr, col_idx, causal: bool = False, block_size: int = 64,
             ws=None, out=None, lse=None, want_lse: bool = False, row_max=None, stream=None):
    """Returns out (bf16 [B,H,N,d]) and, if requested, lse (float32 [B,H,N]).
    ``row_max`` (optional) is a router's row maxima, used as the softmax
    stabiliser instead of computing it in the kernel."""
    B, H, N, d = _expect_qkv(q, k, v)
    M = N // block_size if block_size > 0 else 0
    _expect_attn_inputs(q, kbar, vsum, row_ptr, col_idx, row_max, B, H, M, d)
    if ws is None:
        ws = workspace(B, H, N, d, q.device)
    if out is None:
        out = torch.empty_like(q)
    if lse is None and want_lse:
        lse = torch.empty(B, H, N, dtype=torch.float32, device=q.device)
    _expect_ws(ws, q, B, H, N, d)
    _expect("out", out, q, (B, H, N, d), torch.bfloat16)
    _expect("lse", lse, q, (B, H, N), torch.float32)
    _call("psa_attn", q, _ptr(q), _ptr(k), _ptr(v), _ptr(kbar), _ptr(vsum), _ptr(row_ptr), _ptr(col_idx),
          col_idx.numel(), _ptr(row_max), B, H, N, d, block_size, int(causal), _ptr(out), _ptr(lse), _ptr(ws),
          ws.numel(), _stream(stream, q))
    return (out, lse) if lse is not None else out


def psa_hyd_stat(k, v, kbar, vsum, ws=None, out=None, stream=None):
    """The first-order correction's global statistic: float32 [B, H, d, d],
    the mean over a head's blocks of sum_j (k_j - kbar_J) v_j^T."""
    B, H, N, d = _expect_qkv(k, v, v)
    M = N // 64
    _expect("kbar", kbar, k, (B, H, M, d), torch.float32)
    _expect("vsum", vsum, k, (B, H, M, d), torch.float32)
    if ws is None:
        ws = workspace(B, H, N, d, k.device)
    if out is None:
        out = torch.empty(B, H, d, d, dtype=torch.float32, device=k.device)
    _expect_ws(ws, k, B, H, N, d)
    _expect("hstat", out, k, (B, H, d, d), torch.float32)
    _call("psa_hyd_stat", k, _ptr(k), _ptr(v), _ptr(kbar), _ptr(vsum), B, H, N, d, _ptr(out), _ptr(ws),
          ws.numel(), _stream(stream, k))
    return out


def psa_attn_hyd(q, k, v, kbar, vsum, hstat, row_ptr, col_idx, causal: bool = False, block_size: int = 64,
                 ws=None, out=None, lse=None, want_lse: bool = False, row_max=None, stream=None):
    """psa_attn plus the first-order term of the unselected blocks with the
    global statistic ``hstat`` (float32 [B, H, d, d], from psa_hyd_stat)."""
    B, H, N, d = _expect_qkv(q, k, v)
    M = N // block_size if block_size > 0 else 0
    _expect_attn_inputs(q, kbar, vsum, row_ptr, col_idx, row_max, B, H, M, d)
    _expect("hstat", hstat, q, (B, H, d, d), torch.float32)
    if ws is None:
        ws = workspace(B, H, N, d, q.device)
    if out is None:
        out = torch.empty_like(q)
    if lse is None and want_lse:
        lse = torch.empty(B, H, N, dtype=torch.float32, device=q.device)
    _expect_ws(ws, q, B, H, N, d)
    _expect("out", out, q, (B, H, N, d), torch.bfloat16)
    _expect("lse", lse, q, (B, H, N), torch.float32)
    _call("psa_attn_hyd", q, _ptr(q), _ptr(k), _ptr(v), _ptr(kbar), _ptr(vsum), _ptr(hstat), _ptr(row_ptr),
          _ptr(col_idx), col_idx.numel(), _ptr(row_max), B, H, N, d, block_size, int(causal), _ptr(out),
          _ptr(lse), _ptr(ws), ws.numel(), _stream(stream, q))
    return (out, lse) if lse is not None else out


def psa_attn_bwd(q, k, v, kbar, vsum, row_ptr, col_idx, out, lse, dout, causal: bool = False,
                 block_size: int = 64, ws=None, grads=None, stream=None):
    """Gradients (dq, dk, dv), bf16 [B, H, N, d], of the 0th-order attention
    of psa_attn for fixed block lists, given its output ``out``, its ``lse``
    and dL/dout ``dout``."""
    B, H, N, d = _expect_qkv(q, k, v)
    M = N // block_size if block_size > 0 else 0
    _expect_attn_inputs(q, kbar, vsum, row_ptr, col_idx, None, B, H, M, d)
    _expect("out", out, q, (B, H, N, d), torch.bfloat16)
    _expect("dout", dout, q, (B, H, N, d), torch.bfloat16)
    if lse is None:
        raise ValueError("lse (float32 [B, H, N]) of the forward call is required")
    _expect("lse", lse, q, (B, H, N), torch.float32)
    if ws is None:
        ws = workspace(B, H, N, d, q.device)
    if grads is None:
        grads = tuple(torch.empty_like(q) for _ in range(3))
    dq, dk, dv = grads
    for name, t in (("dq", dq), ("dk", dk), ("dv", dv)):
        _expect(name, t, q, (B, H, N, d), torch.bfloat16)
    _expect_ws(ws, q, B, H, N, d)
    _call("psa_attn_bwd", q, _ptr(q), _ptr(k), _ptr(v), _ptr(kbar), _ptr(vsum), _ptr(row_ptr), _ptr(col_idx),
          col_idx.numel(), B, H, N, d, block_size, int(causal), _ptr(out), _ptr(lse), _ptr(dout), _ptr(dq),
          _ptr(dk), _ptr(dv), _ptr(ws), ws.numel(), _stream(stream, q))
    return dq, dk, dv


def psa_dense(q, k, v, causal: bool = False, ws=None, out=None, lse=None, want_lse: bool = False,
              stream=None):
    """Dense softmax attention through the same tensor-core kernel."""
    B, H, N, d = _expect_qkv(q, k, v)
    if ws is None:
        ws = workspace(B, H, N, d, q.device)
    if out is None:
        out = torch.empty_like(q)
    if lse is None and want_lse:
        lse = torch.empty(B, H, N, dtype=torch.float32, device=q.device)
    _expect_ws(ws, q, B, H, N, d)
    _expect("out", out, q, (B, H, N, d), torch.bfloat16)
    _expect("lse", lse, q, (B, H, N), torch.float32)
    _call("psa_dense", q, _ptr(q), _ptr(k), _ptr(v), B, H, N, d, int(causal), _ptr(out), _ptr(lse), _ptr(ws),
          ws.numel(), _stream(stream, q))
    return (out, lse) if lse is not None else out


def psa_attn_noalloc(q, k, v, kbar, vsum, row_ptr, col_idx, causal: bool = False, block_size: int = 64,
                     out=None, lse=None, status=None, row_max=None, stream=None):
    """psa_attn without a workspace, for callers that cannot allocate device
    memory (framework plugins restricted to the framework's own pool, loops
    that forbid allocation after start-up): the library's own 16 MiB scratch
    array is used instead, and calls that overlap on the GPU race on it.  ``status`` is an optional device
    int32 tensor that receives this call's device status word."""
    B, H, N, d = _expect_qkv(q, k, v)
    M = N // block_size if block_size > 0 else 0
    _expect_attn_inputs(q, kbar, vsum, row_ptr, col_idx, row_max, B, H, M, d)
    if out is None:
        out = torch.empty_like(q)
    _expect("out", out, q, (B, H, N, d), torch.bfloat16)
    _expect("lse", lse, q, (B, H, N), torch.float32)
    _expect("status", status, q, dtype=torch.int32, min_numel=1)
    _call("psa_attn_noalloc", q, _ptr(q), _ptr(k), _ptr(v), _ptr(kbar), _ptr(vsum), _ptr(row_ptr),
          _ptr(col_idx), col_idx.numel(), _ptr(row_max), B, H, N, d, block_size, int(causal), _ptr(out),
          _ptr(lse), _ptr(status), _stream(stream, q))
    return out


_DTYPES = {torch.bfloat16: PSA_BF16, torch.float16: PSA_FP16}


def _dtype16(name, t):
    dt = _DTYPES.get(t.dtype)
    if dt is None:
        raise ValueError(f"{name} must be bfloat16 or float16, got {t.dtype}")
    return dt


def _shape4(name, t):
    if t.dim() != 4:
        raise ValueError(f"{name} must have 4 dimensions, got {tuple(t.shape)}")
    return t.shape


def _arg(name, t, like, shape, dtype):
    """The address of a tensor argument, checked against the problem (None
    stays None).  A serving call takes microseconds on the device, so the
    accepted case is one comparison each."""
    if t is None:
        return None
    if t.shape != shape or t.dtype is not dtype or t.get_device() != like.get_device() or not t.is_contiguous():
        _expect(name, t, like, shape, dtype)
        raise ValueError("tensor must be contiguous")
    return t.data_ptr()


def _on_stream(stream, like):
    """The given stream as the current one: what is allocated under it then
    belongs to it.  It has to be of the problem's device, whose current stream
    the call takes."""
    if stream.device != like.device:
        raise ValueError(f"stream is on {stream.device}, the problem on {like.device}")
    return torch.cuda.stream(stream)


def _serve(fn, like, *args):
    """Call a serving entry point on the problem's device and its current
    stream."""
    dev = like.get_device()   # every other tensor is on it too
    if dev < 0:
        raise ValueError("tensor must live on a CUDA device")
    s = torch._C._cuda_getCurrentRawStream(dev)
    if dev == torch.cuda.current_device():
        status = getattr(lib(), fn)(*args, s)
    else:
        with torch.cuda.device(dev):
            status = getattr(lib(), fn)(*args, s)
    if status != PSA_OK:
        raise PSAError(fn, status)


def _serve_ws(ws, need, like):
    if ws is None:
        ws = torch.empty(max(need, 256), dtype=torch.uint8, device=like.device)
    elif ws.dtype is not torch.uint8 or ws.numel() < need or ws.get_device() != like.get_device() \
            or not ws.is_contiguous():
        _expect("ws", ws, like, dtype=torch.uint8, min_numel=need)
        raise ValueError("tensor must be contiguous")
    return ws


def _new_ws(fn, n, device):
    if n == 0:
        raise PSAError(fn, PSA_ERR_ARG)
    return torch.empty(n, dtype=torch.uint8, device=device or "cuda")


@functools.lru_cache(maxsize=256)
def psa_decode_workspace_size(B: int, Hq: int, Hkv: int, T: int, d: int, Bp: int = 1, P: int = 0, C: int = 0) -> int:
    return int(lib().psa_decode_workspace_size(B, Hq, Hkv, T, d, Bp, P, C))


def decode_workspace(B, Hq, Hkv, T, d, Bp=1, P=0, C=0, device=None) -> torch.Tensor:
    """A device workspace of psa_decode_workspace_size bytes."""
    return _new_ws("psa_decode_workspace_size", psa_decode_workspace_size(B, Hq, Hkv, T, d, Bp, P, C), device)


def psa_decode(q, k_cache=None, v_cache=None, cache_len=None, k_prefix=None, v_prefix=None, prefix_len=None,
               ws=None, out=None, lse=None, want_lse: bool = False, stream=None):
    """Attention of new tokens q [B, Hq, T, d] (bf16 or fp16) over a prefix
    [Bp, Hkv, P, d] that groups of B / Bp sequences share and each sequence's
    own cache [B, Hkv, C, d], in one softmax.  ``prefix_len`` [Bp] and
    ``cache_len`` [B] (int32, None: the capacity) are the valid lengths; the
    last T valid cache entries are the new tokens (query t sees slots below
    cache_len - (T - 1 - t)).  Rows past a length may hold anything; the new
    tokens' values must be finite.  Returns out and, if requested, lse (float32
    [B, Hq, T])."""
    if stream is not None:
        with _on_stream(stream, q):
            return psa_decode(q, k_cache, v_cache, cache_len, k_prefix, v_prefix, prefix_len, ws, out, lse, want_lse)
    if _lib is None:
        lib()
    if _native is not None:
        r = _native.decode(q, k_cache, v_cache, cache_len, k_prefix, v_prefix, prefix_len, ws, out, lse, want_lse)
        if r is not None:
            return r
    B, Hq, T, d = _shape4("q", q)
    dt = _dtype16("q", q)
    if k_cache is None and k_prefix is None:
        raise ValueError("a cache or a prefix is required")
    Bp, P, C, Hkv = 1, 0, 0, 0
    if k_prefix is not None:
        Bp, Hkv, P, _ = _shape4("k_prefix", k_prefix)
        if v_prefix is None:
            raise ValueError("v_prefix is required with k_prefix")
    elif v_prefix is not None or prefix_len is not None:
        raise ValueError("v_prefix and prefix_len need k_prefix")
    if k_cache is not None:
        _, Hc, C, _ = _shape4("k_cache", k_cache)
        Hkv = Hkv or Hc
        if v_cache is None:
            raise ValueError("v_cache is required with k_cache")
    elif v_cache is not None or cache_len is not None:
        raise ValueError("v_cache and cache_len need k_cache")
    pre, own = (Bp, Hkv, P, d), (B, Hkv, C, d)
    args = (_arg("k_prefix", k_prefix, q, pre, q.dtype), _arg("v_prefix", v_prefix, q, pre, q.dtype),
            _arg("prefix_len", prefix_len, q, (Bp,), torch.int32), _arg("k_cache", k_cache, q, own, q.dtype),
            _arg("v_cache", v_cache, q, own, q.dtype), _arg("cache_len", cache_len, q, (B,), torch.int32))
    ws = _serve_ws(ws, psa_decode_workspace_size(B, Hq, Hkv, T, d, Bp, P, C), q)
    at_q = _arg("q", q, q, q.shape, q.dtype)
    if out is None:
        out = torch.empty_like(q)   # (new buffers need no check)
        at_out = out.data_ptr()
    else:
        at_out = _arg("out", out, q, q.shape, q.dtype)
    if lse is None and want_lse:
        lse = torch.empty(B, Hq, T, dtype=torch.float32, device=q.device)
        at_lse = lse.data_ptr()
    else:
        at_lse = _arg("lse", lse, q, (B, Hq, T), torch.float32)
    _serve("psa_decode", q, at_q, *args, B, Hq, Hkv, T, d, Bp, P, C, dt, at_out, at_lse, ws.data_ptr(), ws.numel())
    return (out, lse) if lse is not None else out


@functools.lru_cache(maxsize=256)
def psa_key_weight_workspace_size(B: int, Hq: int, Hkv: int, T: int, d: int, Bk: int, C: int) -> int:
    return int(lib().psa_key_weight_workspace_size(B, Hq, Hkv, T, d, Bk, C))


def key_weight_workspace(B, Hq, Hkv, T, d, Bk, C, device=None) -> torch.Tensor:
    """A device workspace of psa_key_weight_workspace_size bytes."""
    return _new_ws("psa_key_weight_workspace_size", psa_key_weight_workspace_size(B, Hq, Hkv, T, d, Bk, C), device)


def psa_key_weight(q, k, lse, key_len=None, causal: bool = False, score=None, ws=None, out=None, stream=None):
    """Accumulated attention weight of each cached key, float32 [Bk, Hkv, C]:
    ``score`` (None: zero) plus, per slot j of k [Bk, Hkv, C, d], the sum of
    exp(q . k_j / sqrt(d) - lse) over the queries q [B, Hq, T, d] that see it
    (groups of B / Bk sequences read one key set; causal: token t sees slots
    below key_len - (T - 1 - t)).  Slots past ``key_len`` get 0.  ``out`` may
    be ``score`` itself."""
    if stream is not None:
        with _on_stream(stream, q):
            return psa_key_weight(q, k, lse, key_len, causal, score, ws, out)
    if _lib is None:
        lib()
    if _native is not None:
        r = _native.key_weight(q, k, lse, key_len, causal, score, ws, out)
        if r is not None:
            return r
    B, Hq, T, d = _shape4("q", q)
    dt = _dtype16("q", q)
    Bk, Hkv, C, _ = _shape4("k", k)
    if lse is None:
        raise ValueError("lse (float32 [B, Hq, T]) of the queries is required")
    slots = (Bk, Hkv, C)
    args = (_arg("q", q, q, q.shape, q.dtype), _arg("k", k, q, (Bk, Hkv, C, d), q.dtype),
            _arg("lse", lse, q, (B, Hq, T), torch.float32), _arg("key_len", key_len, q, (Bk,), torch.int32),
            _arg("score", score, q, slots, torch.float32))
    ws = _serve_ws(ws, psa_key_weight_workspace_size(B, Hq, Hkv, T, d, Bk, C), q)
    if out is None:
        out = torch.empty(Bk, Hkv, C, dtype=torch.float32, device=q.device)
        at_out = out.data_ptr()
    else:
        at_out = _arg("out", out, q, slots, torch.float32)
    _serve("psa_key_weight", q, *args, B, Hq, Hkv, T, d, Bk, C, int(causal), dt, at_out, ws.data_ptr(), ws.numel())
    return out


@functools.lru_cache(maxsize=256)
def psa_cache_evict_workspace_size(B: int, Hkv: int, C: int, budget: int) -> int:
    return int(lib().psa_cache_evict_workspace_size(B, Hkv, C, budget))


def cache_evict_workspace(B, Hkv, C, budget, device=None) -> torch.Tensor:
    """A device workspace of psa_cache_evict_workspace_size bytes."""
    return _new_ws("psa_cache_evict_workspace_size", psa_cache_evict_workspace_size(B, Hkv, C, budget), device)


def psa_cache_evict(k, v, score, budget: int, pos=None, cache_len=None, sink: int = 0, recent: int = 0, ws=None,
                    out=None, stream=None):
    """Keeps min(cache_len, budget) entries of every (sequence, KV head) of a
    cache k, v [B, Hkv, C, d]: those at positions below ``sink``, the
    ``recent`` latest, and the ones of largest ``score`` (float32 [B, Hkv, C],
    equal scores by slot).  Returns (k, v, score, pos, length, kept): the
    caches [B, Hkv, budget, d], their scores and positions, the new lengths
    [B] and kept [B, Hkv, budget], the slot each entry came from (-1 past the
    length).  ``out`` gives these six buffers instead; with the inputs
    themselves as the first four the eviction is in place."""
    if stream is not None:
        with _on_stream(stream, k):
            return psa_cache_evict(k, v, score, budget, pos, cache_len, sink, recent, ws, out)
    if _lib is None:
        lib()
    if _native is not None:
        r = _native.cache_evict(k, v, score, budget, pos, cache_len, sink, recent, ws, out)
        if r is not None:
            return r
    B, Hkv, C, d = _shape4("k", k)
    _dtype16("k", k)
    need = psa_cache_evict_workspace_size(B, Hkv, C, budget)
    full = (B, Hkv, C, d)
    at_k, at_v = _arg("k", k, k, full, k.dtype), _arg("v", v, k, full, k.dtype)
    at_score = _arg("score", score, k, (B, Hkv, C), torch.float32)
    at_pos = _arg("pos", pos, k, (B, Hkv, C), torch.int32)
    at_len = _arg("cache_len", cache_len, k, (B,), torch.int32)
    ws = _serve_ws(ws, need, k)
    if out is None:
        if need == 0:
            raise PSAError("psa_cache_evict", PSA_ERR_ARG if budget <= 0 else PSA_ERR_SHAPE)
        new = lambda *s, dtype: torch.empty(*s, dtype=dtype, device=k.device)  # noqa: E731
        out = (new(B, Hkv, budget, d, dtype=k.dtype), new(B, Hkv, budget, d, dtype=k.dtype),
               new(B, Hkv, budget, dtype=torch.float32), new(B, Hkv, budget, dtype=torch.int32),
               new(B, dtype=torch.int32), new(B, Hkv, budget, dtype=torch.int32))
    k_out, v_out, score_out, pos_out, len_out, kept = out
    # (in place: the inputs, which are checked)
    if k_out is k and v_out is v and score_out is score:
        C_out, slots, outs = C, (B, Hkv, C), (at_k, at_v, at_score)
    else:
        C_out = _shape4("k_out", k_out)[2]
        rows, slots = (B, Hkv, C_out, d), (B, Hkv, C_out)
        outs = (_arg("k_out", k_out, k, rows, k.dtype), _arg("v_out", v_out, k, rows, k.dtype),
                _arg("score_out", score_out, k, slots, torch.float32))
    _serve("psa_cache_evict", k, at_k, at_v, at_score, at_pos, at_len, B, Hkv, C, d, budget, sink, recent, C_out, *outs,
           at_pos if pos_out is pos and C_out == C else _arg("pos_out", pos_out, k, slots, torch.int32),
           at_len if len_out is cache_len else _arg("len_out", len_out, k, (B,), torch.int32),
           _arg("kept", kept, k, (B, Hkv, budget), torch.int32), ws.data_ptr(), ws.numel())
    return k_out, v_out, score_out, pos_out, len_out, kept


def psa_test_stall_next_attn(on: bool = True) -> None:
    """Failure-path test hook: the next psa_attn call's kernel lets a bounded
    wait run out and records PSA_ERR_TIMEOUT in its workspace status word."""
    _check("psa_test_stall_next_attn", lib().psa_test_stall_next_attn(int(bool(on))))


def psa_test_stall_next_serve(on: bool = True) -> None:
    """The same for the next psa_decode, or psa_key_weight of many queries."""
    _check("psa_test_stall_next_serve", lib().psa_test_stall_next_serve(int(bool(on))))


def psa_read_status(ws, stream=None) -> int:
    """Synchronise the stream and return the device status word of ``ws``."""
    _expect("ws", ws, dtype=torch.uint8, min_numel=256)
    st = ctypes.c_int(-1)
    _call("psa_read_status", ws, _ptr(ws), ctypes.byref(st), _stream(stream, ws))
    return int(st.value)


def psa_read_fixup_count(ws, stream=None):
    """Synchronise the stream and return (rerun, exact): the query blocks the
    last attention call on ``ws`` recomputed with per-query stabilisers on the
    tensor cores, and those of them that needed the exact CUDA-core path."""
    _expect("ws", ws, dtype=torch.uint8, min_numel=256)
    rerun, exact = ctypes.c_int(-1), ctypes.c_int(-1)
    _call("psa_read_fixup_count", ws, _ptr(ws), ctypes.byref(rerun), ctypes.byref(exact), _stream(stream, ws))
    return int(rerun.value), int(exact.value)


def psa_forward(q, k, v, mode: str = "topk", density: float = 0.15, alpha: float = 0.5,
                causal: bool = False, keep_first: bool = False, hyd: bool = False, ws=None, stream=None):
    """The whole path in one call (pool -> route -> attention), as the usage
    line of the PISA summary calls it: f(q, k, v, density=0.15, block_size=64).
    ``hyd`` adds the first-order correction with the global statistic.
    Returns (out, (row_ptr, col_idx, nnz, row_max))."""
    B, H, N, d = _shape(q)
    if ws is None:
        ws = workspace(B, H, N, d, q.device)
    qbar, kbar, vsum = psa_pool(q, k, v, stream=stream)
    if mode == "topk":
        csr = psa_route_topk(qbar, kbar, density, causal, ws=ws, stream=stream)
    elif mode == "thresh":
        csr = psa_route_thresh(qbar, kbar, alpha, causal, keep_first, ws=ws, stream=stream)
    elif mode == "thresh_prob":
        csr = psa_route_thresh_prob(qbar, kbar, alpha, causal, keep_first, ws=ws, stream=stream)
    else:
        raise ValueError("mode must be 'topk', 'thresh' or 'thresh_prob'")
    if hyd:
        hstat = psa_hyd_stat(k, v, kbar, vsum, ws=ws, stream=stream)
        out = psa_attn_hyd(q, k, v, kbar, vsum, hstat, csr[0], csr[1], causal, ws=ws, row_max=csr[3],
                           stream=stream)
    else:
        out = psa_attn(q, k, v, kbar, vsum, csr[0], csr[1], causal, ws=ws, row_max=csr[3], stream=stream)
    return out, csr

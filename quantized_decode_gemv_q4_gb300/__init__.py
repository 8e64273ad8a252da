"""GB300 4-bit decode GEMVs: a thin Python binding over the C ABI in ``include/q4gemv.h``.

Each function has the name of its C entry point and takes CUDA tensors (PyTorch is used only for
device memory and streams). Shapes give the sizes; the call is enqueued on the given stream (default:
the current stream) and returns at once. A refusal or a CUDA failure raises :class:`Q4Error` with the
library's message. There is no CPU path: without the compiled library every call raises.

Layouts (row-major, little-endian):
  * Q4 planar: ``qs`` uint8 ``[N, K/32, 16]`` (or ``[N, K/2]``), ``d`` float16 ``[N, K/32]``.
  * Q4_K: ``w`` uint8 ``[N, K/256, 144]`` (or ``[N, K/256*144]``).
  * inputs and outputs of the GEMVs float32; of the norm/rotation, cache and attention calls float32, float16 or
    bfloat16 (one type per call).
  * 4-bit cache: :class:`KV4Cache`, planar Q4 rows in pages ``[num_pages, num_kv_heads, page_size, ...]``.
"""

from __future__ import annotations

import ctypes
import os

import torch

from . import build as _build

__all__ = [
    "Q4Error", "load", "q4_fma_ceiling", "q4_gemv", "q4_gemv_batched", "fused_rmsnorm_q4k_gemv", "fused_gateup_q4k_gemv",
    "moe_q4_gemv", "q4k_gemv_batched", "fused_gateup_swiglu_q4k_gemv", "moe_q4_swiglu_gemv", "moe_router_q4", "q4_pure_read",
    "q4k_pure_read",
    "moe_q4_pure_read", "q4_dequant", "q4k_dequant",
    "KV4Cache", "qk_norm_rope", "kv4_write", "kv4_read", "kv4_attention", "kv4_attention_workspace",
    "q4_device_faults", "q4_set_launch_overlap", "q4_get_launch_overlap", "q4_set_wait_limit", "q4_get_wait_limit",
    "FAULT_BAD_EXPERT", "FAULT_WAIT_TIMEOUT", "FAULT_COPY_LOST", "DEFAULT_WAIT_LIMIT",
    "FAULT_BAD_SLOT", "FAULT_BAD_PAGE", "FAULT_BAD_LENGTH", "FAULT_BAD_POSITION",
]

Q4_OK, Q4_EINVAL, Q4_EALIGN, Q4_ECUDA, Q4_EUNSUPPORTED = 0, -1, -2, -3, -4
FAULT_BAD_EXPERT = 4
FAULT_WAIT_TIMEOUT = 8
FAULT_COPY_LOST = 16
FAULT_BAD_SLOT = 32
FAULT_BAD_PAGE = 64
FAULT_BAD_LENGTH = 128
FAULT_BAD_POSITION = 256
DEFAULT_WAIT_LIMIT = 4_000_000_000
_CODE_NAMES = {Q4_EINVAL: "EINVAL", Q4_EALIGN: "EALIGN", Q4_ECUDA: "ECUDA", Q4_EUNSUPPORTED: "EUNSUPPORTED"}


class Q4Error(RuntimeError):
    def __init__(self, code: int, message: str):
        super().__init__(f"{_CODE_NAMES.get(code, code)}: {message}")
        self.code = code


_lib = None
_P = ctypes.c_void_p
_I = ctypes.c_int
_L = ctypes.c_longlong

_SIGNATURES = {
    "q4_gemv": [_P, _P, _P, _P, _I, _I, _P],
    "q4_gemv_batched": [_P, _P, _P, _P, _I, _I, _I, _P],
    "fused_rmsnorm_q4k_gemv": [_P, _P, _P, _P, ctypes.c_float, _I, _I, _P],
    "fused_gateup_q4k_gemv": [_P, _P, _P, _P, _P, _P, ctypes.c_float, _I, _I, _P],
    "moe_q4_gemv": [_P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _P, _P],
    "q4_pure_read": [_P, _P, _P, _I, _I, _P],
    "q4k_pure_read": [_P, _P, _I, _I, _P],
    "moe_q4_pure_read": [_P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _P, _P],
    "q4_dequant": [_P, _P, _P, _I, _I, _P],
    "q4k_dequant": [_P, _P, _I, _I, _P],
    "fused_gateup_swiglu_q4k_gemv": [_P, _P, _P, _P, _P, ctypes.c_float, _I, _I, _P],
    "moe_q4_swiglu_gemv": [_P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _P, _P],
    "moe_router_q4": [_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _P],
    "q4k_gemv_batched": [_P, _P, _P, _I, _I, _I, _P],
    "qk_norm_rope": [_P, _P, _P, _P, _P, _P, ctypes.c_float, _P, _P, _I, _I, _I, _I, _I, _I, _I, _L, _L, _L, _L, _I, _P],
    "kv4_write": [_P, _P, _P, _P, _I, _L, _L, _I, _P],
    "kv4_read": [_P, _P, _P, _P, _I, _L, _L, _I, _P],
    "kv4_attention_workspace": [ctypes.POINTER(ctypes.c_size_t), _I, _I, _I, _I, _I],
    "kv4_attention": [_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _L, _L, ctypes.c_float, _I, _I, _P, ctypes.c_size_t, _P],
    "q4_device_faults": [ctypes.POINTER(ctypes.c_uint)],
    "q4_fma_ceiling": [_P, _I, ctypes.c_longlong, ctypes.c_float, ctypes.c_float, ctypes.POINTER(ctypes.c_longlong),
                       _P],
}


def lib_path() -> str:
    return _build.LIB_PATH


def load(path: str | None = None) -> ctypes.CDLL:
    """Load (once) the compiled library; raise if it was never built."""
    global _lib
    if _lib is None:
        p = path or lib_path()
        if not os.path.exists(p):
            raise RuntimeError(f"libq4gemv is not built ({p} missing): run quantized_decode_gemv_q4_gb300/build.py")
        L = ctypes.CDLL(p)
        for name, args in _SIGNATURES.items():
            fn = getattr(L, name)
            fn.argtypes = args
            fn.restype = ctypes.c_int
        L.q4_last_error.argtypes = []
        L.q4_last_error.restype = ctypes.c_char_p
        L.q4_set_launch_overlap.argtypes = [ctypes.c_int]
        L.q4_set_launch_overlap.restype = ctypes.c_int
        L.q4_get_launch_overlap.argtypes = []
        L.q4_get_launch_overlap.restype = ctypes.c_int
        L.q4_set_wait_limit.argtypes = [ctypes.c_longlong]
        L.q4_set_wait_limit.restype = ctypes.c_int
        L.q4_get_wait_limit.argtypes = []
        L.q4_get_wait_limit.restype = ctypes.c_longlong
        _lib = L
    return _lib


def _check(rc: int) -> None:
    if rc != Q4_OK:
        raise Q4Error(rc, load().q4_last_error().decode())


def _ptr(t: torch.Tensor | None, dtype: torch.dtype, name: str) -> int | None:
    if t is None:
        return None
    if t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise TypeError(f"{name}: expected a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous tensor")
    return t.data_ptr()


def _stream(stream) -> int:
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _q4_dims(qs: torch.Tensor, d: torch.Tensor):
    N = d.shape[0]
    K = d.numel() // N * 32
    if qs.numel() != N * K // 2:
        raise ValueError(f"qs holds {qs.numel()} bytes, expected N*K/2 = {N * K // 2}")
    return N, K


def _q4k_dims(w: torch.Tensor):
    N = w.shape[0]
    if (w.numel() // N) % 144:
        raise ValueError("Q4_K rows must be a whole number of 144-byte super-blocks")
    return N, w.numel() // N // 144 * 256


def q4_gemv(y, qs, d, x, stream=None) -> None:
    N, K = _q4_dims(qs, d)
    if x.numel() != K or y.numel() != N:
        raise ValueError("x must hold K values and y N values")
    _check(load().q4_gemv(_ptr(y, torch.float32, "y"), _ptr(qs, torch.uint8, "qs"), _ptr(d, torch.float16, "d"),
                          _ptr(x, torch.float32, "x"), N, K, _stream(stream)))


def q4_gemv_batched(Y, qs, d, X, stream=None) -> None:
    N, K = _q4_dims(qs, d)
    M = X.shape[0] if X.dim() == 2 else 1
    if X.numel() != M * K or Y.numel() != M * N:
        raise ValueError("X must be [M, K] and Y [M, N]")
    _check(load().q4_gemv_batched(_ptr(Y, torch.float32, "Y"), _ptr(qs, torch.uint8, "qs"),
                                  _ptr(d, torch.float16, "d"), _ptr(X, torch.float32, "X"), M, N, K,
                                  _stream(stream)))


def fused_rmsnorm_q4k_gemv(y, w, x, gamma, eps: float = 1e-5, stream=None) -> None:
    N, K = _q4k_dims(w)
    if x.numel() != K or gamma.numel() != K or y.numel() != N:
        raise ValueError("x and gamma must hold K values and y N values")
    _check(load().fused_rmsnorm_q4k_gemv(_ptr(y, torch.float32, "y"), _ptr(w, torch.uint8, "w"),
                                         _ptr(x, torch.float32, "x"), _ptr(gamma, torch.float32, "gamma"),
                                         float(eps), N, K, _stream(stream)))


def q4k_gemv_batched(Y, w, X, stream=None) -> None:
    """Y[m] = W X[m] for the M rows of X (Q4_K weights, no normalisation), one weight sweep."""
    N, K = _q4k_dims(w)
    M = X.numel() // K
    if X.numel() != M * K or Y.numel() != M * N:
        raise ValueError("X must be [M, K] and Y [M, N]")
    _check(load().q4k_gemv_batched(_ptr(Y, torch.float32, "Y"), _ptr(w, torch.uint8, "w"), _ptr(X, torch.float32, "X"),
                                   M, N, K, _stream(stream)))


def fused_gateup_q4k_gemv(y_gate, y_up, w_gate, w_up, x, gamma=None, eps: float = 1e-5, stream=None) -> None:
    N, K = _q4k_dims(w_gate)
    if _q4k_dims(w_up) != (N, K) or x.numel() != K or y_gate.numel() != N or y_up.numel() != N:
        raise ValueError("gate and up must be [N, K/256, 144], x K values, outputs N values")
    if gamma is not None and gamma.numel() != K:
        raise ValueError("gamma must hold K values")
    _check(load().fused_gateup_q4k_gemv(_ptr(y_gate, torch.float32, "y_gate"), _ptr(y_up, torch.float32, "y_up"),
                                        _ptr(w_gate, torch.uint8, "w_gate"), _ptr(w_up, torch.uint8, "w_up"),
                                        _ptr(x, torch.float32, "x"), _ptr(gamma, torch.float32, "gamma"),
                                        float(eps), N, K, _stream(stream)))


def _moe_dims(qs_gate, d_gate, expert_ids, E):
    rows, K = _q4_dims(qs_gate, d_gate)
    if rows % E:
        raise ValueError("the expert stores must hold E*N rows")
    T, topk = expert_ids.shape
    return T, topk, rows // E, K


def moe_q4_gemv(y_gate, y_up, qs_gate, d_gate, qs_up, d_up, x, expert_ids, E: int, dev_status=None,
                stream=None) -> None:
    T, topk, N, K = _moe_dims(qs_gate, d_gate, expert_ids, E)
    if x.numel() != T * K or y_gate.numel() != T * topk * N or y_up.numel() != T * topk * N:
        raise ValueError("x must be [T, K] and outputs [T, topk, N]")
    _check(load().moe_q4_gemv(_ptr(y_gate, torch.float32, "y_gate"), _ptr(y_up, torch.float32, "y_up"),
                              _ptr(qs_gate, torch.uint8, "qs_gate"), _ptr(d_gate, torch.float16, "d_gate"),
                              _ptr(qs_up, torch.uint8, "qs_up"), _ptr(d_up, torch.float16, "d_up"),
                              _ptr(x, torch.float32, "x"), _ptr(expert_ids, torch.int32, "expert_ids"),
                              T, topk, E, N, K, _ptr(dev_status, torch.int32, "dev_status"), _stream(stream)))


def fused_gateup_swiglu_q4k_gemv(y, w_gate, w_up, x, gamma=None, eps: float = 1e-5, stream=None) -> None:
    """y = silu(W_gate xhat) * (W_up xhat), one output (xhat as fused_gateup_q4k_gemv)."""
    N, K = _q4k_dims(w_gate)
    if _q4k_dims(w_up) != (N, K) or x.numel() != K or y.numel() != N:
        raise ValueError("w_gate and w_up must be [N, K/256, 144], x [K], y [N]")
    _check(load().fused_gateup_swiglu_q4k_gemv(_ptr(y, torch.float32, "y"), _ptr(w_gate, torch.uint8, "w_gate"),
                                               _ptr(w_up, torch.uint8, "w_up"), _ptr(x, torch.float32, "x"),
                                               _ptr(gamma, torch.float32, "gamma"), float(eps), N, K, _stream(stream)))


def moe_q4_swiglu_gemv(y, qs_gate, d_gate, qs_up, d_up, x, expert_ids, E: int, dev_status=None, stream=None) -> None:
    """y[t, s] = silu(gate) * up for every routed row (routing as moe_q4_gemv)."""
    T, topk, N, K = _moe_dims(qs_gate, d_gate, expert_ids, E)
    if x.numel() != T * K or y.numel() != T * topk * N:
        raise ValueError("x must be [T, K] and y [T, topk, N]")
    _check(load().moe_q4_swiglu_gemv(_ptr(y, torch.float32, "y"), _ptr(qs_gate, torch.uint8, "qs_gate"),
                                     _ptr(d_gate, torch.float16, "d_gate"), _ptr(qs_up, torch.uint8, "qs_up"),
                                     _ptr(d_up, torch.float16, "d_up"), _ptr(x, torch.float32, "x"),
                                     _ptr(expert_ids, torch.int32, "expert_ids"), T, topk, E, N, K,
                                     _ptr(dev_status, torch.int32, "dev_status"), _stream(stream)))


def moe_router_q4(expert_ids, expert_weights, qs, d, x, topk: int, normalize: bool = True, logits=None,
                  stream=None) -> None:
    """Router logits of E planar-Q4 rows for T tokens, then the top-K experts and their softmax weights."""
    E, K = _q4_dims(qs, d)
    T = x.numel() // K
    if x.numel() != T * K or expert_ids.numel() != T * topk or expert_weights.numel() != T * topk:
        raise ValueError("x must be [T, K], expert_ids and expert_weights [T, topk]")
    if logits is not None and logits.numel() != T * E:
        raise ValueError("logits must be [T, E]")
    _check(load().moe_router_q4(_ptr(expert_ids, torch.int32, "expert_ids"),
                                _ptr(expert_weights, torch.float32, "expert_weights"),
                                _ptr(logits, torch.float32, "logits"), _ptr(qs, torch.uint8, "qs"),
                                _ptr(d, torch.float16, "d"), _ptr(x, torch.float32, "x"), T, E, K, topk,
                                1 if normalize else 0, _stream(stream)))


def q4_pure_read(sink, qs, d, stream=None) -> None:
    N, K = _q4_dims(qs, d)
    _check(load().q4_pure_read(_ptr(sink, torch.float32, "sink"), _ptr(qs, torch.uint8, "qs"),
                               _ptr(d, torch.float16, "d"), N, K, _stream(stream)))


def q4_fma_ceiling(sink, fmas: int, mul: float = 1.0 - 2.0 ** -20, add: float = 2.0 ** -20, stream=None) -> int:
    """Run at least `fmas` fp32 FMAs with no loads (the FMA-ceiling instrument); returns the count run."""
    done = ctypes.c_longlong(0)
    _check(load().q4_fma_ceiling(_ptr(sink, torch.float32, "sink"), sink.numel(), int(fmas), float(mul), float(add),
                                 ctypes.byref(done), _stream(stream)))
    return done.value


def q4k_pure_read(sink, w, stream=None) -> None:
    N, K = _q4k_dims(w)
    _check(load().q4k_pure_read(_ptr(sink, torch.float32, "sink"), _ptr(w, torch.uint8, "w"), N, K,
                                _stream(stream)))


def moe_q4_pure_read(sink_gate, sink_up, qs_gate, d_gate, qs_up, d_up, expert_ids, E: int, dev_status=None,
                     stream=None) -> None:
    T, topk, N, K = _moe_dims(qs_gate, d_gate, expert_ids, E)
    _check(load().moe_q4_pure_read(_ptr(sink_gate, torch.float32, "sink_gate"), _ptr(sink_up, torch.float32, "sink_up"),
                                   _ptr(qs_gate, torch.uint8, "qs_gate"), _ptr(d_gate, torch.float16, "d_gate"),
                                   _ptr(qs_up, torch.uint8, "qs_up"), _ptr(d_up, torch.float16, "d_up"),
                                   _ptr(expert_ids, torch.int32, "expert_ids"), T, topk, E, N, K,
                                   _ptr(dev_status, torch.int32, "dev_status"), _stream(stream)))


def q4_dequant(W, qs, d, stream=None) -> None:
    N, K = _q4_dims(qs, d)
    if W.numel() != N * K:
        raise ValueError("W must be [N, K]")
    _check(load().q4_dequant(_ptr(W, torch.float32, "W"), _ptr(qs, torch.uint8, "qs"), _ptr(d, torch.float16, "d"),
                             N, K, _stream(stream)))


def q4k_dequant(W, w, stream=None) -> None:
    N, K = _q4k_dims(w)
    if W.numel() != N * K:
        raise ValueError("W must be [N, K]")
    _check(load().q4k_dequant(_ptr(W, torch.float32, "W"), _ptr(w, torch.uint8, "w"), N, K, _stream(stream)))


def q4_set_launch_overlap(enable: bool) -> None:
    """Turn launch overlap (programmatic dependent launch) on or off for every later GEMV/MoE launch.

    While on, the kernel that runs directly before a call in the same stream must not write that call's
    weights; inputs and outputs may depend on it freely (each kernel waits for it before touching them).
    """
    _check(load().q4_set_launch_overlap(1 if enable else 0))


def q4_get_launch_overlap() -> bool:
    return bool(load().q4_get_launch_overlap())


def q4_set_wait_limit(cycles: int) -> None:
    """Set the limit, in SM cycles, of each kernel wait for a weight stage (default DEFAULT_WAIT_LIMIT). A wait
    that runs out makes its warp store NaN rows and record FAULT_WAIT_TIMEOUT; 0 makes every such wait give up at
    once, which exercises that path."""
    _check(load().q4_set_wait_limit(int(cycles)))


def q4_get_wait_limit() -> int:
    return int(load().q4_get_wait_limit())


# ---- between two projections of a decode step: q/k norm and rotation, the 4-bit cache, attention over it ----

_DTYPES = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}


class KV4Cache:
    """A paged key/value cache in planar Q4 (``kv4_cache`` of the header).

    ``k_qs``, ``v_qs`` uint8 ``[num_pages, num_kv_heads, page_size, head_dim/2]`` and ``k_d``, ``v_d`` float16
    ``[num_pages, num_kv_heads, page_size, head_dim/32]``, contiguous on one CUDA device. The object keeps the tensors
    (and the struct that the calls take, made once: its attributes cannot be set) and nothing else; :meth:`allocate` makes
    an empty one, whose rows read as zeros.
    """

    class _Struct(ctypes.Structure):
        _fields_ = [("k_qs", _P), ("k_d", _P), ("v_qs", _P), ("v_d", _P), ("num_pages", _I), ("num_kv_heads", _I),
                    ("page_size", _I), ("head_dim", _I)]

    def __init__(self, k_qs, k_d, v_qs, v_d):
        if k_qs.dim() != 4:
            raise ValueError("k_qs must be [num_pages, num_kv_heads, page_size, head_dim/2]")
        pages, heads, page, half = k_qs.shape
        if v_qs.shape != k_qs.shape or half % 16 or any(tuple(t.shape) != (pages, heads, page, half // 16) for t in (k_d, v_d)):
            raise ValueError("the codes must be [num_pages, num_kv_heads, page_size, head_dim/2] and the scales "
                             "[num_pages, num_kv_heads, page_size, head_dim/32], head_dim a multiple of 32")
        if pages * heads * page > 0x7FFFFFFF:
            raise ValueError("a cache holds at most 2^31 - 1 rows")
        if any(t.device != k_qs.device for t in (k_d, v_qs, v_d)):
            raise ValueError("the cache's tensors must be on one device")
        struct = KV4Cache._Struct(_ptr(k_qs, torch.uint8, "k_qs"), _ptr(k_d, torch.float16, "k_d"),
                                  _ptr(v_qs, torch.uint8, "v_qs"), _ptr(v_d, torch.float16, "v_d"), pages, heads, page, half * 2)
        self.__dict__.update(k_qs=k_qs, k_d=k_d, v_qs=v_qs, v_d=v_d, num_pages=pages, num_kv_heads=heads, page_size=page,
                             head_dim=half * 2, device=k_qs.device, _struct=struct, _ref=ctypes.addressof(struct))

    def __setattr__(self, name, value):
        raise AttributeError(f"{name}: a KV4Cache's tensors and sizes are fixed; make another one")

    @classmethod
    def allocate(cls, num_pages: int, page_size: int, num_kv_heads: int, head_dim: int, device="cuda") -> "KV4Cache":
        shape = (num_pages, num_kv_heads, page_size)
        made = []
        for _ in range(2):
            made.append(torch.full((*shape, head_dim // 2), 0x88, dtype=torch.uint8, device=device))
            made.append(torch.zeros(*shape, head_dim // 32, dtype=torch.float16, device=device))
        return cls(*made)


# These calls take a few microseconds on the device, so the checks below are written to cost the host as little: one
# pass over each tensor's properties, and the stream's handle without a Stream object.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _rows(t: torch.Tensor, width: int, dtype: torch.dtype, dev: int, name: str):
    """(address, elements from one token to the next) of token rows [..., heads, D] on device `dev`, width = heads * D (the
    caller has checked the shape)."""
    if t.dtype is not dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if t.get_device() != dev:
        raise ValueError(f"{name}: expected a tensor on device {dev}, got {t.device}")
    if t.is_contiguous():
        return t.data_ptr(), width
    shape, st = t.shape, t.stride()
    if len(st) == 3 and st[2] == 1 and st[1] == shape[2]:  # columns of a wider tensor
        return t.data_ptr(), st[0]
    if st[-1] != 1 or (shape[-2] > 1 and st[-2] != shape[-1]):
        raise ValueError(f"{name}: a token's heads must be contiguous")
    # token axes must lie evenly: the outer ones follow from the innermost that has more than one token
    step, n = 0, 1
    for size, s in zip(shape[-3::-1], st[-3::-1]):
        if size != 1:
            if n == 1:
                step = s
            elif s != step * n:
                raise ValueError(f"{name}: the token rows must be evenly spaced")
            n *= size
    return t.data_ptr(), step if n > 1 else width


def _flat(t: torch.Tensor, dtype: torch.dtype, dev: int, name: str, numel: int) -> int:
    """Address of a contiguous tensor of `numel` values on device `dev`."""
    if t.dtype is not dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if t.get_device() != dev:
        raise ValueError(f"{name}: expected a tensor on device {dev}, got {t.device}")
    if t.numel() != numel or not t.is_contiguous():
        raise ValueError(f"{name}: expected {numel} contiguous values, got {list(t.shape)}")
    return t.data_ptr()


def _act(t: torch.Tensor, name: str):
    """(C code of the activation type, device index) of a call, from its first activation."""
    code = _DTYPES.get(t.dtype)
    if code is None:
        raise TypeError(f"{name}: expected float32, float16 or bfloat16, got {t.dtype}")
    dev = t.get_device()
    if dev < 0 or not t.is_cuda:
        raise TypeError(f"{name}: expected a CUDA tensor")
    return code, dev


def _stream_on(dev: int, stream) -> int:
    """Handle of the given stream, or of the current stream of device `dev`."""
    if stream is None:
        return _raw_stream(dev) if _raw_stream is not None else torch.cuda.current_stream(dev).cuda_stream
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _call(fn, dev: int, *args) -> None:
    """Call a C entry with the tensors' device current."""
    if dev == _current_device():
        rc = fn(*args)
    else:
        with torch.cuda.device(dev):
            rc = fn(*args)
    if rc:
        _check(rc)


def qk_norm_rope(q_out, k_out, q, k, q_gamma, k_gamma, cos_sin, positions, eps: float = 1e-6, interleaved: bool = False,
                 stream=None) -> None:
    """RMSNorm of every head of q [T, Hq, D] and k [T, Hkv, D] (gamma float32 [D], or None: no norm) and the rotary
    rotation of the first ``cos_sin.shape[1]`` elements by the table row cos_sin[positions[t]] (cos, then sin; None: no
    rotation). The outputs may be the inputs."""
    code, dev = _act(q, "q")
    shape, k_shape, dt = q.shape, k.shape, q.dtype
    if q_out.shape != shape or k_out.shape != k_shape:
        raise ValueError("q_out must be [T, Hq, D] and k_out [T, Hkv, D]")
    try:
        T, Hq, D = shape
        k_T, Hkv, k_D = k_shape
    except ValueError:
        raise ValueError("q must be [T, Hq, D] and k [T, Hkv, D]") from None
    if T != k_T or D != k_D:
        raise ValueError("q must be [T, Hq, D] and k [T, Hkv, D]")
    max_pos = rot = 0
    table = where = None
    if cos_sin is not None:
        max_pos, rot = cos_sin.shape
        table = _flat(cos_sin, torch.float32, dev, "cos_sin", max_pos * rot)
        where = _flat(positions, torch.int32, dev, "positions", T)
    qp, qs = _rows(q, Hq * D, dt, dev, "q")
    kp, ks = _rows(k, Hkv * D, dt, dev, "k")
    qop, qos = _rows(q_out, Hq * D, dt, dev, "q_out")
    kop, kos = _rows(k_out, Hkv * D, dt, dev, "k_out")
    _call(load().qk_norm_rope, dev, qop, kop, qp, kp,
          None if q_gamma is None else _flat(q_gamma, torch.float32, dev, "q_gamma", D),
          None if k_gamma is None else _flat(k_gamma, torch.float32, dev, "k_gamma", D), eps, table, where, T, Hq, Hkv, D, rot,
          max_pos, 1 if interleaved else 0, qs, ks, qos, kos, code, _stream_on(dev, stream))


def kv4_write(cache: KV4Cache, k, v, slots, stream=None) -> None:
    """Quantise k and v [T, num_kv_heads, head_dim] into the cache's slots (int32 [T]; negative: skipped; the others
    distinct)."""
    code, dev = _act(k, "k")
    shape, dt, H, D = k.shape, k.dtype, cache.num_kv_heads, cache.head_dim
    if len(shape) != 3 or shape[1] != H or shape[2] != D or v.shape != shape:
        raise ValueError(f"k and v must be [T, {H}, {D}], got {list(shape)} and {list(v.shape)}")
    if dev != cache.device.index:
        raise ValueError(f"k: expected a tensor on {cache.device}, got {k.device}")
    T = shape[0]
    kp, ks = _rows(k, H * D, dt, dev, "k")
    vp, vs = _rows(v, H * D, dt, dev, "v")
    _call(load().kv4_write, dev, cache._ref, kp, vp, _flat(slots, torch.int32, dev, "slots", T), T, ks, vs, code,
          _stream_on(dev, stream))


def kv4_read(k_out, v_out, cache: KV4Cache, slots, stream=None) -> None:
    """Values of the cache's rows at slots (int32 [T]; negative: the row is left as it is) into k_out and v_out
    [T, num_kv_heads, head_dim] (one of them may be None)."""
    first = v_out if k_out is None else k_out
    if first is None:
        raise ValueError("k_out and v_out cannot both be None")
    code, dev = _act(first, "k_out" if k_out is not None else "v_out")
    shape, dt, H, D = first.shape, first.dtype, cache.num_kv_heads, cache.head_dim
    if len(shape) != 3 or shape[1] != H or shape[2] != D or (v_out is not None and v_out.shape != shape):
        raise ValueError(f"k_out and v_out must be [T, {H}, {D}]")
    if dev != cache.device.index:
        raise ValueError(f"k_out: expected a tensor on {cache.device}, got {first.device}")
    T = shape[0]
    kp, ks = (None, 0) if k_out is None else _rows(k_out, H * D, dt, dev, "k_out")
    vp, vs = (None, 0) if v_out is None else _rows(v_out, H * D, dt, dev, "v_out")
    _call(load().kv4_read, dev, kp, vp, cache._ref, _flat(slots, torch.int32, dev, "slots", T), T, ks, vs, code,
          _stream_on(dev, stream))


def kv4_attention_workspace(q, cache: KV4Cache) -> torch.Tensor:
    """Workspace for kv4_attention calls with q's [..., M, Hq, D] and type over `cache` (any batch and lengths). Calls that
    may run at the same time (other streams, other graphs) need one each."""
    code, dev = _act(q, "q")
    if q.dim() not in (3, 4):
        raise ValueError("q must be [B, M, Hq, D] or [B, Hq, D]")
    M, Hq = (1, q.shape[1]) if q.dim() == 3 else q.shape[1:3]
    need = ctypes.c_size_t(0)
    _call(load().kv4_attention_workspace, dev, ctypes.byref(need), M, Hq, cache.num_kv_heads, cache.head_dim, code)
    return torch.empty(max(16, need.value), dtype=torch.uint8, device=q.device)


def kv4_attention(out, q, cache: KV4Cache, block_table, seq_lens, scale: float | None = None, window: int = 0, lse=None,
                  workspace=None, stream=None) -> None:
    """Attention of the newest M tokens of B sequences over the cache: q and out [B, M, Hq, D] ([B, Hq, D]: M = 1),
    block_table int32 [B, max_pages], seq_lens int32 [B] (the M tokens included), scale None: D ** -0.5, window 0: all
    tokens, lse float32 [B, M, Hq] or None. workspace: from kv4_attention_workspace, kept between calls; None: allocated
    for this call."""
    code, dev = _act(q, "q")
    shape, dt, D = q.shape, q.dtype, cache.head_dim
    if len(shape) == 4:
        B, M, Hq, _ = shape
    elif len(shape) == 3:
        B, Hq, _ = shape
        M = 1
    else:
        raise ValueError("q must be [B, M, Hq, D] or [B, Hq, D]")
    if out.shape != shape or shape[-1] != D:
        raise ValueError(f"q and out must be [B, M, Hq, {D}] or [B, Hq, {D}], got {list(shape)} and {list(out.shape)}")
    if dev != cache.device.index:
        raise ValueError(f"q: expected a tensor on {cache.device}, got {q.device}")
    table_shape = block_table.shape
    if len(table_shape) != 2 or table_shape[0] != B:
        raise ValueError("block_table must be [B, max_pages]")
    qp, qs = _rows(q, Hq * D, dt, dev, "q")
    op, os_ = _rows(out, Hq * D, dt, dev, "out")
    if workspace is None:
        # on the stream that uses it, so that the allocator hands it on only to work behind this call
        s = torch.cuda.current_stream(dev) if stream is None else (
            stream if isinstance(stream, torch.cuda.Stream) else torch.cuda.ExternalStream(int(stream), device=dev))
        with torch.cuda.stream(s):
            workspace = kv4_attention_workspace(q, cache)
    size = workspace.numel()
    _call(load().kv4_attention, dev, op, None if lse is None else _flat(lse, torch.float32, dev, "lse", B * M * Hq), qp,
          cache._ref, _flat(block_table, torch.int32, dev, "block_table", B * table_shape[1]),
          _flat(seq_lens, torch.int32, dev, "seq_lens", B), B, M, Hq, min(table_shape[1], 0x7FFFFFFF), qs, os_,
          D ** -0.5 if scale is None else scale, max(-1, min(window, 0x7FFFFFFF)), code, _flat(workspace, torch.uint8, dev, "workspace", size), size,
          _stream_on(dev, stream))


def q4_device_faults() -> int:
    """Synchronise the device and return (and clear) the fault bits the kernels recorded."""
    out = ctypes.c_uint(0)
    _check(load().q4_device_faults(ctypes.byref(out)))
    return out.value

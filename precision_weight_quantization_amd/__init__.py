"""Python binding of liblpq.so, the gfx950 low-precision weight codec library.

Argument marshalling only: every step of the codecs runs in the HIP kernels
behind the C ABI (include/lpq.h).  PyTorch supplies device memory and the
current stream.  The functions carry the C names; each accepts CUDA (HIP)
tensors, allocates any output that is not passed in, launches on the current
stream and returns the outputs.  BF16 data is a ``torch.bfloat16`` tensor (or
its ``int16``/``uint16`` bit view), E4M3 codes come back as
``torch.float8_e4m3fn``, scale bytes and packed FP4 as ``torch.uint8``.

Every call launches on the device of its tensors or of its table, whichever is
current.  With a ``stream`` argument the MXFP4 calls and the microscaled linear
layer (``lpq_quantize_mxfp8_transposed``, ``lpq_rmsnorm_mxfp8``,
``lpq_rmsnorm_backward``, ``lpq_mx_matmul`` and their like) allocate what they
are not given on that stream, the others on the current one.  The routed layers'
calls (``lpq_route_plan``, ``lpq_route_gather``, ``lpq_route_combine``,
``lpq_mx_matmul_routed``, ``lpq_adapters`` and their like) stand in the module
``routed``, which the first use of one of their names here loads.

If the library has not been built the import fails: there is no fallback.
"""
from __future__ import annotations

import contextlib
import ctypes
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
# LPQ_LIBRARY may name another build of the same library (e.g. one compiled
# with different launch parameters); the default is the in-tree build.
LIB_PATH = os.environ.get("LPQ_LIBRARY") or os.path.join(_PKG, "liblpq.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(f"{LIB_PATH} is missing: build it with `python -c \"import __graft_entry__ as g; g.build()\"`")

_L = ctypes.CDLL(LIB_PATH)

LPQ_OK = 0
STATUS_NAMES = {0: "LPQ_OK", 1: "LPQ_ERR_NULL", 2: "LPQ_ERR_SHAPE", 3: "LPQ_ERR_ALIGN",
                4: "LPQ_ERR_GROUP", 5: "LPQ_ERR_HIP", 6: "LPQ_ERR_ARG"}


class LpqError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        msg = _L.lpq_status_string(status).decode()
        if status == 5:
            msg += f" (hipError {_L.lpq_last_hip_error()})"
        super().__init__(f"{where}: {STATUS_NAMES.get(status, status)}: {msg}")


class lpq_tensor(ctypes.Structure):
    _fields_ = [("src", ctypes.c_void_p), ("dst", ctypes.c_void_p), ("scale", ctypes.c_void_p),
                ("rows", ctypes.c_int64), ("cols", ctypes.c_int64),
                ("group", ctypes.c_int32), ("reserved", ctypes.c_int32)]


assert ctypes.sizeof(lpq_tensor) == 48


class lpq_requant_tensor(ctypes.Structure):
    _fields_ = [("src", ctypes.c_void_p), ("src_scale", ctypes.c_void_p), ("dst", ctypes.c_void_p),
                ("dst_scale", ctypes.c_void_p), ("rows", ctypes.c_int64), ("cols", ctypes.c_int64),
                ("group", ctypes.c_int32), ("reserved", ctypes.c_int32)]


assert ctypes.sizeof(lpq_requant_tensor) == 56

_vp, _i64, _i32, _int = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_int
_tp = ctypes.POINTER(lpq_tensor)
_rp = ctypes.POINTER(lpq_requant_tensor)
_SIG = {
    "lpq_status_string": (ctypes.c_char_p, [_int]),
    "lpq_last_hip_error": (_int, []),
    "lpq_version": (_int, []),
    "lpq_quantize_fp8blk": (_int, [_vp, _i64, _i64, _vp, _vp, _vp]),
    "lpq_dequantize_fp8blk": (_int, [_vp, _vp, _i64, _i64, _vp, _vp]),
    "lpq_quantize_mxfp8": (_int, [_vp, _i64, _i64, _vp, _vp, _vp]),
    "lpq_dequantize_mxfp8": (_int, [_vp, _vp, _i64, _i64, _vp, _vp]),
    "lpq_quantize_mxfp8_floor": (_int, [_vp, _i64, _i64, _vp, _vp, _vp]),
    "lpq_quantize_mxfp8_floor_grouped": (_int, [_tp, _vp, _i32, _vp]),
    "lpq_quantize_mxfp4": (_int, [_vp, _i64, _i64, _vp, _vp, _vp]),
    "lpq_quantize_mxfp4_floor": (_int, [_vp, _i64, _i64, _vp, _vp, _vp]),
    "lpq_dequantize_mxfp4": (_int, [_vp, _vp, _i64, _i64, _vp, _vp]),
    "lpq_mxfp4_qdq": (_int, [_vp, _i64, _i64, _vp, _vp]),
    "lpq_mxfp4_qdq_floor": (_int, [_vp, _i64, _i64, _vp, _vp]),
    "lpq_quantize_mxfp4_grouped": (_int, [_tp, _vp, _i32, _vp]),
    "lpq_quantize_mxfp4_floor_grouped": (_int, [_tp, _vp, _i32, _vp]),
    "lpq_dequantize_mxfp4_grouped": (_int, [_tp, _vp, _i32, _vp]),
    "lpq_mxfp4_qdq_grouped": (_int, [_tp, _vp, _i32, _vp]),
    "lpq_mxfp4_qdq_floor_grouped": (_int, [_tp, _vp, _i32, _vp]),
    "lpq_quantize_mxfp8_transposed": (_int, [_vp, _i64, _i64, _int, _vp, _vp, _vp, _vp, _vp]),
    "lpq_quantize_mxfp4_transposed": (_int, [_vp, _i64, _i64, _int, _vp, _vp, _vp, _vp, _vp]),
    "lpq_rmsnorm": (_int, [_vp, _vp, _vp, ctypes.c_float, _i64, _i64, _vp, _vp, _vp, _vp]),
    "lpq_rmsnorm_mxfp8": (_int, [_vp, _vp, _vp, ctypes.c_float, _i64, _i64, _vp, _vp, _vp, _vp, _vp, _vp]),
    "lpq_rmsnorm_backward_workspace": (_i64, [_i64, _i64]),
    "lpq_rmsnorm_backward": (_int, [_vp, _vp, _vp, _vp, _vp, _i64, _i64, _vp, _vp, _int, _vp, _i64, _vp]),
    "lpq_mx_matmul": (_int, [_vp, _vp, _int, _vp, _vp, _int, _i64, _i64, _i64, _vp, _int, _vp]),
    "lpq_route_capacity": (_i64, [_i64, _i32, _i32]),
    "lpq_route_plan_workspace": (_i64, [_i64, _i32]),
    "lpq_route_plan": (_int, [_vp, _int, _i64, _i32, _i32, _vp, _vp, _vp, _i64, _vp, _i64, _vp]),
    "lpq_route_gather": (_int, [_vp, _i64, _i64, _vp, _i64, _vp, _i64, _vp, _vp]),
    "lpq_route_gather_mxfp8": (_int, [_vp, _i64, _i64, _vp, _i64, _vp, _i64, _vp, _vp, _vp]),
    "lpq_route_gather_mxfp4": (_int, [_vp, _i64, _i64, _vp, _i64, _vp, _i64, _vp, _vp, _vp]),
    "lpq_route_combine": (_int, [_vp, _i64, _i64, _vp, _i64, _i64, _vp, _vp, _vp, _vp]),
    "lpq_route_combine_backward": (_int, [_vp, _vp, _i64, _i64, _vp, _vp, _i64, _i64, _vp, _vp, _vp, _vp]),
    "lpq_mx_matmul_routed": (_int, [_vp, _vp, _int, _vp, _vp, _int, _vp, _i32, _i64, _i64, _i64, _vp, _int, _vp]),
    "lpq_mx_matmul_routed_dw": (_int, [_vp, _vp, _int, _vp, _vp, _int, _vp, _i32, _i64, _i64, _i64, _vp, _int, _vp]),
    "lpq_adapters_workspace": (_i64, [_i64, _i64, _i32, _i32, _i64, _i64]),
    "lpq_adapters": (_int, [*[_vp] * 7, _i64, _i64, _i32, _i32, _i64, _i64, _vp, _vp, _vp, _i64, _vp]),
    "lpq_adapters_backward_workspace": (_i64, [_i64, _i64, _i32, _i32, _i64, _i64]),
    "lpq_adapters_backward": (_int, [*[_vp] * 8, _i64, _i64, _i32, _i32, _i64, _i64, _vp, _vp, _vp, _vp, _int, _vp, _i64, _vp]),
    "lpq_nvfp4_global_scale_reciprocal": (_int, [_vp, _i32, _vp, _vp]),
    "lpq_nvfp4_global_scale": (_int, [_vp, _i32, _vp, _vp]),
    "lpq_quantize_nvfp4_ex": (_int, [_vp, _i64, _i64, _vp, _int, _vp, _vp, _vp, _vp]),
    "lpq_nvfp4_qdq_ex": (_int, [_vp, _i64, _i64, _vp, _int, _vp, _vp]),
    "lpq_quantize_nvfp4_grouped_ex": (_int, [_tp, _vp, _i32, _vp, _i32, _int, _int, _vp, _vp]),
    "lpq_nvfp4_qdq_grouped_ex": (_int, [_tp, _vp, _i32, _vp, _i32, _int, _int, _vp]),
    "lpq_observer_reset": (_int, [_vp, _vp]),
    "lpq_nvfp4_observe": (_int, [_vp, _i64, _i64, _int, ctypes.c_float, _vp, _vp, _vp]),
    "lpq_nvfp4_observe_noalloc": (_int, [_vp, _i64, _i64, _int, ctypes.c_float, _vp, _vp, _vp]),
    "lpq_nvfp4_amax": (_int, [_vp, _i64, _i64, _vp, _int, _vp]),
    "lpq_quantize_nvfp4": (_int, [_vp, _i64, _i64, _vp, _vp, _vp, _vp, _vp]),
    "lpq_dequantize_nvfp4": (_int, [_vp, _vp, _vp, _i64, _i64, _vp, _vp]),
    "lpq_nvfp4_qdq": (_int, [_vp, _i64, _i64, _vp, _vp, _vp]),
    "lpq_quantize_fp8blk_grouped": (_int, [_tp, _vp, _i32, _vp]),
    "lpq_dequantize_fp8blk_grouped": (_int, [_tp, _vp, _i32, _vp]),
    "lpq_quantize_mxfp8_grouped": (_int, [_tp, _vp, _i32, _vp]),
    "lpq_dequantize_mxfp8_grouped": (_int, [_tp, _vp, _i32, _vp]),
    "lpq_nvfp4_amax_grouped": (_int, [_tp, _vp, _i32, _vp, _i32, _int, _vp]),
    "lpq_quantize_nvfp4_grouped": (_int, [_tp, _vp, _i32, _vp, _i32, _int, _vp, _vp]),
    "lpq_dequantize_nvfp4_grouped": (_int, [_tp, _vp, _i32, _vp, _i32, _vp]),
    "lpq_nvfp4_qdq_grouped": (_int, [_tp, _vp, _i32, _vp, _i32, _int, _vp]),
    "lpq_requantize_fp8blk": (_int, [_vp, _vp, _i64, _i64, _vp, _vp, _vp]),
    "lpq_requantize_fp8blk_grouped": (_int, [_rp, _vp, _i32, _vp]),
    "lpq_requantize_fp8blk_mxfp8": (_int, [_vp, _vp, _i64, _i64, _vp, _vp, _vp]),
    "lpq_fp8blk_amax": (_int, [_vp, _vp, _i64, _i64, _vp, _int, _vp]),
    "lpq_requantize_fp8blk_nvfp4": (_int, [_vp, _vp, _i64, _i64, _vp, _vp, _vp, _vp, _vp]),
    "lpq_requantize_fp8blk_mxfp8_grouped": (_int, [_rp, _vp, _i32, _vp]),
    "lpq_fp8blk_amax_grouped": (_int, [_rp, _vp, _i32, _vp, _i32, _int, _vp]),
    "lpq_requantize_fp8blk_nvfp4_grouped": (_int, [_rp, _vp, _i32, _vp, _i32, _vp, _vp]),
    "lpq_quantize_int4": (_int, [_vp, _i64, _i64, _i32, _vp, _vp, _vp]),
    "lpq_dequantize_int4": (_int, [_vp, _vp, _i64, _i64, _i32, _vp, _vp]),
    "lpq_int4_qdq": (_int, [_vp, _i64, _i64, _i32, _vp, _vp]),
    "lpq_quantize_int4_grouped": (_int, [_tp, _vp, _i32, _i32, _vp]),
    "lpq_dequantize_int4_grouped": (_int, [_tp, _vp, _i32, _i32, _vp]),
    "lpq_int4_qdq_grouped": (_int, [_tp, _vp, _i32, _i32, _vp]),
}
for _name, (_res, _args) in _SIG.items():
    _fn = getattr(_L, _name)
    _fn.restype = _res
    _fn.argtypes = _args

EXPORTED = sorted(k for k in _SIG)


def _current(index: int) -> int:
    """The handle of the device's current stream, without a Stream object around it where torch offers that."""
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    return raw(index) if raw is not None else torch.cuda.current_stream(index).cuda_stream


def _stream(stream, index: int) -> int:
    if stream is None:
        return _current(index)
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _launch(fn, where: str, like, stream, *args) -> None:
    """Call ``fn(*args, stream)`` with the device of ``like`` (the call's data or table)
    current, on the given stream or that device's current one."""
    index = like.device.index
    if index == torch.cuda.current_device():
        status = fn(*args, _stream(stream, index))
    else:
        with torch.cuda.device(index):
            status = fn(*args, _stream(stream, index))
    if status != LPQ_OK:
        raise LpqError(status, where)


_HERE = contextlib.nullcontext()


def _on(stream, like):
    """Where a call allocates what it is not given: on the stream that it launches on, so
    that the memory's earlier users are ordered before it and its later ones behind it.
    A handle is a stream of the device of ``like``."""
    if stream is None:
        return _HERE
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(getattr(stream, "cuda_stream", stream)), device=like.device)
    return torch.cuda.stream(stream)


def _ptr(t) -> int:
    return 0 if t is None else t.data_ptr()


_BF16 = (torch.bfloat16, torch.int16, torch.uint16)


def _arg(t, name: str, like=None, nbytes: int = 0, esize=None, dtypes=None, dims=None):
    """Check a tensor argument before its address reaches a kernel: a device
    tensor, on the device of ``like`` (the call's data), contiguous, of the
    given element size or dtypes and rank, holding at least ``nbytes`` bytes.
    Raises TypeError or ValueError; nothing has been launched then."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor, got {type(t).__name__}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor, got one on {t.device}")
    if like is not None and t.device != like.device:
        raise ValueError(f"{name} is on {t.device}, the call's data on {like.device}")
    if dtypes is not None and t.dtype not in dtypes:
        raise TypeError(f"{name} must be one of {[str(d) for d in dtypes]}, got {t.dtype}")
    if esize is not None and t.element_size() != esize:
        raise TypeError(f"{name} must have {esize}-byte elements, got {t.dtype}")
    if dims is not None and t.dim() != dims:
        raise ValueError(f"{name} must be {dims}-D, got shape {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    have = t.numel() * t.element_size()
    if have < nbytes:
        raise ValueError(f"{name} holds {have} bytes; the call accesses {nbytes}")
    return t


def _bf16_in(x, name: str):
    """A BF16 [M, N] device tensor (or its 16-bit integer view)."""
    return _arg(x, name, dtypes=_BF16, dims=2)


def _out(t, name: str, like, nbytes: int, shape, dtype, esize):
    """A caller-supplied output, checked; or a new one of ``shape`` and ``dtype``."""
    if t is None:
        return torch.empty(shape, dtype=dtype, device=like.device)
    return _arg(t, name, like, nbytes, esize=esize)


def _outs(like, *specs):
    """Several outputs, each (tensor or None, name, nbytes, shape, dtype, esize):
    every tensor the caller gave is checked before any missing one is allocated."""
    for t, name, nbytes, _, _, esize in specs:
        if t is not None:
            _arg(t, name, like, nbytes, esize=esize)
    return [t if t is not None else torch.empty(shape, dtype=dtype, device=like.device)
            for t, _, _, shape, dtype, _ in specs]


def _f32_words(t, name: str, like, n: int = 1):
    """``n`` FP32 words on the device (an amax, a global scale, ...)."""
    return _arg(t, name, like, 4 * n, dtypes=(torch.float32,))


def _empty(shape, dtype, like: torch.Tensor) -> torch.Tensor:
    return torch.empty(shape, dtype=dtype, device=like.device)


def _tiles(M: int, N: int) -> int:
    return ((M + 127) // 128) * ((N + 127) // 128)


# --------------------------------------------------------------------------- block-wise FP8

def fp8blk_scale_shape(M: int, N: int):
    return ((M + 127) // 128, (N + 127) // 128)


def _codes_in(q, name: str):
    """A 2-D device tensor of 1-byte codes (E4M3 or packed FP4/INT4)."""
    return _arg(q, name, esize=1, dims=2)


def lpq_quantize_fp8blk(w, q=None, s=None, stream=None):
    """BF16 [M,N] -> (codes [M,N] float8_e4m3fn, FP32 tile scales [ceil(M/128), ceil(N/128)])."""
    w = _bf16_in(w, "w")
    M, N = w.shape
    q, s = _outs(w, (q, "q", M * N, (M, N), torch.float8_e4m3fn, 1),
                 (s, "s", 4 * _tiles(M, N), fp8blk_scale_shape(M, N), torch.float32, 4))
    _launch(_L.lpq_quantize_fp8blk, "lpq_quantize_fp8blk", w, stream, w.data_ptr(), M, N, q.data_ptr(), s.data_ptr())
    return q, s


def lpq_dequantize_fp8blk(q, s, y=None, stream=None):
    q = _codes_in(q, "q")
    M, N = q.shape
    _arg(s, "s", q, 4 * _tiles(M, N), esize=4)
    y = _out(y, "y", q, 2 * M * N, (M, N), torch.bfloat16, 2)
    _launch(_L.lpq_dequantize_fp8blk, "lpq_dequantize_fp8blk", q, stream, q.data_ptr(), s.data_ptr(), M, N,
            y.data_ptr())
    return y


# --------------------------------------------------------------------------- MXFP8

def _mxfp8_quantize(fn, where, w, q, e, stream):
    w = _bf16_in(w, "w")
    M, N = w.shape
    q, e = _outs(w, (q, "q", M * N, (M, N), torch.float8_e4m3fn, 1),
                 (e, "e", M * (N // 32), (M, max(N // 32, 1)), torch.uint8, 1))
    _launch(fn, where, w, stream, w.data_ptr(), M, N, q.data_ptr(), e.data_ptr())
    return q, e


def lpq_quantize_mxfp8(w, q=None, e=None, stream=None):
    """BF16 [M,N] (N % 32 == 0) -> (codes [M,N] float8_e4m3fn, UE8M0 bytes [M,N/32] uint8)."""
    return _mxfp8_quantize(_L.lpq_quantize_mxfp8, "lpq_quantize_mxfp8", w, q, e, stream)


def lpq_quantize_mxfp8_floor(w, q=None, e=None, stream=None):
    """As lpq_quantize_mxfp8, with the OCP MX floor exponent rule (saturating)."""
    return _mxfp8_quantize(_L.lpq_quantize_mxfp8_floor, "lpq_quantize_mxfp8_floor", w, q, e, stream)


def lpq_dequantize_mxfp8(q, e, y=None, stream=None):
    q = _codes_in(q, "q")
    M, N = q.shape
    _arg(e, "e", q, M * (N // 32), esize=1)
    y = _out(y, "y", q, 2 * M * N, (M, N), torch.bfloat16, 2)
    _launch(_L.lpq_dequantize_mxfp8, "lpq_dequantize_mxfp8", q, stream, q.data_ptr(), e.data_ptr(), M, N, y.data_ptr())
    return y


# --------------------------------------------------------------------------- MXFP4

def _mxfp4_quantize(fn, where, w, p, e, stream):
    w = _bf16_in(w, "w")
    M, N = w.shape
    with _on(stream, w):
        p, e = _outs(w, (p, "p", M * (N // 2), (M, max(N // 2, 1)), torch.uint8, 1),
                     (e, "e", M * (N // 32), (M, max(N // 32, 1)), torch.uint8, 1))
    _launch(fn, where, w, stream, w.data_ptr(), M, N, p.data_ptr(), e.data_ptr())
    return p, e


def lpq_quantize_mxfp4(w, p=None, e=None, stream=None):
    """BF16 [M,N] (N % 32 == 0) -> (packed E2M1 codes [M,N/2] uint8, UE8M0 bytes [M,N/32] uint8)."""
    return _mxfp4_quantize(_L.lpq_quantize_mxfp4, "lpq_quantize_mxfp4", w, p, e, stream)


def lpq_quantize_mxfp4_floor(w, p=None, e=None, stream=None):
    """As lpq_quantize_mxfp4, with the OCP MX floor exponent rule (saturating)."""
    return _mxfp4_quantize(_L.lpq_quantize_mxfp4_floor, "lpq_quantize_mxfp4_floor", w, p, e, stream)


def lpq_dequantize_mxfp4(p, e, y=None, stream=None):
    """(packed [M,N/2], UE8M0 bytes [M,N/32]) -> BF16 [M,N]."""
    p = _codes_in(p, "p")
    M, N = p.shape[0], p.shape[1] * 2
    _arg(e, "e", p, M * (N // 32), esize=1)
    with _on(stream, p):
        y = _out(y, "y", p, 2 * M * N, (M, N), torch.bfloat16, 2)
    _launch(_L.lpq_dequantize_mxfp4, "lpq_dequantize_mxfp4", p, stream, p.data_ptr(), e.data_ptr(), M, N, y.data_ptr())
    return y


def _mxfp4_qdq(fn, where, x, y, stream):
    x = _bf16_in(x, "x")
    M, N = x.shape
    with _on(stream, x):
        y = _out(y, "y", x, 2 * M * N, (M, N), torch.bfloat16, 2)
    _launch(fn, where, x, stream, x.data_ptr(), M, N, y.data_ptr())
    return y


def lpq_mxfp4_qdq(x, y=None, stream=None):
    """MXFP4 fake quantization of BF16 [M,N] (a straight-through estimator's forward pass)."""
    return _mxfp4_qdq(_L.lpq_mxfp4_qdq, "lpq_mxfp4_qdq", x, y, stream)


def lpq_mxfp4_qdq_floor(x, y=None, stream=None):
    """As lpq_mxfp4_qdq, with the OCP MX floor exponent rule (saturating)."""
    return _mxfp4_qdq(_L.lpq_mxfp4_qdq_floor, "lpq_mxfp4_qdq_floor", x, y, stream)


# --------------------------------------------------------------------------- two-way MXFP8 / MXFP4

def _mx_transposed(fn, where, per_byte, dtype, w, rows, floor, qt, et, q, e, stream):
    w = _bf16_in(w, "w")
    M, N = w.shape
    Mp = (M + 31) // 32 * 32
    if not rows and (q is not None or e is not None):
        raise ValueError("q and e are outputs of the row form: pass rows=True with them")
    specs = [(qt, "qt", N * Mp // per_byte, (N, Mp // per_byte), dtype, 1),
             (et, "et", N * Mp // 32, (N, Mp // 32), torch.uint8, 1)]
    if rows:
        specs += [(q, "q", M * (N // per_byte), (M, max(N // per_byte, 1)), dtype, 1),
                  (e, "e", M * (N // 32), (M, max(N // 32, 1)), torch.uint8, 1)]
    with _on(stream, w):
        qt, et, q, e = (_outs(w, *specs) + [None, None])[:4]
    _launch(fn, where, w, stream, w.data_ptr(), M, N, int(bool(floor)), _ptr(q), _ptr(e), qt.data_ptr(), et.data_ptr())
    return qt, et, q, e


def lpq_quantize_mxfp8_transposed(w, rows=False, floor=False, qt=None, et=None, q=None, e=None, stream=None):
    """BF16 [M,N] (N % 32 == 0, any M) -> (qt [N,Mp] float8_e4m3fn, et [N,Mp/32] uint8, q, e): the
    MXFP8 form of the transpose, zero-padded to Mp = M rounded up to 32, and with ``rows`` the row
    form of lpq_quantize_mxfp8 from the same read (else None, None).  floor: the OCP MX floor
    exponent rule."""
    return _mx_transposed(_L.lpq_quantize_mxfp8_transposed, "lpq_quantize_mxfp8_transposed", 1, torch.float8_e4m3fn,
                          w, rows, floor, qt, et, q, e, stream)


def lpq_quantize_mxfp4_transposed(w, rows=False, floor=False, qt=None, et=None, q=None, e=None, stream=None):
    """As lpq_quantize_mxfp8_transposed in MXFP4: packed codes qt [N,Mp/2] and q [M,N/2] uint8."""
    return _mx_transposed(_L.lpq_quantize_mxfp4_transposed, "lpq_quantize_mxfp4_transposed", 2, torch.uint8,
                          w, rows, floor, qt, et, q, e, stream)


# --------------------------------------------------------------------------- NVFP4

def lpq_nvfp4_amax(w, amax=None, accumulate=False, stream=None):
    """max |w| into a 1-element FP32 device tensor (max-accumulated when accumulate)."""
    w = _bf16_in(w, "w")
    M, N = w.shape
    amax = _empty((1,), torch.float32, w) if amax is None else _f32_words(amax, "amax", w)
    _launch(_L.lpq_nvfp4_amax, "lpq_nvfp4_amax", w, stream, w.data_ptr(), M, N, amax.data_ptr(), int(bool(accumulate)))
    return amax


def lpq_quantize_nvfp4_ex(w, amax=None, e4m3_max=448, p=None, s=None, g=None, stream=None):
    """BF16 [M,N] (N % 16 == 0) -> (packed [M,N/2] uint8, E4M3 block scales [M,N/16]
    float8_e4m3fn, global scale [1] FP32 = fl(A / (6 * e4m3_max))), e4m3_max 448 or 256.
    amax: 1-element FP32 device tensor holding the group amax A, or None for the
    tensor's own (computed by the call)."""
    w = _bf16_in(w, "w")
    M, N = w.shape
    if amax is not None:
        _f32_words(amax, "amax", w)
    p, s, g = _outs(w, (p, "p", M * (N // 2), (M, max(N // 2, 1)), torch.uint8, 1),
                    (s, "s", M * (N // 16), (M, max(N // 16, 1)), torch.float8_e4m3fn, 1),
                    (g, "g", 4, (1,), torch.float32, 4))
    _launch(_L.lpq_quantize_nvfp4_ex, "lpq_quantize_nvfp4_ex", w, stream, w.data_ptr(), M, N, _ptr(amax), int(e4m3_max),
            p.data_ptr(), s.data_ptr(), g.data_ptr())
    return p, s, g


def lpq_quantize_nvfp4(w, amax=None, p=None, s=None, g=None, stream=None):
    """BF16 [M,N] (N % 16 == 0) with group amax (1-element FP32 device tensor, or None
    for the tensor's own, computed by the call) -> (packed [M,N/2] uint8, E4M3 block
    scales [M,N/16] float8_e4m3fn, global scale [1] FP32)."""
    w = _bf16_in(w, "w")
    M, N = w.shape
    if amax is not None:
        _f32_words(amax, "amax", w)
    p, s, g = _outs(w, (p, "p", M * (N // 2), (M, max(N // 2, 1)), torch.uint8, 1),
                    (s, "s", M * (N // 16), (M, max(N // 16, 1)), torch.float8_e4m3fn, 1),
                    (g, "g", 4, (1,), torch.float32, 4))
    _launch(_L.lpq_quantize_nvfp4, "lpq_quantize_nvfp4", w, stream, w.data_ptr(), M, N, _ptr(amax), p.data_ptr(),
            s.data_ptr(), g.data_ptr())
    return p, s, g


def lpq_nvfp4_qdq_ex(x, amax, e4m3_max=448, y=None, stream=None):
    x = _bf16_in(x, "x")
    M, N = x.shape
    if amax is not None:
        _f32_words(amax, "amax", x)
    y = _out(y, "y", x, 2 * M * N, (M, N), torch.bfloat16, 2)
    _launch(_L.lpq_nvfp4_qdq_ex, "lpq_nvfp4_qdq_ex", x, stream, x.data_ptr(), M, N, _ptr(amax), int(e4m3_max),
            y.data_ptr())
    return y


def lpq_nvfp4_global_scale_reciprocal(group_amax, out=None, stream=None):
    """fl(2688 / A) per group (the reciprocal export form of the global scale)."""
    _f32_words(group_amax, "group_amax", None, group_amax.numel() if isinstance(group_amax, torch.Tensor) else 1)
    out = torch.empty_like(group_amax) if out is None else _f32_words(out, "out", group_amax, group_amax.numel())
    _launch(_L.lpq_nvfp4_global_scale_reciprocal, "lpq_nvfp4_global_scale_reciprocal", group_amax, stream,
            group_amax.data_ptr(), group_amax.numel(), out.data_ptr())
    return out


def lpq_nvfp4_global_scale(amax, out=None, stream=None):
    """fl(A / 2688) per entry (the multiplier form of a global scale)."""
    _f32_words(amax, "amax", None, amax.numel() if isinstance(amax, torch.Tensor) else 1)
    out = torch.empty_like(amax) if out is None else _f32_words(out, "out", amax, amax.numel())
    _launch(_L.lpq_nvfp4_global_scale, "lpq_nvfp4_global_scale", amax, stream, amax.data_ptr(), amax.numel(),
            out.data_ptr())
    return out


# W4A4 activation observers (the C constants of the same names)
OBSERVERS = {"memoryless_minmax": 0, "static_minmax": 1, "minmax": 2}
OBSERVER_STATE_FLOATS = 128


def lpq_observer_reset(state=None, device=None, stream=None):
    """A reset observer state (8 FP32 words on the device; allocated when not given)."""
    if state is None:
        state = torch.empty(OBSERVER_STATE_FLOATS, dtype=torch.float32, device=device or "cuda")
    else:
        _f32_words(state, "state", None, OBSERVER_STATE_FLOATS)
    _launch(_L.lpq_observer_reset, "lpq_observer_reset", state, stream, state.data_ptr())
    return state


def lpq_nvfp4_observe(x, state, observer="static_minmax", averaging_constant=0.01, amax=None, stream=None):
    """Update the observer state with the BF16 batch x; returns the activation amax (1 FP32, device)."""
    x = _bf16_in(x, "x")
    M, N = x.shape
    _f32_words(state, "state", x, OBSERVER_STATE_FLOATS)
    amax = _empty((1,), torch.float32, x) if amax is None else _f32_words(amax, "amax", x)
    kind = OBSERVERS[observer] if isinstance(observer, str) else int(observer)
    _launch(_L.lpq_nvfp4_observe, "lpq_nvfp4_observe", x, stream, x.data_ptr(), M, N, kind, float(averaging_constant),
            state.data_ptr(), amax.data_ptr())
    return amax


def lpq_nvfp4_observe_noalloc(x, state, observer="static_minmax", averaging_constant=0.01, amax=None, stream=None):
    """lpq_nvfp4_observe with the call's control words in a block the library holds on
    the device: ``state`` needs only 3 FP32 words (min, max, batches seen).  Calls
    that overlap on one device race.  Pass ``amax`` (1 FP32 on the device) for a call
    that allocates nothing; without it this wrapper allocates the output."""
    x = _bf16_in(x, "x")
    M, N = x.shape
    _f32_words(state, "state", x, 3)
    amax = _empty((1,), torch.float32, x) if amax is None else _f32_words(amax, "amax", x)
    kind = OBSERVERS[observer] if isinstance(observer, str) else int(observer)
    _launch(_L.lpq_nvfp4_observe_noalloc, "lpq_nvfp4_observe_noalloc", x, stream, x.data_ptr(), M, N, kind,
            float(averaging_constant), state.data_ptr(), amax.data_ptr())
    return amax


def lpq_dequantize_nvfp4(p, s, g, y=None, stream=None):
    p = _codes_in(p, "p")
    M, N = p.shape[0], p.shape[1] * 2
    _arg(s, "s", p, M * (N // 16), esize=1)
    _f32_words(g, "g", p)
    y = _out(y, "y", p, 2 * M * N, (M, N), torch.bfloat16, 2)
    _launch(_L.lpq_dequantize_nvfp4, "lpq_dequantize_nvfp4", p, stream, p.data_ptr(), s.data_ptr(), g.data_ptr(), M, N,
            y.data_ptr())
    return y


def lpq_nvfp4_qdq(x, amax=None, y=None, stream=None):
    """NVFP4 fake quantization of BF16 [M,N] under the group amax (1-element FP32 device
    tensor); returns BF16 [M,N].  amax None: the tensor's own, computed by the library."""
    x = _bf16_in(x, "x")
    M, N = x.shape
    if amax is not None:
        _f32_words(amax, "amax", x)
    y = _out(y, "y", x, 2 * M * N, (M, N), torch.bfloat16, 2)
    _launch(_L.lpq_nvfp4_qdq, "lpq_nvfp4_qdq", x, stream, x.data_ptr(), M, N, _ptr(amax), y.data_ptr())
    return y


# --------------------------------------------------------------------------- INT4, group-wise

INT4_GROUPS = (32, 128)


def _int4_group(group) -> int:
    return max(int(group), 1)


def lpq_quantize_int4(w, group=128, p=None, s=None, stream=None):
    """BF16 [M,N] (N % group == 0) -> (packed two's-complement nibbles [M,N/2] uint8,
    FP32 group scales [M,N/group])."""
    w = _bf16_in(w, "w")
    M, N = w.shape
    G = _int4_group(group)
    p, s = _outs(w, (p, "p", M * (N // 2), (M, max(N // 2, 1)), torch.uint8, 1),
                 (s, "s", 4 * M * (N // G), (M, max(N // G, 1)), torch.float32, 4))
    _launch(_L.lpq_quantize_int4, "lpq_quantize_int4", w, stream, w.data_ptr(), M, N, int(group), p.data_ptr(),
            s.data_ptr())
    return p, s


def lpq_dequantize_int4(p, s, group=128, y=None, stream=None):
    p = _codes_in(p, "p")
    M, N = p.shape[0], p.shape[1] * 2
    _arg(s, "s", p, 4 * M * (N // _int4_group(group)), esize=4)
    y = _out(y, "y", p, 2 * M * N, (M, N), torch.bfloat16, 2)
    _launch(_L.lpq_dequantize_int4, "lpq_dequantize_int4", p, stream, p.data_ptr(), s.data_ptr(), M, N, int(group),
            y.data_ptr())
    return y


def lpq_int4_qdq(x, group=128, y=None, stream=None):
    """INT4 fake quantization (the straight-through estimator's forward pass) of BF16 [M,N]."""
    x = _bf16_in(x, "x")
    M, N = x.shape
    y = _out(y, "y", x, 2 * M * N, (M, N), torch.bfloat16, 2)
    _launch(_L.lpq_int4_qdq, "lpq_int4_qdq", x, stream, x.data_ptr(), M, N, int(group), y.data_ptr())
    return y


# --------------------------------------------------------------------------- root-mean-square norm

def _norm_inputs(x, gamma, residual):
    x = _bf16_in(x, "x")
    M, N = x.shape
    _arg(gamma, "gamma", x, 2 * N, dtypes=_BF16)
    if residual is not None:
        _arg(residual, "residual", x, 2 * M * N, dtypes=_BF16)
    return x, M, N


def lpq_rmsnorm(x, gamma, eps=1e-6, residual=None, h=None, rstd=None, y=None, stream=None):
    """BF16 x [M,N] (N % 32 == 0, N <= 32768), gamma [N] -> (y [M,N] BF16, h [M,N] BF16, rstd [M] FP32):
    the root-mean-square norm of h = x + residual.  Without a residual h is x itself."""
    x, M, N = _norm_inputs(x, gamma, residual)
    if residual is None and h is not None:
        raise ValueError("h is an output of the residual's addition: pass residual with it")
    specs = [(y, "y", 2 * M * N, (M, N), torch.bfloat16, 2), (rstd, "rstd", 4 * M, (M,), torch.float32, 4)]
    if residual is not None:
        specs.append((h, "h", 2 * M * N, (M, N), torch.bfloat16, 2))
    with _on(stream, x):
        y, rstd, h = (_outs(x, *specs) + [None])[:3]
    _launch(_L.lpq_rmsnorm, "lpq_rmsnorm", x, stream, x.data_ptr(), _ptr(residual), gamma.data_ptr(), float(eps), M, N, _ptr(h),
            rstd.data_ptr(), y.data_ptr())
    return y, (x if h is None else h), rstd


def lpq_rmsnorm_mxfp8(x, gamma, eps=1e-6, residual=None, h=None, rstd=None, y=None, q=None, e=None, stream=None):
    """As lpq_rmsnorm, quantized: -> (q [M,N] float8_e4m3fn, e [M,N/32] uint8, h, rstd), the MXFP8 form of y.
    Pass a BF16 tensor ``y`` to have the unquantized result as well."""
    x, M, N = _norm_inputs(x, gamma, residual)
    if residual is None and h is not None:
        raise ValueError("h is an output of the residual's addition: pass residual with it")
    if y is not None:
        _arg(y, "y", x, 2 * M * N, esize=2)
    specs = [(q, "q", M * N, (M, N), torch.float8_e4m3fn, 1), (e, "e", M * (N // 32), (M, max(N // 32, 1)), torch.uint8, 1),
             (rstd, "rstd", 4 * M, (M,), torch.float32, 4)]
    if residual is not None:
        specs.append((h, "h", 2 * M * N, (M, N), torch.bfloat16, 2))
    with _on(stream, x):
        q, e, rstd, h = (_outs(x, *specs) + [None])[:4]
    _launch(_L.lpq_rmsnorm_mxfp8, "lpq_rmsnorm_mxfp8", x, stream, x.data_ptr(), _ptr(residual), gamma.data_ptr(), float(eps),
            M, N, _ptr(h), rstd.data_ptr(), _ptr(y), q.data_ptr(), e.data_ptr())
    return q, e, (x if h is None else h), rstd


def lpq_rmsnorm_backward_workspace(M, N):
    """Bytes of workspace that lpq_rmsnorm_backward needs for dgamma (0 for a shape it refuses)."""
    return int(_L.lpq_rmsnorm_backward_workspace(int(M), int(N)))


def lpq_rmsnorm_backward(dy, h, gamma, rstd, dres=None, dx=None, dgamma=None, accumulate=False, want_dgamma=True,
                         workspace=None, stream=None):
    """Gradients of lpq_rmsnorm (of lpq_rmsnorm_mxfp8 under a straight-through estimator) from its h and rstd:
    (dx [M,N] BF16, of x and of residual alike, with dres [M,N] added; dgamma [N] FP32, None without
    ``want_dgamma``).  accumulate: add to the ``dgamma`` passed in.  workspace: a device tensor of at least
    lpq_rmsnorm_backward_workspace(M, N) bytes, used by one call at a time; allocated when not given."""
    dy = _bf16_in(dy, "dy")
    M, N = dy.shape
    for t, name in ((h, "h"), (dres, "dres")):
        if t is not None or name == "h":
            _arg(t, name, dy, 2 * M * N, dtypes=_BF16)
    _arg(gamma, "gamma", dy, 2 * N, dtypes=_BF16)
    _f32_words(rstd, "rstd", dy, M)
    if accumulate and dgamma is None:
        raise ValueError("accumulate adds to a dgamma that is passed in")
    if dgamma is not None and not want_dgamma:
        raise ValueError("dgamma was passed in, and want_dgamma is False")
    need = lpq_rmsnorm_backward_workspace(M, N) if want_dgamma else 0
    if workspace is not None:
        _arg(workspace, "workspace", dy, need)
    specs = [(dx, "dx", 2 * M * N, (M, N), torch.bfloat16, 2)]
    if want_dgamma:
        specs.append((dgamma, "dgamma", 4 * N, (N,), torch.float32, 4))
    with _on(stream, dy):
        dx, dgamma = (_outs(dy, *specs) + [None])[:2]
        if need and workspace is None:
            workspace = _empty((need,), torch.uint8, dy)
    _launch(_L.lpq_rmsnorm_backward, "lpq_rmsnorm_backward", dy, stream, dy.data_ptr(), h.data_ptr(), gamma.data_ptr(),
            rstd.data_ptr(), _ptr(dres), M, N, dx.data_ptr(), _ptr(dgamma), int(bool(accumulate)), _ptr(workspace),
            0 if workspace is None else workspace.numel() * workspace.element_size())
    return dx, dgamma


# --------------------------------------------------------------------------- microscaled products

MX_FORMATS = {"mxfp8": 0, "mxfp4": 1}
_MX_OUT = {torch.bfloat16: 0, torch.float32: 1}


def _mx_operand(codes, scales, fmt, name, like=None):
    """(format, rows, columns) of a microscaled operand, from its format's name or its codes' dtype."""
    _arg(codes, name, like, esize=1, dims=2)
    if fmt is None:
        if codes.dtype not in (torch.float8_e4m3fn, torch.uint8):
            raise TypeError(f"{name} holds float8_e4m3fn codes (MXFP8) or uint8 (packed MXFP4), got {codes.dtype}")
        fmt = "mxfp8" if codes.dtype == torch.float8_e4m3fn else "mxfp4"
    elif fmt not in MX_FORMATS:
        raise ValueError(f"the format of {name} is one of {sorted(MX_FORMATS)}, got {fmt!r}")
    rows, cols = codes.shape
    cols *= 2 if fmt == "mxfp4" else 1
    _arg(scales, name + "e", codes, rows * (cols // 32), esize=1)
    return MX_FORMATS[fmt], rows, cols


def lpq_mx_matmul(a, ae, b, be, out_dtype=torch.bfloat16, y=None, a_format=None, b_format=None, stream=None):
    """y [M,N] = a b^T of two microscaled matrices: a [M,K] and b [N,K] codes with UE8M0 scale bytes ae
    [M,K/32] and be [N,K/32].  float8_e4m3fn codes are MXFP8, uint8 codes packed MXFP4, unless ``a_format`` /
    ``b_format`` ("mxfp8", "mxfp4") say otherwise.  out_dtype: bfloat16, or float32 when both are MXFP4."""
    fa, M, K = _mx_operand(a, ae, a_format, "a")
    fb, N, Kb = _mx_operand(b, be, b_format, "b", a)
    if K != Kb:
        raise ValueError(f"a has {K} columns, b {Kb}")
    if out_dtype not in _MX_OUT:
        raise TypeError(f"out_dtype must be one of {[str(d) for d in _MX_OUT]}, got {out_dtype}")
    size = 4 if out_dtype == torch.float32 else 2
    with _on(stream, a):
        y = _out(y, "y", a, size * M * N, (M, N), out_dtype, size)
    _launch(_L.lpq_mx_matmul, "lpq_mx_matmul", a, stream, a.data_ptr(), ae.data_ptr(), fa, b.data_ptr(), be.data_ptr(), fb,
            M, N, K, y.data_ptr(), _MX_OUT[out_dtype])
    return y


# --------------------------------------------------------------------------- FP8 re-quantization

def lpq_requantize_fp8blk(q, s, q_out=None, s_out=None, stream=None):
    """Block-wise FP8 (codes [M,N], FP32 tile scales) -> block-wise FP8 of the dequantized
    BF16 values (codes [M,N] float8_e4m3fn, new FP32 tile scales), in one pass."""
    q = _codes_in(q, "q")
    M, N = q.shape
    _arg(s, "s", q, 4 * _tiles(M, N), esize=4)
    q_out, s_out = _outs(q, (q_out, "q_out", M * N, (M, N), torch.float8_e4m3fn, 1),
                         (s_out, "s_out", 4 * _tiles(M, N), fp8blk_scale_shape(M, N), torch.float32, 4))
    _launch(_L.lpq_requantize_fp8blk, "lpq_requantize_fp8blk", q, stream, q.data_ptr(), s.data_ptr(), M, N,
            q_out.data_ptr(), s_out.data_ptr())
    return q_out, s_out


def lpq_requantize_fp8blk_mxfp8(q, s, q_out=None, e_out=None, stream=None):
    """Block-wise FP8 (codes [M,N], FP32 tile scales) -> MXFP8 (codes [M,N] float8_e4m3fn,
    UE8M0 bytes [M,N/32] uint8) of the dequantized BF16 values, in one pass."""
    q = _codes_in(q, "q")
    M, N = q.shape
    _arg(s, "s", q, 4 * _tiles(M, N), esize=4)
    q_out, e_out = _outs(q, (q_out, "q_out", M * N, (M, N), torch.float8_e4m3fn, 1),
                         (e_out, "e_out", M * (N // 32), (M, max(N // 32, 1)), torch.uint8, 1))
    _launch(_L.lpq_requantize_fp8blk_mxfp8, "lpq_requantize_fp8blk_mxfp8", q, stream, q.data_ptr(), s.data_ptr(), M, N,
            q_out.data_ptr(), e_out.data_ptr())
    return q_out, e_out


def lpq_fp8blk_amax(q, s, amax=None, accumulate=False, stream=None):
    """max |y| of the dequantized BF16 values into a 1-element FP32 device tensor."""
    q = _codes_in(q, "q")
    M, N = q.shape
    _arg(s, "s", q, 4 * _tiles(M, N), esize=4)
    amax = _empty((1,), torch.float32, q) if amax is None else _f32_words(amax, "amax", q)
    _launch(_L.lpq_fp8blk_amax, "lpq_fp8blk_amax", q, stream, q.data_ptr(), s.data_ptr(), M, N, amax.data_ptr(),
            int(bool(accumulate)))
    return amax


def lpq_requantize_fp8blk_nvfp4(q, s, amax, p=None, sb=None, g=None, stream=None):
    """Block-wise FP8 -> NVFP4 (packed [M,N/2] uint8, E4M3 block scales [M,N/16], global scale [1])
    of the dequantized BF16 values under the group amax (1-element FP32 device tensor)."""
    q = _codes_in(q, "q")
    M, N = q.shape
    _arg(s, "s", q, 4 * _tiles(M, N), esize=4)
    _f32_words(amax, "amax", q)
    p, sb, g = _outs(q, (p, "p", M * (N // 2), (M, max(N // 2, 1)), torch.uint8, 1),
                     (sb, "sb", M * (N // 16), (M, max(N // 16, 1)), torch.float8_e4m3fn, 1),
                     (g, "g", 4, (1,), torch.float32, 4))
    _launch(_L.lpq_requantize_fp8blk_nvfp4, "lpq_requantize_fp8blk_nvfp4", q, stream, q.data_ptr(), s.data_ptr(), M, N,
            amax.data_ptr(), p.data_ptr(), sb.data_ptr(), g.data_ptr())
    return p, sb, g


# --------------------------------------------------------------------------- grouped

# Bytes each descriptor array of a grouped call accesses, per operation, for a
# tensor of M x N elements: (src, dst, scale) of lpq_tensor, or (src,
# src_scale, dst, dst_scale) of lpq_requant_tensor; None = not accessed.
def _grouped_bytes(op: str, M: int, N: int, G: int = 128):
    MN, t = M * N, 4 * _tiles(M, N)
    return _GROUPED_BYTES[op](MN, t, G)


_GROUPED_BYTES = {
    "fp8blk_q": lambda MN, t, G: (2 * MN, MN, t),
    "fp8blk_dq": lambda MN, t, G: (MN, 2 * MN, t),
    "mxfp8_q": lambda MN, t, G: (2 * MN, MN, MN // 32),
    "mxfp8_dq": lambda MN, t, G: (MN, 2 * MN, MN // 32),
    "mxfp4_q": lambda MN, t, G: (2 * MN, MN // 2, MN // 32),
    "mxfp4_dq": lambda MN, t, G: (MN // 2, 2 * MN, MN // 32),
    "mxfp4_qdq": lambda MN, t, G: (2 * MN, 2 * MN, None),
    "nvfp4_amax": lambda MN, t, G: (2 * MN, None, None),
    "nvfp4_q": lambda MN, t, G: (2 * MN, MN // 2, MN // 16),
    "nvfp4_dq": lambda MN, t, G: (MN // 2, 2 * MN, MN // 16),
    "nvfp4_qdq": lambda MN, t, G: (2 * MN, 2 * MN, None),
    "int4_q": lambda MN, t, G: (2 * MN, MN // 2, 4 * (MN // G)),
    "int4_dq": lambda MN, t, G: (MN // 2, 2 * MN, 4 * (MN // G)),
    "int4_qdq": lambda MN, t, G: (2 * MN, 2 * MN, None),
    "rq_fp8": lambda MN, t, G: (MN, t, MN, t),
    "rq_mx": lambda MN, t, G: (MN, t, MN, MN // 32),
    "rq_amax": lambda MN, t, G: (MN, t, None, None),
    "rq_nv": lambda MN, t, G: (MN, t, MN // 2, MN // 16),
}


class _Table:
    """Descriptors of a grouped call in host memory and, copied once, on the device.

    The device copy is a blocking host-to-device copy: it has completed when the
    constructor returns, so the table serves calls on any stream.  The tensors
    named by the entries must stay alive while the table is used."""

    _CTYPE = None
    _FIELDS = ()

    def __init__(self, entries, device=None):
        n = len(entries)
        if n == 0:
            raise ValueError("a grouped call needs at least one tensor")
        first = entries[0][0]
        _arg(first, f"entry 0 {self._FIELDS[0]}")
        dev = torch.device(device) if device is not None else first.device
        if dev.type == "cuda" and dev.index is None:
            dev = torch.device("cuda", torch.cuda.current_device())
        self.host = (self._CTYPE * n)()
        self.keep = []
        for i, e in enumerate(entries):
            tensors, (rows, cols, group) = e[:-3], e[-3:]
            for name, t in zip(self._FIELDS, tensors):
                if t is not None and (not isinstance(t, torch.Tensor) or not t.is_cuda or t.device != dev
                                      or not t.is_contiguous()):
                    raise ValueError(f"entry {i} {name}: a contiguous tensor on {dev} is required")
            h = self.host[i]
            for name, t in zip(self._FIELDS, tensors):
                setattr(h, name, _ptr(t))
            h.rows, h.cols, h.group, h.reserved = int(rows), int(cols), int(group), 0
            self.keep.append(tuple(tensors))
        raw = torch.frombuffer(bytearray(bytes(self.host)), dtype=torch.uint8)
        self.dev = torch.empty(raw.numel(), dtype=torch.uint8, device=dev)
        self.dev.copy_(raw, non_blocking=False)
        self.device = dev
        self.n = n
        self._checked = set()

    def check(self, op: str, G: int = 128):
        """Raise ValueError unless every tensor an operation accesses is large enough
        (checked once per operation and group size: the entries do not change)."""
        if (op, G) in self._checked:
            return self
        for i, tensors in enumerate(self.keep):
            h = self.host[i]
            for name, t, need in zip(self._FIELDS, tensors, _grouped_bytes(op, h.rows, h.cols, G)):
                if need is None:
                    continue
                if t is None:
                    raise ValueError(f"entry {i}: {op} needs {name}")
                have = t.numel() * t.element_size()
                if have < need:
                    raise ValueError(f"entry {i} {name} holds {have} bytes; {op} accesses {need}")
        self._checked.add((op, G))
        return self

    def args(self):
        return self.host, self.dev.data_ptr(), self.n


class TensorTable(_Table):
    """The n descriptors of a grouped call.  ``entries`` is a list of (src, dst,
    scale, rows, cols, group): device tensors (dst / scale may be None where the
    call ignores them), the logical shape M x N of the BF16 tensor, and the
    NVFP4 sibling group."""

    _CTYPE = lpq_tensor
    _FIELDS = ("src", "dst", "scale")


class RequantTable(_Table):
    """Descriptors of a grouped re-quantization call: ``entries`` is a list of
    (src codes, src tile scales, dst, dst scales, rows, cols, group)."""

    _CTYPE = lpq_requant_tensor
    _FIELDS = ("src", "src_scale", "dst", "dst_scale")


def _group_words(t, name, table, n=None):
    return _f32_words(t, name, table.dev, t.numel() if n is None and isinstance(t, torch.Tensor) else (n or 1))


def lpq_quantize_fp8blk_grouped(table: TensorTable, stream=None):
    _launch(_L.lpq_quantize_fp8blk_grouped, "lpq_quantize_fp8blk_grouped", table, stream,
            *table.check("fp8blk_q").args())


def lpq_dequantize_fp8blk_grouped(table: TensorTable, stream=None):
    _launch(_L.lpq_dequantize_fp8blk_grouped, "lpq_dequantize_fp8blk_grouped", table, stream,
            *table.check("fp8blk_dq").args())


def lpq_quantize_mxfp8_grouped(table: TensorTable, stream=None):
    _launch(_L.lpq_quantize_mxfp8_grouped, "lpq_quantize_mxfp8_grouped", table, stream, *table.check("mxfp8_q").args())


def lpq_quantize_mxfp8_floor_grouped(table: TensorTable, stream=None):
    _launch(_L.lpq_quantize_mxfp8_floor_grouped, "lpq_quantize_mxfp8_floor_grouped", table, stream,
            *table.check("mxfp8_q").args())


def lpq_dequantize_mxfp8_grouped(table: TensorTable, stream=None):
    _launch(_L.lpq_dequantize_mxfp8_grouped, "lpq_dequantize_mxfp8_grouped", table, stream,
            *table.check("mxfp8_dq").args())


def lpq_quantize_mxfp4_grouped(table: TensorTable, stream=None):
    _launch(_L.lpq_quantize_mxfp4_grouped, "lpq_quantize_mxfp4_grouped", table, stream, *table.check("mxfp4_q").args())


def lpq_quantize_mxfp4_floor_grouped(table: TensorTable, stream=None):
    _launch(_L.lpq_quantize_mxfp4_floor_grouped, "lpq_quantize_mxfp4_floor_grouped", table, stream,
            *table.check("mxfp4_q").args())


def lpq_dequantize_mxfp4_grouped(table: TensorTable, stream=None):
    _launch(_L.lpq_dequantize_mxfp4_grouped, "lpq_dequantize_mxfp4_grouped", table, stream,
            *table.check("mxfp4_dq").args())


def lpq_mxfp4_qdq_grouped(table: TensorTable, stream=None):
    _launch(_L.lpq_mxfp4_qdq_grouped, "lpq_mxfp4_qdq_grouped", table, stream, *table.check("mxfp4_qdq").args())


def lpq_mxfp4_qdq_floor_grouped(table: TensorTable, stream=None):
    _launch(_L.lpq_mxfp4_qdq_floor_grouped, "lpq_mxfp4_qdq_floor_grouped", table, stream,
            *table.check("mxfp4_qdq").args())


def lpq_nvfp4_amax_grouped(table: TensorTable, group_amax, accumulate=False, stream=None):
    _group_words(group_amax, "group_amax", table)
    _launch(_L.lpq_nvfp4_amax_grouped, "lpq_nvfp4_amax_grouped", table, stream, *table.check("nvfp4_amax").args(),
            group_amax.data_ptr(), group_amax.numel(), int(bool(accumulate)))
    return group_amax


def lpq_quantize_nvfp4_grouped(table: TensorTable, group_amax, group_g, amax_valid=True, stream=None):
    """amax_valid False: the call fills group_amax (every member's max |w| folded into
    its group's slot) before it encodes."""
    _group_words(group_amax, "group_amax", table)
    _group_words(group_g, "group_g", table, group_amax.numel())
    _launch(_L.lpq_quantize_nvfp4_grouped, "lpq_quantize_nvfp4_grouped", table, stream, *table.check("nvfp4_q").args(),
            group_amax.data_ptr(), group_amax.numel(), int(bool(amax_valid)), group_g.data_ptr())
    return group_g


def lpq_quantize_nvfp4_grouped_ex(table: TensorTable, group_amax, group_g, e4m3_max=448, amax_valid=True,
                                  stream=None):
    _group_words(group_amax, "group_amax", table)
    _group_words(group_g, "group_g", table, group_amax.numel())
    _launch(_L.lpq_quantize_nvfp4_grouped_ex, "lpq_quantize_nvfp4_grouped_ex", table, stream,
            *table.check("nvfp4_q").args(), group_amax.data_ptr(), group_amax.numel(), int(bool(amax_valid)),
            int(e4m3_max), group_g.data_ptr())
    return group_g


def lpq_nvfp4_qdq_grouped_ex(table: TensorTable, group_amax, e4m3_max=448, amax_valid=True, stream=None):
    _group_words(group_amax, "group_amax", table)
    _launch(_L.lpq_nvfp4_qdq_grouped_ex, "lpq_nvfp4_qdq_grouped_ex", table, stream, *table.check("nvfp4_qdq").args(),
            group_amax.data_ptr(), group_amax.numel(), int(bool(amax_valid)), int(e4m3_max))


def lpq_dequantize_nvfp4_grouped(table: TensorTable, group_g, stream=None):
    _group_words(group_g, "group_g", table)
    _launch(_L.lpq_dequantize_nvfp4_grouped, "lpq_dequantize_nvfp4_grouped", table, stream,
            *table.check("nvfp4_dq").args(), group_g.data_ptr(), group_g.numel())


def lpq_nvfp4_qdq_grouped(table: TensorTable, group_amax, amax_valid=True, stream=None):
    """amax_valid False: the call fills group_amax before it encodes."""
    _group_words(group_amax, "group_amax", table)
    _launch(_L.lpq_nvfp4_qdq_grouped, "lpq_nvfp4_qdq_grouped", table, stream, *table.check("nvfp4_qdq").args(),
            group_amax.data_ptr(), group_amax.numel(), int(bool(amax_valid)))


def lpq_quantize_int4_grouped(table: TensorTable, group=128, stream=None):
    _launch(_L.lpq_quantize_int4_grouped, "lpq_quantize_int4_grouped", table, stream,
            *table.check("int4_q", _int4_group(group)).args(), int(group))


def lpq_dequantize_int4_grouped(table: TensorTable, group=128, stream=None):
    _launch(_L.lpq_dequantize_int4_grouped, "lpq_dequantize_int4_grouped", table, stream,
            *table.check("int4_dq", _int4_group(group)).args(), int(group))


def lpq_int4_qdq_grouped(table: TensorTable, group=128, stream=None):
    _launch(_L.lpq_int4_qdq_grouped, "lpq_int4_qdq_grouped", table, stream, *table.check("int4_qdq").args(), int(group))


def lpq_requantize_fp8blk_grouped(table: RequantTable, stream=None):
    _launch(_L.lpq_requantize_fp8blk_grouped, "lpq_requantize_fp8blk_grouped", table, stream,
            *table.check("rq_fp8").args())


def lpq_requantize_fp8blk_mxfp8_grouped(table: RequantTable, stream=None):
    _launch(_L.lpq_requantize_fp8blk_mxfp8_grouped, "lpq_requantize_fp8blk_mxfp8_grouped", table, stream,
            *table.check("rq_mx").args())


def lpq_fp8blk_amax_grouped(table: RequantTable, group_amax, accumulate=False, stream=None):
    _group_words(group_amax, "group_amax", table)
    _launch(_L.lpq_fp8blk_amax_grouped, "lpq_fp8blk_amax_grouped", table, stream, *table.check("rq_amax").args(),
            group_amax.data_ptr(), group_amax.numel(), int(bool(accumulate)))
    return group_amax


def lpq_requantize_fp8blk_nvfp4_grouped(table: RequantTable, group_amax, group_g, stream=None):
    _group_words(group_amax, "group_amax", table)
    _group_words(group_g, "group_g", table, group_amax.numel())
    _launch(_L.lpq_requantize_fp8blk_nvfp4_grouped, "lpq_requantize_fp8blk_nvfp4_grouped", table, stream,
            *table.check("rq_nv").args(), group_amax.data_ptr(), group_amax.numel(), group_g.data_ptr())
    return group_g


def raw():
    """The ctypes handle of liblpq.so (for tests of the C ABI itself)."""
    return _L


# --------------------------------------------------------------------------- routed layers

# The calls of layers whose rows go to different weights (routed.py), found here under their C names.
_ROUTED = ("lpq_route_capacity", "lpq_route_plan", "lpq_route_gather", "lpq_route_gather_mxfp8", "lpq_route_gather_mxfp4",
           "lpq_adapters", "lpq_adapters_backward", "lpq_mx_matmul_routed", "lpq_mx_matmul_routed_dw", "lpq_route_combine", "lpq_route_combine_backward")


_found = {}


def __getattr__(name):
    fn = _found.get(name)
    if fn is None:
        if name not in _ROUTED:
            raise AttributeError(f"module {__name__!r} has no attribute {name!r}")
        from . import routed
        fn = _found[name] = getattr(routed, name)
    return fn


def __dir__():
    return sorted([*globals(), *_ROUTED])

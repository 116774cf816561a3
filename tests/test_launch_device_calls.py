"""Every call of the binding launches on the device of its data, on that device's current
stream or the one given: tensors and tables on device 1 while device 0 is current, the
library and the runtime's queries replaced (CPU)."""
import inspect
import types

import pytest
import torch

import precision_weight_quantization_amd as lpq
from tests.test_abi import _OtherDevice
from tests.test_launch_device import runtime  # noqa: F401  (fixture)


def on1(dtype, *shape):
    return torch.Tensor._make_subclass(_OtherDevice, torch.zeros(shape, dtype=dtype))


BF, U8, F32 = torch.bfloat16, torch.uint8, torch.float32


def table(cls, fields):
    """A table on device 1, without its copy there."""
    t = cls.__new__(cls)
    t.host = (cls._CTYPE * 1)()
    t.host[0].rows, t.host[0].cols = 128, 128
    t.keep = [tuple(on1(U8, 4 * 128 * 128) for _ in range(fields))]
    t.dev, t.device, t.n, t._checked = on1(U8, 64), torch.device("cuda", 1), 1, set()
    return t


T, Q = lambda: table(lpq.TensorTable, 3), lambda: table(lpq.RequantTable, 4)
w, q, p = (lambda: on1(BF, 128, 128)), (lambda: on1(U8, 128, 128)), (lambda: on1(U8, 128, 64))
one, many, b = (lambda: on1(F32, 1)), (lambda: on1(F32, 128)), (lambda: on1(U8, 128, 128))

SINGLE = {
    "lpq_quantize_fp8blk": lambda **k: lpq.lpq_quantize_fp8blk(w(), q(), one(), **k),
    "lpq_dequantize_fp8blk": lambda **k: lpq.lpq_dequantize_fp8blk(q(), one(), w(), **k),
    "lpq_quantize_mxfp8": lambda **k: lpq.lpq_quantize_mxfp8(w(), q(), b(), **k),
    "lpq_quantize_mxfp8_floor": lambda **k: lpq.lpq_quantize_mxfp8_floor(w(), q(), b(), **k),
    "lpq_dequantize_mxfp8": lambda **k: lpq.lpq_dequantize_mxfp8(q(), b(), w(), **k),
    "lpq_quantize_mxfp4": lambda **k: lpq.lpq_quantize_mxfp4(w(), p(), b(), **k),
    "lpq_quantize_mxfp4_floor": lambda **k: lpq.lpq_quantize_mxfp4_floor(w(), p(), b(), **k),
    "lpq_dequantize_mxfp4": lambda **k: lpq.lpq_dequantize_mxfp4(p(), b(), w(), **k),
    "lpq_mxfp4_qdq": lambda **k: lpq.lpq_mxfp4_qdq(w(), w(), **k),
    "lpq_mxfp4_qdq_floor": lambda **k: lpq.lpq_mxfp4_qdq_floor(w(), w(), **k),
    "lpq_quantize_mxfp8_transposed": lambda **k: lpq.lpq_quantize_mxfp8_transposed(w(), True, False, q(), b(), q(), b(), **k),
    "lpq_quantize_mxfp4_transposed": lambda **k: lpq.lpq_quantize_mxfp4_transposed(w(), True, False, p(), b(), p(), b(), **k),
    "lpq_nvfp4_amax": lambda **k: lpq.lpq_nvfp4_amax(w(), one(), **k),
    "lpq_quantize_nvfp4_ex": lambda **k: lpq.lpq_quantize_nvfp4_ex(w(), one(), 448, p(), b(), one(), **k),
    "lpq_quantize_nvfp4": lambda **k: lpq.lpq_quantize_nvfp4(w(), one(), p(), b(), one(), **k),
    "lpq_nvfp4_qdq_ex": lambda **k: lpq.lpq_nvfp4_qdq_ex(w(), one(), 448, w(), **k),
    "lpq_nvfp4_global_scale_reciprocal": lambda **k: lpq.lpq_nvfp4_global_scale_reciprocal(one(), one(), **k),
    "lpq_nvfp4_global_scale": lambda **k: lpq.lpq_nvfp4_global_scale(one(), one(), **k),
    "lpq_dequantize_nvfp4": lambda **k: lpq.lpq_dequantize_nvfp4(p(), b(), one(), w(), **k),
    "lpq_nvfp4_qdq": lambda **k: lpq.lpq_nvfp4_qdq(w(), one(), w(), **k),
    "lpq_observer_reset": lambda **k: lpq.lpq_observer_reset(on1(F32, 128), **k),
    "lpq_nvfp4_observe": lambda **k: lpq.lpq_nvfp4_observe(w(), on1(F32, 128), amax=one(), **k),
    "lpq_nvfp4_observe_noalloc": lambda **k: lpq.lpq_nvfp4_observe_noalloc(w(), on1(F32, 3), amax=one(), **k),
    "lpq_quantize_int4": lambda **k: lpq.lpq_quantize_int4(w(), 128, p(), many(), **k),
    "lpq_dequantize_int4": lambda **k: lpq.lpq_dequantize_int4(p(), many(), 128, w(), **k),
    "lpq_int4_qdq": lambda **k: lpq.lpq_int4_qdq(w(), 128, w(), **k),
    "lpq_rmsnorm": lambda **k: lpq.lpq_rmsnorm(w(), on1(BF, 128), 1e-6, w(), w(), many(), w(), **k),
    "lpq_rmsnorm_mxfp8": lambda **k: lpq.lpq_rmsnorm_mxfp8(w(), on1(BF, 128), 1e-6, w(), w(), many(), w(), q(), b(), **k),
    "lpq_rmsnorm_backward": lambda **k: lpq.lpq_rmsnorm_backward(w(), w(), on1(BF, 128), many(), w(), w(), many(),
                                                                 workspace=on1(U8, 1 << 20), **k),
    "lpq_mx_matmul": lambda **k: lpq.lpq_mx_matmul(p(), b(), p(), b(), y=w(), **k),
    "lpq_requantize_fp8blk": lambda **k: lpq.lpq_requantize_fp8blk(q(), one(), q(), one(), **k),
    "lpq_requantize_fp8blk_mxfp8": lambda **k: lpq.lpq_requantize_fp8blk_mxfp8(q(), one(), q(), b(), **k),
    "lpq_fp8blk_amax": lambda **k: lpq.lpq_fp8blk_amax(q(), one(), one(), **k),
    "lpq_requantize_fp8blk_nvfp4": lambda **k: lpq.lpq_requantize_fp8blk_nvfp4(q(), one(), one(), p(), b(), one(), **k),
}
GROUPED = {
    **{n: (lambda n: lambda **k: getattr(lpq, n)(T(), **k))(n) for n in (
        "lpq_quantize_fp8blk_grouped", "lpq_dequantize_fp8blk_grouped", "lpq_quantize_mxfp8_grouped",
        "lpq_quantize_mxfp8_floor_grouped", "lpq_dequantize_mxfp8_grouped", "lpq_quantize_mxfp4_grouped",
        "lpq_quantize_mxfp4_floor_grouped", "lpq_dequantize_mxfp4_grouped", "lpq_mxfp4_qdq_grouped",
        "lpq_mxfp4_qdq_floor_grouped", "lpq_quantize_int4_grouped", "lpq_dequantize_int4_grouped", "lpq_int4_qdq_grouped")},
    **{n: (lambda n: lambda **k: getattr(lpq, n)(T(), one(), **k))(n) for n in (
        "lpq_nvfp4_amax_grouped", "lpq_dequantize_nvfp4_grouped", "lpq_nvfp4_qdq_grouped", "lpq_nvfp4_qdq_grouped_ex")},
    **{n: (lambda n: lambda **k: getattr(lpq, n)(T(), one(), group_g=one(), **k))(n) for n in (
        "lpq_quantize_nvfp4_grouped", "lpq_quantize_nvfp4_grouped_ex")},
    **{n: (lambda n: lambda **k: getattr(lpq, n)(Q(), **k))(n) for n in (
        "lpq_requantize_fp8blk_grouped", "lpq_requantize_fp8blk_mxfp8_grouped")},
    "lpq_fp8blk_amax_grouped": lambda **k: lpq.lpq_fp8blk_amax_grouped(Q(), one(), **k),
    "lpq_requantize_fp8blk_nvfp4_grouped": lambda **k: lpq.lpq_requantize_fp8blk_nvfp4_grouped(Q(), one(), group_g=one(), **k),
}
CALLS = {**SINGLE, **GROUPED}


def test_every_call_is_listed():
    takes_a_stream = {n for n, f in vars(lpq).items() if n.startswith("lpq_") and inspect.isfunction(f)
                      and "stream" in inspect.signature(f).parameters}
    assert takes_a_stream == set(CALLS)


@pytest.mark.parametrize("name", sorted(CALLS))
def test_follows_its_data(runtime, monkeypatch, name):  # noqa: F811
    seen = []

    class Library:
        def __getattr__(self, fn):
            if fn == "lpq_rmsnorm_backward_workspace":
                return lambda M, N: 1 << 10
            return lambda *args: seen.append((fn, runtime.current, args[-1])) or 0

    monkeypatch.setattr(lpq, "_L", Library())
    CALLS[name]()
    CALLS[name](stream=77)
    assert seen == [(name, 1, 1001), (name, 1, 77)]
    assert runtime.current == 0


def test_a_torch_without_raw_streams(runtime, monkeypatch):  # noqa: F811
    """The current stream's handle comes from the Stream object then."""
    monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream")
    monkeypatch.setattr(torch.cuda, "current_stream", lambda index: types.SimpleNamespace(cuda_stream=2000 + index))
    seen = []
    lpq._launch(lambda *a: seen.append(a) or 0, "fn", types.SimpleNamespace(device=torch.device("cuda", 1)), None)
    assert seen == [(2001,)]

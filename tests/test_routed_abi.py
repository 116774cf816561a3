"""Refusals of the routed layers' calls, and the device that each launches on (CPU)."""
import inspect

import pytest
import torch

import precision_weight_quantization_amd as lpq
from precision_weight_quantization_amd import routed
from tests.test_abi import P, _OtherDevice, fake, lib, recorder  # noqa: F401  (fixtures)
from tests.test_launch_device import runtime  # noqa: F401  (fixture)

Q = [P + (i << 24) for i in range(12)]   # ranges that do not meet


def caller(fn, **ok):
    return lambda **change: fn(*{**ok, **change}.values())


def refusals(call, status, *changes):
    for c in changes:
        assert call(**c) == status, (c, call(**c))


def test_names():
    """Every call of the module is found in the package, and the other way round."""
    mine = {n for n, f in vars(routed).items() if n.startswith("lpq_") and inspect.isfunction(f)}
    assert mine == set(lpq._ROUTED) and mine <= set(dir(lpq))
    assert all(getattr(lpq, n) is getattr(routed, n) for n in mine)
    with pytest.raises(AttributeError):
        lpq.lpq_no_such_call


def test_capacity(lib):
    C = lib.raw().lpq_route_capacity
    assert [C(8, 64, 1), C(8, 64, 32), C(65536, 128, 32), C(5, 2, 7)] == [8, 256, 65536 + 128 * 31, 21]
    assert all(C(*a) == 0 for a in ((0, 4, 1), (-1, 4, 1), (4, 0, 1), (4, 1025, 1), (4, 4, 0), (4, 4, 1025), ((1 << 30) + 1, 4, 1),
                                    (1 << 30, 4, 2)))
    W = lib.raw().lpq_route_plan_workspace
    assert W(4096, 128) == 0 and W(65536, 128) == 4 * 64 * 128 and W(0, 4) == 0 and W(1 << 30, 1024) == 4 * 256 * 1024


def test_plan_refusals(lib):
    call = caller(lib.raw().lpq_route_plan, ids=Q[0], bytes=4, pairs=8192, groups=128, align=32, offsets=Q[1], rows=Q[2], src=Q[3],
                  capacity=8192 + 128 * 31, ws=Q[4], ws_bytes=4 * 8 * 128, stream=None)
    refusals(call, 1, *({k: None} for k in ("ids", "offsets", "rows", "src", "ws")))
    refusals(call, 2, dict(pairs=0), dict(groups=0), dict(groups=1025), dict(align=0), dict(align=1025), dict(capacity=8192 + 128 * 31 - 1),
             dict(capacity=(1 << 30) + 1))
    refusals(call, 3, dict(ids=Q[0] + 2), dict(bytes=8, ids=Q[0] + 4), dict(offsets=Q[1] + 1), dict(rows=Q[2] + 2), dict(src=Q[3] + 2),
             dict(ws=Q[4] + 2))
    refusals(call, 6, dict(bytes=2), dict(ws_bytes=4 * 8 * 128 - 1), dict(rows=Q[0]), dict(offsets=Q[3]), dict(ws=Q[2] + 64))
    assert lib.raw().lpq_last_hip_error() == 0


def test_gather_refusals(lib):
    L = lib.raw()
    ok = dict(x=Q[0], T=64, N=128, rows=Q[1], k=2, src=Q[2], R=128, q=Q[3], e=Q[4], stream=None)
    plain = {k: v for k, v in ok.items() if k != "e"}
    for call, names in ((caller(L.lpq_route_gather, **plain), "x rows src q"), (caller(L.lpq_route_gather_mxfp8, **ok), "x rows src q e"),
                        (caller(L.lpq_route_gather_mxfp4, **ok), "x rows src q e")):
        refusals(call, 1, *({k: None} for k in names.split()))
        refusals(call, 2, dict(T=0), dict(N=0), dict(N=48), dict(k=0), dict(R=0), dict(R=(1 << 30) + 1), dict(T=1 << 30, k=2), dict(N=1 << 31),
                 dict(T=1 << 29, N=4096), dict(R=1 << 29, N=4096))
        refusals(call, 3, dict(x=Q[0] + 8), dict(q=Q[3] + 8), dict(rows=Q[1] + 2), dict(src=Q[2] + 1))
        refusals(call, 6, dict(q=Q[0] + 16), dict(q=Q[2]), dict(q=Q[1]))
    refusals(caller(L.lpq_route_gather_mxfp8, **ok), 6, dict(e=Q[3] + 128))
    assert L.lpq_last_hip_error() == 0


def test_combine_refusals(lib):
    L = lib.raw()
    call = caller(L.lpq_route_combine, y=Q[0], R=128, N=128, rows=Q[1], T=64, k=2, w=Q[2], res=Q[3], out=Q[4], stream=None)
    refusals(call, 1, *({k: None} for k in ("y", "rows", "out")))
    refusals(call, 2, dict(R=0), dict(N=16), dict(T=0), dict(k=0), dict(T=1 << 30), dict(T=1 << 28, N=2048, k=1))
    refusals(call, 3, dict(y=Q[0] + 8), dict(rows=Q[1] + 2), dict(w=Q[2] + 2), dict(res=Q[3] + 8), dict(out=Q[4] + 8))
    refusals(call, 6, dict(out=Q[0]), dict(out=Q[1]), dict(out=Q[2]), dict(out=Q[3] + 16))
    back = caller(L.lpq_route_combine_backward, dout=Q[0], y=Q[1], R=128, N=128, rows=Q[2], src=Q[3], T=64, k=2, w=Q[4], dy=Q[5],
                  dw=Q[6], stream=None)
    refusals(back, 1, *({k: None} for k in ("dout", "y", "rows", "src", "dy")))
    refusals(back, 2, dict(R=0), dict(N=16), dict(T=0), dict(k=0))
    refusals(back, 3, dict(dout=Q[0] + 8), dict(y=Q[1] + 8), dict(rows=Q[2] + 2), dict(src=Q[3] + 2), dict(w=Q[4] + 2), dict(dy=Q[5] + 8),
             dict(dw=Q[6] + 2))
    refusals(back, 6, dict(dy=Q[0]), dict(dy=Q[1]), dict(dw=Q[5]), dict(dw=Q[4]), dict(dy=Q[3]))
    assert L.lpq_last_hip_error() == 0


def test_product_refusals(lib):
    L = lib.raw()
    call = caller(L.lpq_mx_matmul_routed, a=Q[0], ae=Q[1], fa=0, b=Q[2], be=Q[3], fb=1, off=Q[4], groups=3, R=64, N=128, K=256, y=Q[5],
                  type=0, stream=None)
    dw = caller(L.lpq_mx_matmul_routed_dw, a=Q[0], ae=Q[1], fa=0, b=Q[2], be=Q[3], fb=1, off=Q[4], groups=3, M=64, N=128, R=256, y=Q[5],
                type=0, stream=None)
    for f in (call, dw):
        refusals(f, 1, *({k: None} for k in ("a", "ae", "b", "be", "off", "y")))
        refusals(f, 2, dict(groups=0), dict(groups=1025), dict(R=0), dict(N=0), dict(R=(1 << 30) + 32), dict(N=(1 << 30) + 1),
                 dict(R=1 << 28, N=1 << 13))
        refusals(f, 3, dict(a=Q[0] + 8), dict(b=Q[2] + 8), dict(y=Q[5] + 8), dict(off=Q[4] + 2))
        refusals(f, 6, dict(fa=2), dict(fb=-1), dict(type=2), dict(type=1), dict(type=1, fa=1, fb=0), dict(y=Q[0]), dict(y=Q[3]), dict(y=Q[4]))
    refusals(call, 2, dict(K=0), dict(K=48), dict(K=(1 << 30) + 32), dict(N=1 << 15, K=1 << 24), dict(R=1 << 28, K=1 << 13))
    refusals(dw, 2, dict(M=0), dict(M=(1 << 30) + 1), dict(R=48), dict(M=1 << 20, N=1 << 19), dict(M=1 << 28, R=1 << 13))
    assert L.lpq_last_hip_error() == 0


def test_adapter_refusals(lib):
    L = lib.raw()
    dims = dict(T=64, R=64, groups=3, rank=16, N=128, K=256)
    W, WB = L.lpq_adapters_workspace, L.lpq_adapters_backward_workspace
    need, back_need = W(*dims.values()), WB(*dims.values())
    assert need >= 4 * 64 * 16 and back_need >= 2 * 3 * 16 * 384 + 8 * 64 * 16
    bad = [dict(T=0), dict(R=0), dict(groups=0), dict(groups=1025), dict(rank=0), dict(rank=12), dict(rank=136), dict(N=0), dict(N=12), dict(K=0),
           dict(K=20), dict(N=(1 << 18) + 8), dict(K=(1 << 18) + 8), dict(T=(1 << 24) + 1), dict(R=(1 << 24) + 1), dict(T=1 << 23, N=1 << 13)]
    assert all(f(*{**dims, **c}.values()) == 0 for f in (W, WB) for c in bad)
    call = caller(L.lpq_adapters, x=Q[0], A=Q[1], B=Q[2], scale=Q[3], off=Q[4], rows=Q[5], src=Q[6], **dims, base=Q[7], y=Q[8], ws=Q[9],
                  bytes=need, stream=None)
    back = caller(L.lpq_adapters_backward, dy=Q[10], x=Q[0], A=Q[1], B=Q[2], scale=Q[3], off=Q[4], rows=Q[5], src=Q[6], **dims, dres=Q[7],
                  dx=Q[8], dA=Q[9], dB=Q[11], acc=0, ws=P + (12 << 24), bytes=back_need, stream=None)
    refusals(call, 1, *({k: None} for k in ("x", "A", "B", "off", "rows", "src", "y", "ws")))
    refusals(back, 1, *({k: None} for k in ("dy", "x", "A", "B", "off", "rows", "src", "dx", "dA", "dB", "ws")))
    refusals(call, 2, *bad)
    refusals(back, 2, *bad)
    refusals(call, 3, *({k: Q[i] + 8} for k, i in (("x", 0), ("A", 1), ("B", 2), ("base", 7), ("y", 8), ("ws", 9))),
             *({k: Q[i] + 2} for k, i in (("scale", 3), ("off", 4), ("rows", 5), ("src", 6))))
    refusals(back, 3, *({k: Q[i] + 8} for k, i in (("dy", 10), ("x", 0), ("A", 1), ("B", 2), ("dres", 7), ("dx", 8), ("dA", 9), ("dB", 11))),
             dict(ws=P + (12 << 24) + 8))
    refusals(call, 6, dict(bytes=need - 1), dict(y=Q[0]), dict(y=Q[2]), dict(y=Q[7] + 16), dict(ws=Q[8]), dict(ws=Q[4]))
    refusals(back, 6, dict(bytes=back_need - 1), dict(dx=Q[0]), dict(dx=Q[7] + 16), dict(dA=Q[1]), dict(dB=Q[9]), dict(dB=Q[10]), dict(ws=Q[6]))
    assert L.lpq_last_hip_error() == 0


def bf(*s):
    return fake(torch.zeros(s, dtype=torch.bfloat16))


def u8(*s):
    return fake(torch.zeros(s, dtype=torch.uint8))


def f32(*s):
    return fake(torch.zeros(s, dtype=torch.float32))


def i32(*s):
    return fake(torch.zeros(s, dtype=torch.int32))


def refused(cases):
    for exc, call in cases:
        with pytest.raises(exc):
            call()


def test_plan_binding(lib, recorder, monkeypatch):
    monkeypatch.setattr(recorder, "lpq_route_capacity", lambda *a: 8, raising=False)
    refused([(TypeError, lambda: lib.lpq_route_plan(f32(4, 2), 4)), (ValueError, lambda: lib.lpq_route_plan(torch.zeros(4, 2, dtype=torch.int32), 4)),
             (ValueError, lambda: lib.lpq_route_plan(i32(4, 2), 4, offsets=i32(4))), (ValueError, lambda: lib.lpq_route_plan(i32(4, 2), 4, src=i32(7))),
             (ValueError, lambda: lib.lpq_route_plan(i32(4, 2), 4, rows=i32(7))),
             (TypeError, lambda: lib.lpq_route_plan(i32(4, 2), 4, rows=f32(4, 2))), (ValueError, lambda: lib.lpq_route_plan(i32(2, 4).t(), 4))])
    monkeypatch.setattr(recorder, "lpq_route_capacity", lambda *a: 0, raising=False)
    refused([(ValueError, lambda: lib.lpq_route_plan(i32(4, 2), 4000))])
    assert [c for c in recorder.calls if c != "lpq_route_plan_workspace"] == []


def test_route_binding(lib, recorder):
    x, rows, src = bf(4, 64), i32(4, 2), i32(8)
    refused([(ValueError, lambda: lib.lpq_route_gather(x, i32(3, 2), src)), (TypeError, lambda: lib.lpq_route_gather(x, f32(4, 2), src)),
             (TypeError, lambda: lib.lpq_route_gather(f32(4, 64), rows, src)), (TypeError, lambda: lib.lpq_route_gather(x, rows, f32(8))),
             (ValueError, lambda: lib.lpq_route_gather(x, i32(4, 2, 1), src)), (ValueError, lambda: lib.lpq_route_gather(x, rows, src, y=bf(7, 64))),
             (ValueError, lambda: lib.lpq_route_gather_mxfp8(x, rows, src, q=u8(8, 63))),
             (ValueError, lambda: lib.lpq_route_gather_mxfp4(x, rows, src, e=u8(8, 1))),
             (ValueError, lambda: lib.lpq_route_combine(bf(8, 64), rows, f32(4, 1))), (TypeError, lambda: lib.lpq_route_combine(bf(8, 64), rows, bf(4, 2))),
             (ValueError, lambda: lib.lpq_route_combine(bf(8, 64), rows, residual=bf(3, 64))),
             (ValueError, lambda: lib.lpq_route_combine(bf(8, 64), rows, out=bf(4, 63))),
             (ValueError, lambda: lib.lpq_route_combine_backward(x, rows, src)),
             (ValueError, lambda: lib.lpq_route_combine_backward(x, rows, src, y=bf(7, 64))),
             (ValueError, lambda: lib.lpq_route_combine_backward(x, rows, src, dweights=f32(4, 2), want_dweights=False)),
             (ValueError, lambda: lib.lpq_route_combine_backward(x, rows, src, y=bf(8, 64), dy=bf(7, 64)))])
    assert recorder.calls == []


def test_product_binding(lib, recorder):
    f8 = lambda *s: fake(torch.zeros(s, dtype=torch.uint8).view(torch.float8_e4m3fn))
    a, ae, b, be, off = f8(8, 64), u8(8, 2), u8(3, 16, 32), u8(3, 16, 2), i32(4)
    f = lib.lpq_mx_matmul_routed
    refused([(TypeError, lambda: f(bf(8, 64), ae, b, be, off)), (ValueError, lambda: f(a, u8(8, 1), b, be, off)),
             (ValueError, lambda: f(a, ae, u8(16, 32), be, off)), (ValueError, lambda: f(a, ae, b, u8(3, 16, 1), off)),
             (ValueError, lambda: f(a, ae, u8(3, 16, 16), u8(3, 16, 1), off)), (ValueError, lambda: f(a, ae, b, be, i32(3))),
             (TypeError, lambda: f(a, ae, b, be, fake(torch.zeros(4, dtype=torch.int64)))), (ValueError, lambda: f(a, ae, b, be, i32(1))),
             (TypeError, lambda: f(a, ae, b, be, off, out_dtype=torch.float16)), (ValueError, lambda: f(a, ae, b, be, off, y=bf(8, 15))),
             (TypeError, lambda: f(a, ae, b, be, off, y=f32(8, 16))), (ValueError, lambda: f(a, ae, b, be, off, b_format="int4"))])
    a, ae, b, be = f8(16, 64), u8(16, 2), f8(24, 64), u8(24, 2)
    f = lib.lpq_mx_matmul_routed_dw
    refused([(ValueError, lambda: f(a, ae, f8(24, 32), u8(24, 1), off)), (ValueError, lambda: f(a, ae, b, u8(23, 2), off)),
             (ValueError, lambda: f(a, ae, b, be, i32(2, 2))), (ValueError, lambda: f(a, ae, b, be, off, y=bf(3, 16, 23))),
             (TypeError, lambda: f(a, ae, b, be, f32(4)))])
    assert recorder.calls == []


def test_adapter_binding(lib, recorder):
    x, A, B, plan = bf(4, 64), bf(3, 8, 64), bf(3, 16, 8), (i32(4), i32(4), i32(4))
    f = lib.lpq_adapters
    refused([(TypeError, lambda: f(f32(4, 64), A, B, *plan)), (ValueError, lambda: f(x, bf(3, 8, 32), B, *plan)),
             (ValueError, lambda: f(x, A, bf(2, 16, 8), *plan)), (ValueError, lambda: f(x, A, bf(3, 16, 16), *plan)),
             (ValueError, lambda: f(x, bf(8, 64), B, *plan)), (ValueError, lambda: f(x, A, B, i32(5), i32(4), i32(4))),
             (ValueError, lambda: f(x, A, B, i32(4), i32(3), i32(4))), (ValueError, lambda: f(x, A, B, i32(4), i32(4, 2), i32(8))),
             (TypeError, lambda: f(x, A, B, i32(4), i32(4), f32(4))), (ValueError, lambda: f(x, A, B, *plan, scale=f32(2))),
             (TypeError, lambda: f(x, A, B, *plan, scale=bf(3))), (ValueError, lambda: f(x, A, B, *plan, base=bf(4, 15))),
             (ValueError, lambda: f(x, A, B, *plan, y=bf(3, 16)))])
    f = lib.lpq_adapters_backward
    dy = bf(4, 16)
    refused([(ValueError, lambda: f(bf(4, 15), x, A, B, *plan)), (ValueError, lambda: f(dy, x, A, B, *plan, accumulate=True)),
             (ValueError, lambda: f(dy, x, A, B, *plan, dres=bf(4, 63))), (ValueError, lambda: f(dy, x, A, B, *plan, dA=f32(3, 8, 63))),
             (TypeError, lambda: f(dy, x, A, B, *plan, dB=bf(3, 16, 8))), (ValueError, lambda: f(dy, x, A, B, *plan, dx=bf(4, 63)))])
    assert [c for c in recorder.calls if not c.endswith("_workspace")] == []


# ----------------------------------------------------------------------------- device and stream

def on1(dtype, *shape):
    return torch.Tensor._make_subclass(_OtherDevice, torch.zeros(shape, dtype=dtype))


BF, U8, F32, I32 = torch.bfloat16, torch.uint8, torch.float32, torch.int32
x, q, p, e, y = (lambda: on1(BF, 4, 64)), (lambda: on1(U8, 8, 64)), (lambda: on1(U8, 8, 32)), (lambda: on1(U8, 8, 2)), (lambda: on1(BF, 8, 64))
rows, src, weights = (lambda: on1(I32, 4, 2)), (lambda: on1(I32, 8)), (lambda: on1(F32, 4, 2))
AB = lambda: (on1(BF, 4, 8, 64), on1(BF, 4, 64, 8), on1(I32, 5), on1(I32, 4), on1(I32, 4))
CALLS = {
    "lpq_adapters": lambda **k: lpq.lpq_adapters(x(), *AB(), base=x(), y=x(), workspace=on1(U8, 64), **k),
    "lpq_adapters_backward": lambda **k: lpq.lpq_adapters_backward(x(), x(), *AB(), dres=x(), dx=x(), dA=on1(F32, 4, 8, 64),
                                                                   dB=on1(F32, 4, 64, 8), workspace=on1(U8, 64), **k),
    "lpq_route_plan": lambda **k: lpq.lpq_route_plan(rows(), 4, 1, on1(I32, 5), rows(), src(), **k),
    "lpq_route_gather": lambda **k: lpq.lpq_route_gather(x(), rows(), src(), y(), **k),
    "lpq_route_gather_mxfp8": lambda **k: lpq.lpq_route_gather_mxfp8(x(), rows(), src(), q(), e(), **k),
    "lpq_route_gather_mxfp4": lambda **k: lpq.lpq_route_gather_mxfp4(x(), rows(), src(), p(), e(), **k),
    "lpq_mx_matmul_routed": lambda **k: lpq.lpq_mx_matmul_routed(p(), e(), on1(U8, 4, 16, 32), on1(U8, 4, 16, 2), on1(I32, 5),
                                                                 y=on1(BF, 8, 16), **k),
    "lpq_mx_matmul_routed_dw": lambda **k: lpq.lpq_mx_matmul_routed_dw(p(), e(), p(), e(), on1(I32, 5), y=on1(BF, 4, 8, 8), **k),
    "lpq_route_combine": lambda **k: lpq.lpq_route_combine(y(), rows(), weights(), x(), x(), **k),
    "lpq_route_combine_backward": lambda **k: lpq.lpq_route_combine_backward(x(), rows(), src(), weights(), y(), y(), weights(), **k),
}


def test_every_call_is_listed():
    assert {n for n in lpq._ROUTED if "stream" in inspect.signature(getattr(lpq, n)).parameters} == set(CALLS)


@pytest.mark.parametrize("name", sorted(CALLS))
def test_follows_its_data(runtime, monkeypatch, name):  # noqa: F811
    seen = []

    class Library:
        def __getattr__(self, fn):
            if fn == "lpq_route_capacity" or fn.endswith("_workspace"):
                return lambda *args: 8 if fn == "lpq_route_capacity" else 0
            return lambda *args: seen.append((fn, runtime.current, args[-1])) or 0

    monkeypatch.setattr(lpq, "_L", Library())
    CALLS[name]()
    CALLS[name](stream=77)
    assert seen == [(name, 1, 1001), (name, 1, 77)]
    assert runtime.current == 0

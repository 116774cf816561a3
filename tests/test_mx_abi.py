"""Refusals of the microscaled operators: each invalid call returns its status, or
raises in the binding, before anything is enqueued (CPU)."""
import pytest
import torch

from tests.test_abi import P, _table, fake, lib, recorder  # noqa: F401  (fixtures)


def test_mxfp4_validation(lib):
    L = lib.raw()
    for q in (L.lpq_quantize_mxfp4, L.lpq_quantize_mxfp4_floor):
        assert q(None, 4, 32, P, P, None) == 1
        assert q(P, 4, 32, None, P, None) == 1
        assert q(P, 4, 32, P, None, None) == 1
        assert q(P, 0, 32, P, P, None) == 2
        assert q(P, 4, 48, P, P, None) == 2
        assert q(P, 1 << 40, 32, P, P, None) == 2
        assert q(P + 8, 4, 32, P, P, None) == 3
        assert q(P, 4, 32, P + 2, P, None) == 3
    assert L.lpq_dequantize_mxfp4(P, None, 4, 32, P, None) == 1
    assert L.lpq_dequantize_mxfp4(P, P, 4, 33, P, None) == 2
    assert L.lpq_dequantize_mxfp4(P + 2, P, 4, 32, P, None) == 3
    assert L.lpq_dequantize_mxfp4(P, P, 4, 32, P + 8, None) == 3
    for f in (L.lpq_mxfp4_qdq, L.lpq_mxfp4_qdq_floor):
        assert f(P, 4, 32, None, None) == 1
        assert f(P, 4, 16, P, None) == 2
        assert f(P, 4, 32, P + 8, None) == 3
    good = (P, P, P, 8, 64, 0, 0)
    t = _table(lib, [good, (P, P, P, 8, 48, 0, 0)])
    t2 = _table(lib, [good, (P, P, P, 8, 64, 0, 7)])
    for g in (L.lpq_quantize_mxfp4_grouped, L.lpq_quantize_mxfp4_floor_grouped, L.lpq_dequantize_mxfp4_grouped,
              L.lpq_mxfp4_qdq_grouped, L.lpq_mxfp4_qdq_floor_grouped):
        assert g(t, P, 2, None) == 2
        assert g(t2, P, 2, None) == 6
        assert g(t, P, 0, None) == 2
        assert g(None, P, 2, None) == 1
    assert L.lpq_last_hip_error() == 0


def test_mxfp4_binding(lib, recorder):
    bf = lambda *s: fake(torch.zeros(s, dtype=torch.bfloat16))
    u8 = lambda *s: fake(torch.zeros(s, dtype=torch.uint8))
    for exc, call in [
            (ValueError, lambda: lib.lpq_quantize_mxfp4(torch.zeros(4, 64, dtype=torch.bfloat16))),
            (TypeError, lambda: lib.lpq_quantize_mxfp4_floor(fake(torch.zeros(4, 64)))),
            (ValueError, lambda: lib.lpq_quantize_mxfp4(bf(4, 64), p=u8(4, 31))),
            (ValueError, lambda: lib.lpq_quantize_mxfp4(bf(4, 64), e=u8(4, 1))),
            (ValueError, lambda: lib.lpq_dequantize_mxfp4(u8(4, 32), u8(4, 1))),
            (ValueError, lambda: lib.lpq_mxfp4_qdq(bf(4, 64), y=bf(4, 32)))]:
        with pytest.raises(exc):
            call()
    assert recorder.calls == []


def test_transposed_validation(lib):
    L = lib.raw()
    for f, a in ((L.lpq_quantize_mxfp8_transposed, 8), (L.lpq_quantize_mxfp4_transposed, 4)):
        assert f(None, 4, 32, 0, P, P, P, P, None) == 1
        assert f(P, 4, 32, 0, P, P, None, P, None) == 1
        assert f(P, 4, 32, 0, P, P, P, None, None) == 1
        assert f(P, 4, 32, 0, P, None, P, P, None) == 1      # q and e go together
        assert f(P, 4, 32, 0, None, P, P, P, None) == 1
        assert f(P, 0, 32, 0, P, P, P, P, None) == 2
        assert f(P, 4, 48, 0, P, P, P, P, None) == 2
        assert f(P, 1 << 40, 32, 0, P, P, P, P, None) == 2
        assert f(P, 4, 32, 2, P, P, P, P, None) == 6
        assert f(P, 4, 32, -1, P, P, P, P, None) == 6
        assert f(P + 8, 4, 32, 0, P, P, P, P, None) == 3
        assert f(P, 4, 32, 0, P, P, P + 8, P, None) == 3
        assert f(P, 4, 32, 0, P + a // 2, P, P, P, None) == 3
        far = [P + (i << 20) for i in range(1, 5)]
        assert f(P, 4, 32, 0, far[0], far[1], P + 128, far[2], None) == 6          # over w
        assert f(P, 4, 32, 0, far[0], far[1], far[2], far[0] + 4, None) == 6       # one over another
    assert L.lpq_last_hip_error() == 0


def test_transposed_binding(lib, recorder):
    bf = lambda *s: fake(torch.zeros(s, dtype=torch.bfloat16))
    u8 = lambda *s: fake(torch.zeros(s, dtype=torch.uint8))
    for exc, call in [
            (ValueError, lambda: lib.lpq_quantize_mxfp8_transposed(bf(4, 64), qt=u8(64, 31))),   # padded to 32 rows
            (ValueError, lambda: lib.lpq_quantize_mxfp8_transposed(bf(40, 64), et=u8(64, 1))),
            (ValueError, lambda: lib.lpq_quantize_mxfp4_transposed(bf(4, 64), qt=u8(64, 15))),
            (ValueError, lambda: lib.lpq_quantize_mxfp4_transposed(bf(4, 64), rows=True, q=u8(4, 31))),
            (ValueError, lambda: lib.lpq_quantize_mxfp8_transposed(bf(4, 64), q=u8(4, 64))),     # without rows
            (TypeError, lambda: lib.lpq_quantize_mxfp8_transposed(fake(torch.zeros(4, 64))))]:
        with pytest.raises(exc):
            call()
    assert recorder.calls == []


def test_rmsnorm_validation(lib):
    L = lib.raw()
    Q = [P + (i << 24) for i in range(12)]   # ranges that do not meet
    x, res, gm, h, rs, y, q, e = Q[:8]
    f, fq = L.lpq_rmsnorm, L.lpq_rmsnorm_mxfp8
    assert f(None, None, gm, 1e-6, 4, 64, None, rs, y, None) == 1
    assert f(x, None, None, 1e-6, 4, 64, None, rs, y, None) == 1
    assert f(x, None, gm, 1e-6, 4, 64, None, rs, None, None) == 1
    assert f(x, res, gm, 1e-6, 4, 64, None, rs, y, None) == 1            # the sum needs a place
    assert f(x, None, gm, 1e-6, 4, 64, h, rs, y, None) == 6              # h without a residual
    assert f(x, None, gm, 1e-6, 0, 64, None, rs, y, None) == 2
    assert f(x, None, gm, 1e-6, 4, 48, None, rs, y, None) == 2
    assert f(x, None, gm, 1e-6, 4, 32800, None, rs, y, None) == 2
    assert f(x, None, gm, 1e-6, 4, 64 + (1 << 32), None, rs, y, None) == 2
    assert f(x, None, gm, 1e-6, 1 << 40, 64, None, rs, y, None) == 2
    for eps in (0.0, -1e-6, float("inf"), float("nan")):
        assert f(x, None, gm, eps, 4, 64, None, rs, y, None) == 6
    assert f(x + 8, None, gm, 1e-6, 4, 64, None, rs, y, None) == 3
    assert f(x, None, gm + 8, 1e-6, 4, 64, None, rs, y, None) == 3
    assert f(x, res + 2, gm, 1e-6, 4, 64, h, rs, y, None) == 3
    assert f(x, None, gm, 1e-6, 4, 64, None, rs + 2, y, None) == 3
    assert f(x, None, gm, 1e-6, 4, 64, None, rs, x, None) == 6           # y over x
    assert f(x, res, gm, 1e-6, 4, 64, x + 64, rs, y, None) == 6          # h over a part of x
    assert f(x, res, gm, 1e-6, 4, 64, h, rs, h + 16, None) == 6
    assert f(x, None, gm, 1e-6, 4, 64, None, gm, y, None) == 6           # rstd over gamma
    assert fq(x, None, gm, 1e-6, 4, 64, None, rs, None, None, e, None) == 1
    assert fq(x, None, gm, 1e-6, 4, 64, None, rs, None, q, None, None) == 1
    assert fq(x, None, gm, 1e-6, 4, 64, None, rs, None, q + 4, e, None) == 3
    assert fq(x, None, gm, 1e-6, 4, 64, None, rs, None, q, q + 128, None) == 6
    b = L.lpq_rmsnorm_backward
    dy, hh, g2, r2, dr, dx, dg, ws = Q[:8]
    need = L.lpq_rmsnorm_backward_workspace(1000, 64)
    assert need > 0 and need % 256 == 0
    assert L.lpq_rmsnorm_backward_workspace(0, 64) == 0
    assert L.lpq_rmsnorm_backward_workspace(4, 40) == 0
    ok = [dy, hh, g2, r2, dr, 1000, 64, dx, dg, 0, ws, need, None]

    def call(**change):
        a = list(ok)
        for k, v in change.items():
            a["dy h gamma rstd dres M N dx dgamma accumulate ws bytes stream".split().index(k)] = v
        return b(*a)

    for k in ("dy", "h", "gamma", "rstd", "dx", "ws"):
        assert call(**{k: None}) == 1, k
    assert call(M=0) == 2 and call(N=48) == 2 and call(N=40000) == 2
    assert call(bytes=need - 1) == 6
    for k, v in (("dy", dy + 8), ("h", hh + 8), ("gamma", g2 + 2), ("rstd", r2 + 2), ("dres", dr + 8), ("dx", dx + 8),
                 ("dgamma", dg + 2), ("ws", ws + 8)):
        assert call(**{k: v}) == 3, k
    assert call(dx=hh) == 6 and call(dx=dy + 64) == 6 and call(dgamma=ws) == 6 and call(ws=dx + 1024) == 6
    assert L.lpq_last_hip_error() == 0


def test_rmsnorm_binding(lib, recorder):
    bf = lambda *s: fake(torch.zeros(s, dtype=torch.bfloat16))
    u8 = lambda *s: fake(torch.zeros(s, dtype=torch.uint8))
    f32 = lambda *s: fake(torch.zeros(s, dtype=torch.float32))
    x, g = bf(4, 64), bf(64)
    for exc, call in [
            (TypeError, lambda: lib.lpq_rmsnorm(f32(4, 64), g)),
            (ValueError, lambda: lib.lpq_rmsnorm(x, bf(63))),
            (TypeError, lambda: lib.lpq_rmsnorm(x, f32(64))),
            (ValueError, lambda: lib.lpq_rmsnorm(x, g, residual=bf(4, 32))),
            (ValueError, lambda: lib.lpq_rmsnorm(x, g, h=bf(4, 64))),
            (ValueError, lambda: lib.lpq_rmsnorm(x, g, rstd=f32(3))),
            (ValueError, lambda: lib.lpq_rmsnorm_mxfp8(x, g, q=u8(4, 63))),
            (ValueError, lambda: lib.lpq_rmsnorm_mxfp8(x, g, y=bf(4, 63))),
            (ValueError, lambda: lib.lpq_rmsnorm_backward(x, bf(3, 64), g, f32(4))),
            (ValueError, lambda: lib.lpq_rmsnorm_backward(x, x, g, f32(3))),
            (ValueError, lambda: lib.lpq_rmsnorm_backward(x, x, g, f32(4), accumulate=True)),
            (ValueError, lambda: lib.lpq_rmsnorm_backward(x, x, g, f32(4), dgamma=f32(64), want_dgamma=False)),
            (ValueError, lambda: lib.lpq_rmsnorm_backward(x, x, g, f32(4), dgamma=f32(63)))]:
        with pytest.raises(exc):
            call()
    assert [c for c in recorder.calls if c != "lpq_rmsnorm_backward_workspace"] == []


def test_matmul_validation(lib):
    L = lib.raw()
    Q = [P + (i << 24) for i in range(6)]
    ok = dict(a=Q[0], ae=Q[1], fa=0, b=Q[2], be=Q[3], fb=1, M=4, N=16, K=64, y=Q[4], type=0, stream=None)

    def call(**change):
        return L.lpq_mx_matmul(*{**ok, **change}.values())

    for k in ("a", "ae", "b", "be", "y"):
        assert call(**{k: None}) == 1, k
    for k, v in (("M", 0), ("N", -1), ("K", 0), ("K", 48), ("M", 1 << 31), ("N", 1 << 31), ("K", 1 << 31),
                 ("M", (1 << 30) + 1), ("N", (1 << 30) + 1), ("K", (1 << 30) + 32)):
        assert call(**{k: v}) == 2, (k, v)
    assert call(M=1 << 21, N=1 << 21) == 2 and call(M=1 << 21, K=1 << 21) == 2 and call(N=1 << 21, K=1 << 21) == 2
    for k, v in (("fa", 2), ("fb", -1), ("type", 2), ("type", -1)):
        assert call(**{k: v}) == 6, (k, v)
    assert call(type=1) == 6 and call(type=1, fa=1, fb=0) == 6      # FP32 with an E4M3 operand
    for k in ("a", "b", "y"):
        assert call(**{k: ok[k] + 8}) == 3, k
    assert call(y=Q[0] + 16) == 6 and call(y=Q[3]) == 6 and call(y=Q[2]) == 6
    assert L.lpq_last_hip_error() == 0


def test_matmul_binding(lib, recorder):
    u8 = lambda *s: fake(torch.zeros(s, dtype=torch.uint8))
    f8 = lambda *s: fake(torch.zeros(s, dtype=torch.uint8).view(torch.float8_e4m3fn))
    a, ae, b, be = f8(4, 64), u8(4, 2), u8(16, 32), u8(16, 2)
    bf = lambda *s: fake(torch.zeros(s, dtype=torch.bfloat16))
    for exc, call in [
            (TypeError, lambda: lib.lpq_mx_matmul(bf(4, 64), ae, b, be)),
            (TypeError, lambda: lib.lpq_mx_matmul(fake(torch.zeros(4, 64, dtype=torch.int8)), ae, b, be)),
            (ValueError, lambda: lib.lpq_mx_matmul(a, u8(4, 1), b, be)),
            (ValueError, lambda: lib.lpq_mx_matmul(a, ae, b, u8(15, 2))),
            (ValueError, lambda: lib.lpq_mx_matmul(a, ae, u8(16, 16), u8(16, 2))),          # another K
            (ValueError, lambda: lib.lpq_mx_matmul(a, ae, b, be, b_format="nvfp4")),
            (ValueError, lambda: lib.lpq_mx_matmul(a, ae, b, be, b_format="mxfp8")),         # then K differs
            (TypeError, lambda: lib.lpq_mx_matmul(a, ae, b, be, out_dtype=torch.float16)),
            (TypeError, lambda: lib.lpq_mx_matmul(a, ae, b, be, y=fake(torch.zeros(4, 16)))),
            (ValueError, lambda: lib.lpq_mx_matmul(a, ae, b, be, y=bf(4, 15))),
            (ValueError, lambda: lib.lpq_mx_matmul(f8(64, 4).t(), ae, b, be))]:
        with pytest.raises(exc):
            call()
    assert recorder.calls == []


def test_matmul_constants(lib):
    import re
    from tests.test_abi import HEADER
    defs = {k: int(v) for k, v in re.findall(r"#define (LPQ_\w+) (\d+)", open(HEADER).read())}
    assert {k: defs["LPQ_" + k.upper()] for k in lib.MX_FORMATS} == lib.MX_FORMATS
    assert lib._MX_OUT == {torch.bfloat16: defs["LPQ_BF16"], torch.float32: defs["LPQ_F32"]}

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

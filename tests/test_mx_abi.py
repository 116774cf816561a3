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

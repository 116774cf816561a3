"""MXFP4 quantize, dequantize and QDQ, both exponent rules, single and grouped,
bit for bit against a 64-bit reference: seeded weights and activations at sizes
from one block to several workgroups, blocks of zeros and signed zeros, every
finite BF16 pattern alone in a block and beside a larger anchor."""
import numpy as np
import pytest
import torch

from synth import synth
from tests import mx_ref as R
from tests.gpu_util import brute_blocks, host_u8, host_u16, report, to_dev_bf16

pytestmark = pytest.mark.gpu

SHAPES = [(1, 32), (1, 2560), (3, 96), (33, 160), (128, 2048), (129, 1056), (300, 4096), (1000, 2080)]


@pytest.fixture(scope="module")
def lpq():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import precision_weight_quantization_amd as m
    return m


def calls(lpq, floor):
    return (lpq.lpq_quantize_mxfp4_floor, lpq.lpq_mxfp4_qdq_floor) if floor else (lpq.lpq_quantize_mxfp4, lpq.lpq_mxfp4_qdq)


def check(lpq, w_np, floor, tag):
    quantize, qdq = calls(lpq, floor)
    codes, e_ref = R.quantize(R.bf16_to_f64(w_np), R.FP4, floor)
    y_ref = R.f64_to_bf16(R.values(codes, e_ref, R.FP4))
    y_ref = np.where((codes == 8), np.uint16(0x8000), y_ref)   # a negative zero keeps its sign
    w = to_dev_bf16(w_np)
    p, e = quantize(w)
    y = lpq.lpq_dequantize_mxfp4(p, e)
    bad = report(f"{tag} codes", host_u8(p), R.pack(codes)) + report(f"{tag} scales", host_u8(e), e_ref)
    bad += report(f"{tag} dequantized", host_u16(y), y_ref) + report(f"{tag} qdq", host_u16(qdq(w)), y_ref)
    qdq(w, y=w)   # in place
    bad += report(f"{tag} qdq in place", host_u16(w), y_ref)
    assert bad == 0


@pytest.mark.parametrize("floor", [False, True])
@pytest.mark.parametrize("shape", SHAPES)
def test_shapes(lpq, shape, floor):
    check(lpq, synth.generate(900, shape[0], *shape, 0.02, 0.0, 1e-3, 100.0), floor, f"{shape}")


@pytest.mark.parametrize("floor", [False, True])
def test_every_bf16_pattern(lpq, floor):
    check(lpq, brute_blocks(32, 5), floor, "brute")


@pytest.mark.parametrize("floor", [False, True])
def test_zero_blocks(lpq, floor):
    w = synth.generate(901, 0, 8, 128, 0.02, 0.0, 0.0, 1.0)
    w[2] = 0
    w[3, 32:64] = 0x8000
    w[4, ::2] = 0x8000
    check(lpq, w, floor, "zeros")


@pytest.mark.parametrize("floor", [False, True])
def test_grouped(lpq, floor):
    shapes = [(256, 384), (64, 384), (384, 256), (1, 32), (300, 1024), (129, 2048), (129, 2048)]
    w_np = [synth.generate(902, i, M, N, *synth.DIST_MOE) for i, (M, N) in enumerate(shapes)]
    w = [to_dev_bf16(x) for x in w_np]
    p = [torch.empty((M, N // 2), dtype=torch.uint8, device="cuda") for M, N in shapes]
    e = [torch.empty((M, N // 32), dtype=torch.uint8, device="cuda") for M, N in shapes]
    y = [torch.empty((M, N), dtype=torch.bfloat16, device="cuda") for M, N in shapes]
    f = [torch.empty((M, N), dtype=torch.bfloat16, device="cuda") for M, N in shapes]
    T = lpq.TensorTable
    idx = list(enumerate(shapes))
    tq = T([(w[i], p[i], e[i], M, N, 0) for i, (M, N) in idx])
    td = T([(p[i], y[i], e[i], M, N, 0) for i, (M, N) in idx])
    tf = T([(w[i], f[i], None, M, N, 0) for i, (M, N) in idx])
    (lpq.lpq_quantize_mxfp4_floor_grouped if floor else lpq.lpq_quantize_mxfp4_grouped)(tq)
    lpq.lpq_dequantize_mxfp4_grouped(td)
    (lpq.lpq_mxfp4_qdq_floor_grouped if floor else lpq.lpq_mxfp4_qdq_grouped)(tf)
    bad = 0
    for i, _ in idx:
        codes, er = R.quantize(R.bf16_to_f64(w_np[i]), R.FP4, floor)
        yr = np.where(codes == 8, np.uint16(0x8000), R.f64_to_bf16(R.values(codes, er, R.FP4)))
        bad += report(f"{i} codes", host_u8(p[i]), R.pack(codes)) + report(f"{i} scales", host_u8(e[i]), er)
        bad += report(f"{i} dequantized", host_u16(y[i]), yr) + report(f"{i} qdq", host_u16(f[i]), yr)
    assert bad == 0

"""Two-way quantization, bit for bit against the 64-bit reference: the row form of
the matrix and the row form of its zero-padded transpose, both formats and rules,
at sizes that end inside tiles and blocks; nothing is written outside the outputs."""
import numpy as np
import pytest
import torch

from synth import synth
from tests import mx_ref as R
from tests.gpu_util import brute_blocks, host_u8, report, to_dev_bf16

pytestmark = pytest.mark.gpu

SHAPES = [(1, 32), (31, 64), (32, 32), (33, 96), (127, 160), (128, 128), (160, 256), (300, 1056), (1237, 416)]


@pytest.fixture(scope="module")
def lpq():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import precision_weight_quantization_amd as m
    return m


def padded_transpose(v):
    out = np.zeros((v.shape[1], -(-v.shape[0] // 32) * 32))
    out[:, :v.shape[0]] = v.T
    return out


def packed(codes, fmt):
    return R.pack(codes) if fmt == R.FP4 else codes


def check(lpq, w_np, fmt, floor, rows, tag):
    fn = lpq.lpq_quantize_mxfp4_transposed if fmt == R.FP4 else lpq.lpq_quantize_mxfp8_transposed
    v = R.bf16_to_f64(w_np)
    ct, et = R.quantize(padded_transpose(v), fmt, floor)
    want = packed(ct, fmt)
    guard = 256   # bytes behind each output that the call must leave alone
    qt = torch.full((want.size + guard,), 0xA5, dtype=torch.uint8, device="cuda")
    e = torch.full((et.size + guard,), 0xA5, dtype=torch.uint8, device="cuda")
    _, _, q, eb = fn(to_dev_bf16(w_np), rows=rows, floor=floor, qt=qt, et=e)
    bad = report(f"{tag} codes^T", host_u8(qt[:want.size]), want.reshape(-1))
    bad += report(f"{tag} scales^T", host_u8(e[:et.size]), et.reshape(-1))
    bad += int((qt[want.size:] != 0xA5).sum()) + int((e[et.size:] != 0xA5).sum())
    if rows:
        c, er = R.quantize(v, fmt, floor)
        bad += report(f"{tag} codes", host_u8(q), packed(c, fmt)) + report(f"{tag} scales", host_u8(eb), er)
    else:
        assert q is None and eb is None
    assert bad == 0


@pytest.mark.parametrize("rows", [False, True])
@pytest.mark.parametrize("floor", [False, True])
@pytest.mark.parametrize("fmt", [R.FP8, R.FP4])
@pytest.mark.parametrize("shape", SHAPES)
def test_shapes(lpq, shape, fmt, floor, rows):
    check(lpq, synth.generate(910, shape[0], *shape, 1.0, 0.0, 1e-2, 100.0), fmt, floor, rows, f"{shape} {fmt}")


@pytest.mark.parametrize("floor", [False, True])
@pytest.mark.parametrize("fmt", [R.FP8, R.FP4])
def test_every_bf16_pattern_down_the_columns(lpq, fmt, floor):
    blocks = brute_blocks(32, 6)[:: 7]
    w = np.ascontiguousarray(blocks[: blocks.shape[0] // 32 * 32].T)   # [32, many]: one column block per pattern
    check(lpq, w, fmt, floor, False, f"brute {fmt}")

"""The 64-bit references of the microscaled formats against worked values (CPU)."""
import numpy as np

from tests import mx_ref as R


def test_grids():
    assert R.GRID[R.FP4].tolist() == [0, 0.5, 1, 1.5, 2, 3, 4, 6]
    assert R.GRID[R.FP8][1] == 2.0 ** -9 and R.GRID[R.FP8][8] == 2.0 ** -6


def test_ties_go_to_the_even_code():
    u = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.9, -0.0, -0.25])
    assert (R.nearest_code(u, R.FP4) & 7).tolist() == [0, 2, 2, 4, 4, 6, 6, 7, 0, 0]
    assert (R.nearest_code(u, R.FP4) >> 3).tolist()[-2:] == [1, 1]


def test_exponents():
    b = np.zeros((6, 32))
    b[:, 3] = [6.0, 6.0625, 448.0, 450.0, 0.0, 2.0 ** -130]
    assert R.exponents(b, R.FP4, False).tolist() == [0, 1, 7, 7, -127, -127]
    assert R.exponents(b, R.FP4, True).tolist() == [0, 0, 6, 6, -127, -127]
    assert R.exponents(b, R.FP8, False)[2:4].tolist() == [0, 1]
    assert R.exponents(b, R.FP8, True)[2:4].tolist() == [0, 0]


def test_bf16_rounding():
    x = np.array([1.0, 1 + 2.0 ** -8, 1 + 3 * 2.0 ** -8, -3.1415926, 2.0 ** -130, 0.0])
    assert R.bf16_to_f64(R.f64_to_bf16(x)).tolist() == [1.0, 1.0, 1 + 2.0 ** -6, -3.140625, 2.0 ** -130, 0.0]


def test_agrees_with_the_mxfp8_oracle(oracle):
    from oracle import oracle as O
    from synth import synth
    w = synth.generate(77, 0, 40, 96, 1.5, 0.0, 1e-2, 100.0)
    for floor, fn in ((False, O.mxfp8_quantize), (True, O.mxfp8_floor_quantize)):
        q, e = fn(w)
        rq, re = R.quantize(R.bf16_to_f64(w), R.FP8, floor)
        assert np.array_equal(q, rq) and np.array_equal(e, re)

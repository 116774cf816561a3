"""Plain 64-bit references of the microscaled formats, for the tests (numpy).

Values are found by searching the format's table of values, exponents by
comparing with powers of two: nothing of the kernels' bit manipulation."""
from __future__ import annotations

import numpy as np

FP8, FP4 = "mxfp8", "mxfp4"


def _grid(fmt):
    mant, bias, last = (3, 7, 126) if fmt == FP8 else (1, 1, 7)
    out = []
    for c in range(last + 1):
        exp, frac = c >> mant, c & ((1 << mant) - 1)
        out.append(np.ldexp(frac / (1 << mant), 1 - bias) if exp == 0
                   else np.ldexp(1 + frac / (1 << mant), exp - bias))
    return np.array(out, np.float64)


GRID = {FP8: _grid(FP8), FP4: _grid(FP4)}
assert GRID[FP8][-1] == 448 and GRID[FP4][-1] == 6


def bf16_to_f64(u):
    return (np.asarray(u, np.uint16).astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def f64_to_bf16(x):
    """Nearest-even BF16 bit patterns of 64-bit values (one rounding; subnormals included)."""
    x = np.asarray(x, np.float64)
    _, e = np.frexp(np.abs(x))
    step = np.ldexp(1.0, np.maximum(e - 8, -133))
    return (np.rint(x / step) * step).astype(np.float32).view(np.uint32).__rshift__(16).astype(np.uint16)


def exponents(b, fmt, floor):
    """Shared exponents of blocks b [..., 32] (64-bit)."""
    top = np.abs(b).max(-1)
    _, e = np.frexp(top)
    fl = np.where(top > 0, e - 1, -10000)   # floor(log2)
    if floor:
        r = fl - (8 if fmt == FP8 else 2)
    else:
        big = GRID[fmt][-1]
        r = fl - 12
        for _ in range(16):
            r = np.where((top > 0) & (top > big * np.ldexp(1.0, r)), r + 1, r)
    return np.maximum(r, -127)


def nearest_code(u, fmt):
    """Codes (sign in the top bit) of the nearest value, ties to the even code, saturating."""
    g = GRID[fmt]
    a = np.minimum(np.abs(u), g[-1])
    lo = np.clip(np.searchsorted(g, a, side="right") - 1, 0, len(g) - 2)
    below, above = a - g[lo], g[lo + 1] - a
    c = np.where((above < below) | ((above == below) & (lo % 2 == 1)), lo + 1, lo)
    return (c | np.where(np.signbit(u), 128 if fmt == FP8 else 8, 0)).astype(np.uint8)


def quantize(v, fmt, floor=False):
    """v [M, N] 64-bit -> (codes [M, N], scale bytes [M, N/32])."""
    M, N = v.shape
    b = v.reshape(M, N // 32, 32)
    e = exponents(b, fmt, floor)
    return nearest_code(np.ldexp(b, -e[..., None]), fmt).reshape(M, N), (e + 127).astype(np.uint8)


def values(codes, bytes_, fmt):
    """The 64-bit numbers that codes [M, N] with scale bytes [M, N/32] stand for."""
    mask, sign = (127, 128) if fmt == FP8 else (7, 8)
    v = GRID[fmt][np.minimum(codes & mask, len(GRID[fmt]) - 1)]
    v = np.where(codes & sign, -v, v)
    return np.ldexp(v, np.repeat(bytes_.astype(np.int64) - 127, 32, axis=1))


def pack(codes):
    return (codes[:, 0::2] | (codes[:, 1::2] << 4)).astype(np.uint8)


def unpack(p):
    return np.stack([p & 15, p >> 4], -1).reshape(p.shape[0], -1)

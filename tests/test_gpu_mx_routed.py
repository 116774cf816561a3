"""Products grouped by a plan against 64-bit products of the numbers that the codes stand for.

Each result is a sum as lpq_mx_matmul takes it, so test_gpu_mx_matmul's tolerance holds per
group, with the group's rows as the contraction of a weight gradient."""
import numpy as np
import pytest
import torch

from tests import mx_ref as M
from tests.gpu_util import DEV
from tests.test_gpu_mx_matmul import FORMATS, bound, operand

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lpq():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import precision_weight_quantization_amd as m
    return m


def many(rows, K, fmt, seed, scale=1.0):
    """An operand of many rows: 97 rows of drawn values in a shuffled order."""
    held, e, v = operand(min(rows, 97), K, fmt, seed, scale)
    at = torch.randint(0, held.shape[0], (rows,), device=DEV, generator=torch.Generator(device=DEV).manual_seed(seed))
    held = held.view(torch.uint8)[at]
    return (held if fmt == M.FP4 else held.view(torch.float8_e4m3fn)), e[at], v[at]


def offsets_of(sizes, lead):
    return [lead, *(lead + np.cumsum(sizes)).tolist()]


def sizes_of(groups, most, seed, empty=0.3):
    rng = np.random.default_rng(seed)
    return np.where(rng.random(groups) < empty, 0, rng.integers(1, most + 1, groups)).tolist()


# rows of each group, rows before the first, rows behind the last, N, K
ROWS = [([1], 0, 0, 1, 32), ([0, 3, 0], 0, 5, 40, 96), ([1, 0, 0, 5], 3, 2, 130, 160), ([16, 17, 0, 33, 1], 0, 0, 96, 1056),
        ([0, 0], 0, 40, 64, 128), (sizes_of(130, 3, 1), 1, 7, 144, 768), (sizes_of(64, 40, 2), 0, 100, 257, 544),
        (sizes_of(1024, 2, 3, 0.8), 0, 11, 72, 288), (sizes_of(37, 25, 4), 9, 0, 2053, 416),
        # tiles: 128 x 64, 128 x 128, then 256 x 256; whole, ragged, one row, none, one stage and many
        ([64, 0, 63, 65, 1, 30], 3, 0, 128, 544), (sizes_of(90, 30, 9), 0, 5, 390, 1056), ([6, 6, 60, 0, 8], 0, 0, 136, 512),
        ([128, 128, 128], 0, 0, 256, 512), ([100, 0, 1, 129, 200], 5, 3, 130, 288), ([1, 1, 380], 0, 40, 200, 1056),
        ([0, 0, 0, 0], 100, 300, 160, 416), (sizes_of(70, 300, 5), 3, 0, 264, 544), (sizes_of(130, 200, 6), 0, 60, 129, 320),
        ([256, 256], 0, 0, 512, 1024), ([257, 511, 0, 1, 300], 7, 11, 520, 288), ([700], 0, 0, 256, 544), ([10, 1300, 2], 0, 500, 1021, 1056),
        (sizes_of(33, 700, 7), 1, 2, 768, 416)]


@pytest.mark.parametrize("fmts", FORMATS)
@pytest.mark.parametrize("case", range(len(ROWS)))
def test_rows(lpq, case, fmts):
    sizes, lead, tail, N, K = ROWS[case]
    off, groups = offsets_of(sizes, lead), len(sizes)
    R = off[-1] + tail
    a, ae, va = many(R, K, fmts[0], 1)
    b, be, vb = many(groups * N, K, fmts[1], 2, 0.02)
    b, be, vb = b.view(groups, N, -1), be.view(groups, N, -1), vb.view(groups, N, K)
    offsets = torch.tensor(off, dtype=torch.int32, device=DEV)
    for f32 in ((False, True) if fmts == (M.FP4, M.FP4) else (False,)):
        dtype = torch.float32 if f32 else torch.bfloat16
        print(f"  {sizes[:8]} {lead} {tail} {N}x{K} {fmts} {dtype}", flush=True)
        buf = torch.full((R * N + 256,), 5.0, dtype=dtype, device=DEV)
        y = lpq.lpq_mx_matmul_routed(a, ae, b, be, offsets, out_dtype=dtype, y=buf)[:R * N].view(R, N)
        assert bool((buf[R * N:] == 5).all()) and bool((y[:lead] == 5).all()) and bool((y[off[-1]:] == 5).all())
        for g in range(groups):
            r = slice(off[g], off[g + 1])
            if off[g] < off[g + 1]:
                exact = va[r] @ vb[g].T
                err = (y[r].double() - exact).abs()
                assert bool((err <= bound(va[r], vb[g], exact, fmts, f32)).all()), (g, float(err.max()))
        again = torch.full_like(buf, 5.0)
        lpq.lpq_mx_matmul_routed(a, ae, b, be, offsets, out_dtype=dtype, y=again)
        assert torch.equal(again, buf)


# rows of each group (multiples of 32), rows before the first, rows behind the last, M, N
SUMS = [([32], 0, 0, 1, 1), ([0, 64, 0], 32, 32, 40, 17), ([32, 0, 160, 1056], 0, 0, 100, 300), ([64] * 40 + [0] * 30, 0, 64, 33, 70),
        # tiles: of 128 x 128, then of 256 x 256; groups of no stage, a part of one, one, several
        ([128, 256, 512], 0, 0, 128, 128), ([0, 32, 64, 96, 0, 160], 32, 0, 130, 200), ([0, 0, 0], 64, 32, 256, 128),
        ([32] * 300, 0, 0, 136, 129), ([544, 32, 0, 1600, 64] * 12, 32, 0, 512, 776), ([320] * 70, 0, 64, 517, 512), ([2048, 0, 544, 2080], 0, 96, 255, 512), ([416, 128, 0, 384], 0, 0, 256, 256),
        ([0, 32, 0, 64, 96, 1056, 128, 0], 32, 64, 520, 264), ([32 * s for s in sizes_of(50, 20, 8)], 0, 0, 300, 513), ([0], 0, 32, 512, 256)]


@pytest.mark.parametrize("fmts", FORMATS)
@pytest.mark.parametrize("case", range(len(SUMS)))
def test_sums(lpq, case, fmts):
    sizes, lead, tail, m, n = SUMS[case]
    off, groups = offsets_of(sizes, lead), len(sizes)
    R = off[-1] + tail
    (a, ae, va), (b, be, vb) = many(m, R, fmts[0], 3), many(n, R, fmts[1], 4, 1e-3)
    # what lies outside the groups is not read into a result: NaN scales there would show
    for e in (ae, be):
        e[:, :lead // 32] = 255
        e[:, off[-1] // 32:] = 255
    offsets = torch.tensor(off, dtype=torch.int32, device=DEV)
    for f32 in ((False, True) if fmts == (M.FP4, M.FP4) else (False,)):
        dtype = torch.float32 if f32 else torch.bfloat16
        print(f"  {sizes[:8]} {lead} {tail} {m}x{n} {fmts} {dtype}", flush=True)
        buf = torch.full((groups * m * n + 256,), 5.0, dtype=dtype, device=DEV)
        y = lpq.lpq_mx_matmul_routed_dw(a, ae, b, be, offsets, out_dtype=dtype, y=buf)[:groups * m * n].view(groups, m, n)
        assert bool((buf[groups * m * n:] == 5).all())
        for g in range(groups):
            r = slice(off[g], off[g + 1])
            if off[g] == off[g + 1]:
                assert bool((y[g] == 0).all()), g
                continue
            exact = va[:, r] @ vb[:, r].T
            err = (y[g].double() - exact).abs()
            assert bool((err <= bound(va[:, r], vb[:, r], exact, fmts, f32)).all()), (g, float(err.max()))
        again = lpq.lpq_mx_matmul_routed_dw(a, ae, b, be, offsets, out_dtype=dtype)
        assert torch.equal(again, y)


@pytest.mark.parametrize("K,N,rows", [(544, 200, 40), (544, 264, 200), (544, 512, 900)])
def test_offsets_outside_the_buffers(lpq, K, N, rows):
    """A plan that was not made by lpq_route_plan: nothing outside the buffers is touched."""
    a, ae, _ = many(rows, K, M.FP8, 5)
    b, be, _ = many(3 * N, K, M.FP4, 6)
    b, be = b.view(3, N, -1), be.view(3, N, -1)
    buf = torch.full((rows * N + 512,), 5.0, dtype=torch.bfloat16, device=DEV)
    for off in ([-5, 10, 1 << 30, -(1 << 31)], [rows, rows + 9, rows - 3, 2 * rows], [(1 << 31) - 1, 0, 4, 1 << 30]):
        lpq.lpq_mx_matmul_routed(a, ae, b, be, torch.tensor(off, dtype=torch.int32, device=DEV), y=buf)
        assert bool((buf[rows * N:] == 5).all())
    at, ate, _ = many(N, 32 * rows, M.FP8, 7)
    bt, bte, _ = many(N + 8, 32 * rows, M.FP8, 8)
    for off in ([-5, 10, 1 << 30, -(1 << 31)], [32 * rows, 32 * rows + 9, 32 * rows - 3, 1 << 30], [(1 << 31) - 1, 0, 4, 1 << 30]):
        y = lpq.lpq_mx_matmul_routed_dw(at, ate, bt, bte, torch.tensor(off, dtype=torch.int32, device=DEV))
        assert y.shape == (3, N, N + 8)


@pytest.mark.parametrize("groups,m,n", [(4, 40, 17), (5, 130, 200), (3, 256, 512)])
def test_not_finite(lpq, groups, m, n):
    """NaN codes and scale bytes of one group show in no other group's results."""
    sizes = ([32, 96, 160, 64, 224] * 2)[:groups]
    off = offsets_of(sizes, 0)
    offsets = torch.tensor(off, dtype=torch.int32, device=DEV)
    R, bad = off[-1], slice(off[1], off[2])
    (a, ae, _), (b, be, _) = many(m, R, M.FP8, 3), many(n, R, M.FP8, 4)
    others = [g for g in range(groups) if g != 1]
    want = lpq.lpq_mx_matmul_routed_dw(a, ae, b, be, offsets)
    a.view(torch.uint8)[:, bad] = 0x7f
    be[:, bad.start // 32:bad.stop // 32] = 255
    got = lpq.lpq_mx_matmul_routed_dw(a, ae, b, be, offsets)
    assert torch.equal(got[others], want[others]) and bool(got[1].isnan().all())
    (a, ae, _), (b, be, _) = many(R, 544, M.FP8, 5), many(groups * n, 544, M.FP4, 6)
    b, be = b.view(groups, n, -1), be.view(groups, n, -1)
    want = lpq.lpq_mx_matmul_routed(a, ae, b, be, offsets)
    a.view(torch.uint8)[bad] = 0x7f
    be[1] = 255
    got = lpq.lpq_mx_matmul_routed(a, ae, b, be, offsets)
    rows = torch.ones(R, dtype=torch.bool, device=DEV)
    rows[bad] = False
    assert torch.equal(got[rows], want[rows]) and bool(got[~rows].isnan().all())


def test_past_32_bits(lpq):
    """Results of more than 2^32 elements, or bytes behind 2^32 of them: the last group's rows, and its gradient."""
    sizes = [270000, 0, 33]
    off = offsets_of(sizes, 0)
    offsets = torch.tensor(off, dtype=torch.int32, device=DEV)
    R, N, K = off[-1], 16400, 288
    a, ae, va = many(R, K, M.FP8, 1)
    b, be, vb = many(3 * N, K, M.FP8, 2)
    y = lpq.lpq_mx_matmul_routed(a, ae, b.view(3, N, K), be.view(3, N, -1), offsets)
    assert y.numel() > 1 << 32
    for r, g in ((slice(0, 40), 0), (slice(off[1] - 40, off[1]), 0), (slice(off[2], R), 2)):
        w = vb[g * N:(g + 1) * N]
        exact = va[r] @ w.T
        assert bool(((y[r].double() - exact).abs() <= bound(va[r], w, exact, (M.FP8, M.FP8), False)).all())
    del y, a, ae, va, b, be, vb
    (a, ae, va), (b, be, vb) = many(8200, 65 * 32, M.FP8, 3), many(8208, 65 * 32, M.FP8, 4)
    dw = lpq.lpq_mx_matmul_routed_dw(a, ae, b, be, torch.arange(66, dtype=torch.int32, device=DEV) * 32)
    assert dw.numel() > 1 << 32
    for g in (0, 64):
        p, q = va[:, g * 32:g * 32 + 32], vb[:, g * 32:g * 32 + 32]
        exact = p @ q.T
        assert bool(((dw[g].double() - exact).abs() <= bound(p, q, exact, (M.FP8, M.FP8), False)).all())

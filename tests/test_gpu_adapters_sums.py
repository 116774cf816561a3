"""Adapters' sums in between: the bits that u and du carry into the second product, and what infinities
and NaN make of them.

Where a test asks for equality every sum in between is exact in FP32, so that the result is the 64-bit one
rounded once.  The others take test_gpu_adapters' tolerances, with u in three BF16 numbers, which leave 2^-24 of
it and not 2^-16; the second and third number's products are 2^-8 and 2^-16 of the first's, and so are the roundings of
their sums: 1.01 times the first's."""
import numpy as np
import pytest
import torch

from tests import routed_ref as R
from tests.gpu_util import DEV
from tests.test_gpu_adapters import rounded
from tests.test_gpu_rmsnorm import bf16, f64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lpq():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import precision_weight_quantization_amd as m
    return m


def bf(a):
    """Numbers that BF16 holds, on the device."""
    t = torch.from_numpy(np.ascontiguousarray(a, np.float32))
    assert torch.equal(t.to(torch.bfloat16).float(), t), "values of the format only"
    return t.to(torch.bfloat16).to(DEV)


def plan_of(lpq, ids, groups, align=1):
    return lpq.lpq_route_plan(torch.from_numpy(np.asarray(ids, np.int32)).to(DEV), groups, align)


@pytest.mark.parametrize("rank", [8, 40, 128])
@pytest.mark.parametrize("tokens", [20, 300])   # rows by waves of their own, and tiles of 64 rows
def test_all_bits_of_u(lpq, tokens, rank):
    """u = a0 + a1 2^-8 + a2 2^-16 has 24 bits; each result is the difference of two u that share a0 and a1, so what is
    left of it are the last 8.  Every partial sum is a multiple of 2^-16 up to 2^8 (times a token's power of two): exact."""
    L, wide, long = 2, 136, 72
    rng = np.random.default_rng(rank + tokens)
    ids = rng.integers(0, L, tokens)
    plan = plan_of(lpq, ids, L)
    digits = rng.integers(0, 256, (3, L, rank))
    digits[0] |= 128
    digits[:2, :, 1::2] = digits[:2, :, 0::2]   # of a pair the last digit differs only
    first = np.zeros((L, rank, long))
    first[:, :, :3] = np.moveaxis(digits, 0, 2)
    second = np.zeros((L, wide, rank))
    for n in range(wide):
        j = 2 * (n % (rank // 2))
        second[:, n, j], second[:, n, j + 1] = 2.0 ** (n % 3), -2.0 ** (n % 3)
    x = np.zeros((tokens, long))
    x[:, :3] = (rng.choice([-1.0, 1.0], tokens) * 2.0 ** rng.integers(-3, 4, tokens))[:, None] * 2.0 ** np.array([0, -8, -16])
    scale = np.array([0.5, 4.0])
    want = np.stack([scale[g] * (x[t] @ first[g].T) @ second[g].T for t, g in enumerate(ids)])
    assert np.abs(want).max() > 0
    want = torch.from_numpy(want).to(torch.float32).to(torch.bfloat16)   # 9 bits at most: one rounding
    s = torch.from_numpy(scale.astype(np.float32)).to(DEV)
    y = lpq.lpq_adapters(bf(x), bf(first), bf(second), *plan, scale=s)
    assert torch.equal(y.cpu(), want)
    # the same numbers through the backward pass: du = dy B, dx = du A
    dx, _, _ = lpq.lpq_adapters_backward(bf(x), bf(np.zeros((tokens, wide))), bf(second.transpose(0, 2, 1)), bf(first.transpose(0, 2, 1)),
                                         *plan, scale=s)
    assert torch.equal(dx.cpu(), want)


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("shape,align", [((40, 6, 16, 72, 136), 1), ((300, 40, 24, 640, 1032), 1), ((600, 3, 72, 264, 520), 32)])
def test_scale_of_an_adapter_without_tokens(lpq, shape, align, value):
    """It is in nobody's gradients: zeros for its own, or what was there.  Gradients of one part of the rows
    and of several."""
    T, L, r, N, K = shape
    ids = np.arange(T) % (L - 1) + 1   # none goes to the first
    plan = plan_of(lpq, ids, L, align)
    rng = np.random.default_rng(T)
    x, A, B, dy = (bf16(s, i).to(DEV) for i, s in enumerate(((T, K), (L, r, K), (L, N, r), (T, N))))
    scale = torch.from_numpy(rng.uniform(0.5, 2, L).astype(np.float32)).to(DEV)
    held = [torch.randn((L, r, K), device=DEV), torch.randn((L, N, r), device=DEV)]
    call = lambda **k: lpq.lpq_adapters_backward(dy, x, A, B, *plan, scale=scale, **k)
    plain, added = call(), call(dA=held[0].clone(), dB=held[1].clone(), accumulate=True)
    scale[0] = value
    for want, got in ((plain, call()), (added, call(dA=held[0].clone(), dB=held[1].clone(), accumulate=True))):
        assert all(torch.equal(a, b) for a, b in zip(want, got))
    assert bool((plain[1][0] == 0).all()) and bool((plain[2][0] == 0).all())
    assert torch.equal(added[1][0], held[0][0]) and torch.equal(added[2][0], held[1][0])


def test_infinite_scale_and_parts_without_tokens(lpq):
    """A group's infinite gradients stay so where parts of its rows are empty, or padding: positive numbers, so that
    every gradient is an infinity."""
    T, L, r, N, K = 500, 4, 24, 136, 264
    ids = np.where(np.arange(T) < 420, 3, np.arange(T) % 3)
    x, A, B, dy = (bf16(s, i).abs().clamp(min=2.0 ** -6).to(DEV) for i, s in enumerate(((T, K), (L, r, K), (L, N, r), (T, N))))
    scale = torch.ones(L, device=DEV)
    scale[1] = float("inf")
    for align in (1, 32, 1024):
        _, dA, dB = lpq.lpq_adapters_backward(dy, x, A, B, *plan_of(lpq, ids, L, align), scale=scale)
        for d in (dA, dB):
            assert bool((d[1] == float("inf")).all()) and bool(d[[0, 2, 3]].isfinite().all())


# tokens, groups, rank, N, K: rows by waves of their own, tiles of 64, parts of the gradients' rows
SHAPES = [(100, 7, 16, 264, 520), (400, 5, 72, 136, 1032), (900, 2, 24, 72, 264), (70, 1, 40, 2000, 64)]


def kinds(t):
    """0 finite, 1 and -1 infinite, 2 NaN."""
    a = f64(t) if isinstance(t, torch.Tensor) else t
    return np.where(np.isnan(a), 2, np.where(np.isinf(a), np.sign(a), 0)).astype(int)


def positive(shape, seed, scale=1.0):
    return bf16(shape, seed).abs().clamp(min=2.0 ** -6).mul(scale).to(torch.bfloat16).to(DEV)


def check(lpq, c, ids, plan):
    """Results and gradients against the formula: the same infinities, the same NaN, and near it elsewhere."""
    L, r, K = c["A"].shape
    N = c["B"].shape[1]
    names = "dy x A B scale base dres".split()
    d = {k: f64(c[k]) for k in names}
    kept = np.where((ids >= 0) & (ids < L), ids, -1)
    most = max(int((kept == g).sum()) for g in range(L))
    with np.errstate(all="ignore"):
        y, size = R.adapters(d["x"], d["A"], d["B"], ids, d["scale"], d["base"])
        want = R.adapters_grad(d["dy"], d["x"], d["A"], d["B"], ids, d["scale"], d["dres"])
        (dx, dA, dB), (sx, sA, sB) = want
        tols = [rounded(y, 1.01 * (K + r + 19) * 2.0 ** -24 * size, size), rounded(dx, 1.01 * (N + r + 19) * 2.0 ** -24 * sx, sx),
                1.01 * (N + most + 51) * 2.0 ** -24 * sA, 1.01 * (K + most + 51) * 2.0 ** -24 * sB]
        got = [lpq.lpq_adapters(c["x"], c["A"], c["B"], *plan, scale=c["scale"], base=c["base"]),
               *lpq.lpq_adapters_backward(c["dy"], c["x"], c["A"], c["B"], *plan, scale=c["scale"], dres=c["dres"])]
        for name, g, w, tol in zip(("y", "dx", "dA", "dB"), got, (y, dx, dA, dB), tols):
            assert np.array_equal(kinds(g), kinds(w)), (name, np.argwhere(kinds(g) != kinds(w))[:4])
            at = np.isfinite(w)
            assert (np.abs(f64(g) - w)[at] <= tol[at]).all(), name
    return got, (y, dx, dA, dB)


@pytest.mark.parametrize("value", [float("inf"), -float("inf"), float("nan")])
@pytest.mark.parametrize("where", ["x", "dy", "A", "B", "scale"])
@pytest.mark.parametrize("shape", SHAPES)
def test_infinities_as_the_formula(lpq, shape, where, value):
    """Factors and tokens of one sign, so that the formula itself gives infinities and few NaN."""
    T, L, r, N, K = shape
    rng = np.random.default_rng(T)
    ids = rng.integers(-1, L, T)
    ids[0] = 0
    c = {"x": positive((T, K), 1), "A": positive((L, r, K), 2, 0.05), "B": positive((L, N, r), 3, 0.3),
         "scale": torch.from_numpy(rng.uniform(0.5, 2, L).astype(np.float32)).to(DEV), "base": bf16((T, N), 4).to(DEV),
         "dy": positive((T, N), 5, 2.0 ** -10), "dres": bf16((T, K), 6, 1e-3).to(DEV)}
    t = c[where]
    if where in ("x", "dy"):
        some = np.nonzero(ids == 0)[0]
        t[int(some[0]), 5] = value
        t[int(some[-1]), t.shape[1] - 1] = value
    elif where == "scale":
        t[0] = value
    else:
        t[0, 3, 5] = value
    got, want = check(lpq, c, ids, lpq.lpq_route_plan(torch.from_numpy(ids.astype(np.int32)).to(DEV), L))
    if value == value and where != "dy":   # the infinities are there to be met
        assert np.isinf(want[0]).any() and np.isinf(want[1 if where != "x" else 2]).any()


@pytest.mark.parametrize("value", [float("inf"), -float("inf")])
@pytest.mark.parametrize("shape", SHAPES)
def test_infinities_beside_both_signs(lpq, shape, value):
    """Infinite tokens and factors among numbers of both signs: each infinity goes by the sign that it meets, and
    two that meet are a NaN."""
    T, L, r, N, K = shape
    ids = np.random.default_rng(T).integers(-1, L, T)
    ids[:2] = 0
    plan = lpq.lpq_route_plan(torch.from_numpy(ids.astype(np.int32)).to(DEV), L)
    for where in ("x", "A", "B", "dy"):
        c = {"x": bf16((T, K), 1).to(DEV), "A": bf16((L, r, K), 2, 0.05).to(DEV), "B": bf16((L, N, r), 3, 0.3).to(DEV),
             "scale": torch.linspace(-1, 2, L, device=DEV), "base": bf16((T, N), 4).to(DEV), "dy": bf16((T, N), 5, 1e-3).to(DEV),
             "dres": bf16((T, K), 6, 1e-3).to(DEV)}
        c["scale"][0] = 0.75
        c["A"][0][c["A"][0] == 0] = 0.5   # 0 times an infinity is another matter
        c["B"][0][c["B"][0] == 0] = 0.5
        if where in ("x", "dy"):
            c[where][1, 3] = value
        else:
            c[where][0, 2, 1] = value
        check(lpq, c, ids, plan)


@pytest.mark.parametrize("value", [float("inf"), float("nan")])
@pytest.mark.parametrize("shape", SHAPES)
def test_padding_beside_infinite_factors(lpq, shape, value):
    """Padding rows of a group whose factors hold infinities or NaN add nothing to its gradients."""
    T, L, r, N, K = shape
    ids = np.random.default_rng(T).integers(0, L, T)
    for where in ("A", "B"):
        c = {"x": positive((T, K), 1), "A": positive((L, r, K), 2, 0.05), "B": positive((L, N, r), 3, 0.3),
             "scale": torch.linspace(0.5, 2, L, device=DEV), "base": bf16((T, N), 4).to(DEV),
             "dy": positive((T, N), 5, 2.0 ** -10), "dres": bf16((T, K), 6, 1e-3).to(DEV)}
        c[where][0, 3, 5] = value
        for align in (5, 64):
            _, want = check(lpq, c, ids, plan_of(lpq, ids, L, align))
            d = want[3 if where == "A" else 2][0]   # dB or dA of that adapter
            assert value != value or np.isinf(d).any() and not np.isnan(d).any()


def test_above_the_largest_bf16(lpq):
    """u and du between BF16's largest number and FP32's: finite, and their products as exact as others."""
    high = 2.0 ** 63 * 1.9921875, 2.0 ** 62                    # of a token
    low = 2.0 ** 64, 2.0 ** 57 * 1.0625                         # of the first factor
    u = high[0] * low[0] + high[1] * low[1]                     # rounds to an infinity in BF16
    assert 2.0 ** 127 * 1.9921875 < u < 2.0 ** 128 and np.float32(u) == u
    for tokens, rank in ((3, 8), (200, 24), (200, 72)):
        ids = np.arange(tokens) % 2
        plan = plan_of(lpq, ids, 2)
        N, K = 72, 40
        x, first, second = np.zeros((tokens, K)), np.zeros((2, rank, K)), np.zeros((2, N, rank))
        sign = np.where(np.arange(tokens) % 3 == 0, -1.0, 1.0)
        x[:, :2] = sign[:, None] * np.array(high)
        first[:, :, :2] = np.array(low)
        for n in range(N):
            second[:, n, n % rank] = (1 + n % 5) * 2.0 ** -121
        want = torch.from_numpy(sign[:, None] * u * second.sum(2)[ids]).float().to(torch.bfloat16)   # one product: 13 bits by 3
        assert bool(want.isfinite().all())
        assert torch.equal(lpq.lpq_adapters(bf(x), bf(first), bf(second), *plan).cpu(), want)
        dx, _, _ = lpq.lpq_adapters_backward(bf(x), bf(np.zeros((tokens, N))), bf(second.transpose(0, 2, 1)), bf(first.transpose(0, 2, 1)), *plan)
        assert torch.equal(dx.cpu(), want)
        # the FP32 gradients: one token of group 0 has the other factor, 2^-120
        one = np.zeros((tokens, N))
        one[0, 7] = 3 * 2.0 ** -121
        _, _, dB = lpq.lpq_adapters_backward(bf(one), bf(x), bf(first), bf(np.zeros((2, N, rank))), *plan)
        exact = np.zeros((2, N, rank))
        exact[0, 7] = sign[0] * u * one[0, 7]
        assert np.array_equal(f64(dB), exact)
        _, dA, _ = lpq.lpq_adapters_backward(bf(x), bf(one), bf(np.zeros((2, rank, N))), bf(first.transpose(0, 2, 1)), *plan)
        assert np.array_equal(f64(dA), exact.transpose(0, 2, 1))

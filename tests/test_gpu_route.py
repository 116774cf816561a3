"""The plan, the gather and the combination of routed layers against plain references.

Plans and gathered codes are whole numbers: equal.  A combination is an FP32 sum of k + 1
terms, each step off by at most 2^-24 of a partial sum, no more than the sum S of the terms'
magnitudes, then one rounding to BF16 (2^-8): (k + 1) 2^-24 S + 2^-8 (|exact| + that).  dy is one FP32
product and one rounding: (2^-24 + 2^-8) |exact|, and half a step of BF16's smallest.  dweights is an FP32 sum of N
products: N 2^-24 S."""
import numpy as np
import pytest
import torch

from tests import routed_ref as R
from tests.gpu_util import DEV
from tests.test_gpu_rmsnorm import bf16, f64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lpq():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import precision_weight_quantization_amd as m
    return m


def routing(T, k, groups, seed, drop=0.2):
    """Distinct ids a token where they reach, some outside [0, groups)."""
    rng = np.random.default_rng(seed)
    ids = np.argsort(rng.random((T, max(k, groups))) + 0.5 * rng.random(max(k, groups)), axis=1)[:, :k]
    return np.where(rng.random((T, k)) < drop, rng.choice([-1, groups, -(1 << 31), (1 << 31) - 1], (T, k)), ids)


def dev(a, dtype=torch.int32):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV).to(dtype)


def equal(got, want):
    for g, w in zip(got, want):
        assert np.array_equal(g.cpu().numpy(), w), (g, w)


@pytest.mark.parametrize("align", [1, 7, 32])
@pytest.mark.parametrize("pairs,groups", [(1, 1), (1, 1024), (8, 64), (63, 5), (64, 64), (65, 65), (1023, 2), (1025, 60), (4096, 128),
                                          (4097, 128), (5120, 1000), (65536, 128), (300001, 1024), (700000, 3)])
def test_plan(lpq, pairs, groups, align):
    rng = np.random.default_rng(pairs + groups)
    ids = np.where(rng.random(pairs) < 0.1, rng.integers(-3, groups + 3, pairs), (groups * rng.random(pairs) ** 2).astype(np.int64))
    want = R.plan(ids, groups, align)
    assert len(want[2]) == lpq.lpq_route_capacity(pairs, groups, align)
    equal(lpq.lpq_route_plan(dev(ids), groups, align), want)
    far = np.where(ids < 0, ids - (1 << 40), np.where(ids >= groups, ids + (1 << 32), ids))   # low words that look valid
    equal(lpq.lpq_route_plan(dev(far, torch.int64), groups, align), want)


@pytest.mark.parametrize("what", ["one group", "none", "last"])
@pytest.mark.parametrize("pairs", [5, 2000, 9000])
def test_plan_of_one_kind(lpq, pairs, what):
    ids = np.full(pairs, {"one group": 3, "none": -1, "last": 11}[what])
    equal(lpq.lpq_route_plan(dev(ids), 12, 32), R.plan(ids, 12, 32))


def test_plan_into_larger_buffers(lpq):
    """A larger src is filled, and nothing behind offsets, rows and src is written."""
    for T, k in ((300, 3), (3000, 3)):
        ids = routing(T, k, 40, 5)
        capacity = lpq.lpq_route_capacity(T * k, 40, 32) + 1000
        off, rows, src = (torch.full((n + 64,), 77, dtype=torch.int32, device=DEV) for n in (41, T * k, capacity))
        got = lpq.lpq_route_plan(dev(ids), 40, 32, offsets=off[:41], rows=rows[:T * k].view(T, k), src=src[:capacity])
        equal(got, R.plan(ids, 40, 32, capacity))
        assert all(bool((t[-64:] == 77).all()) for t in (off, rows, src))


@pytest.mark.parametrize("align", [1, 32])
@pytest.mark.parametrize("T,k,groups,N", [(1, 1, 1, 32), (1, 8, 64, 2048), (3, 2, 5, 96), (77, 6, 60, 1056), (513, 8, 128, 2048),
                                          (130, 9, 40, 7168), (1000, 1, 7, 64)])
def test_gather(lpq, T, k, groups, N, align):
    x = bf16((T, N), 3, outliers=1e-3).to(DEV)
    ids = routing(T, k, groups, 4)
    _, rows, src = lpq.lpq_route_plan(dev(ids), groups, align)
    at = src.long().clamp(min=0) // k
    real = (src >= 0)[:, None]
    want = torch.where(real, x.view(torch.int16)[at], 0)
    assert torch.equal(lpq.lpq_route_gather(x, rows, src).view(torch.int16), want)
    for gather, quantize in ((lpq.lpq_route_gather_mxfp8, lpq.lpq_quantize_mxfp8), (lpq.lpq_route_gather_mxfp4, lpq.lpq_quantize_mxfp4)):
        q, e = quantize(x)
        R_ = src.numel()
        codes = torch.full((R_ * q.shape[1] + 64,), 77, dtype=torch.uint8, device=DEV)
        scales = torch.full((R_ * e.shape[1] + 64,), 77, dtype=torch.uint8, device=DEV)
        gather(x, rows, src, codes, scales)
        assert torch.equal(codes[:-64].view(R_, -1), torch.where(real, q.view(torch.uint8)[at], 0))
        assert torch.equal(scales[:-64].view(R_, -1), torch.where(real, e[at], 0))
        assert bool((codes[-64:] == 77).all()) and bool((scales[-64:] == 77).all())


SHAPES = [(1, 1, 1, 32), (1, 8, 64, 2048), (3, 2, 5, 96), (77, 6, 60, 1056), (513, 8, 128, 2048), (130, 19, 40, 512), (40, 9, 12, 7168),
          (1000, 1, 7, 544)]


def inputs(lpq, T, k, groups, N, align):
    ids = routing(T, k, groups, 6)
    _, rows, src = lpq.lpq_route_plan(dev(ids), groups, align)
    y = bf16((src.numel(), N), 7).to(DEV)
    y[src < 0] = float("nan")   # rows of no token: never looked at
    w = torch.from_numpy(np.random.default_rng(8).normal(size=(T, k)).astype(np.float32)).to(DEV)
    w[rows < 0] = float("nan")
    return rows, src, y, w


@pytest.mark.parametrize("align", [1, 32])
@pytest.mark.parametrize("T,k,groups,N", SHAPES)
def test_combine(lpq, T, k, groups, N, align):
    rows, src, y, w = inputs(lpq, T, k, groups, N, align)
    res = bf16((T, N), 9, 2.0).to(DEV)
    r, y64 = rows.cpu().numpy(), np.nan_to_num(f64(y))
    for weights, residual in ((w, res), (None, None), (w, None)):
        exact, size = R.combine(y64, r, np.ones(r.shape) if weights is None else np.nan_to_num(f64(w)),
                                np.zeros((T, N)) if residual is None else f64(res))
        tol = (k + 1) * 2.0 ** -24 * size
        tol = tol + 2.0 ** -8 * (np.abs(exact) + tol)
        got = lpq.lpq_route_combine(y, rows, weights, residual)
        assert (np.abs(f64(got) - exact) <= tol).all()
        if residual is not None:   # in place
            again = res.clone()
            lpq.lpq_route_combine(y, rows, weights, again, out=again)
            assert torch.equal(again.view(torch.int16), got.view(torch.int16))


@pytest.mark.parametrize("align", [1, 32])
@pytest.mark.parametrize("T,k,groups,N", SHAPES)
def test_combine_backward(lpq, T, k, groups, N, align):
    rows, src, y, w = inputs(lpq, T, k, groups, N, align)
    dout = bf16((T, N), 10, 1e-3).to(DEV)
    for weights in (w, None):
        w64 = np.ones((T, k)) if weights is None else np.nan_to_num(f64(w))
        dy, dw, size = R.combine_grad(f64(dout), np.nan_to_num(f64(y)), rows.cpu().numpy(), src.cpu().numpy(), w64)
        gy, gw = lpq.lpq_route_combine_backward(dout, rows, src, weights, y=y)
        assert (np.abs(f64(gy) - dy) <= (2.0 ** -24 + 2.0 ** -8) * np.abs(dy) + 2.0 ** -134).all()
        assert (np.abs(f64(gw) - dw) <= N * 2.0 ** -24 * size).all()
        only, none = lpq.lpq_route_combine_backward(dout, rows, src, weights, want_dweights=False)
        assert none is None and torch.equal(only.view(torch.int16), gy.view(torch.int16))
        again = lpq.lpq_route_combine_backward(dout, rows, src, weights, y=y)
        assert torch.equal(again[1], gw)


def test_past_32_bits(lpq):
    """A routed matrix of more than 2^32 elements."""
    T, k, N = 135000, 2, 16000
    x = torch.randn((T, N), device=DEV, dtype=torch.bfloat16)
    ids = torch.arange(2 * T, device=DEV, dtype=torch.int32).view(T, k) % 3
    offsets, rows, src = lpq.lpq_route_plan(ids, 3, 32)
    y = lpq.lpq_route_gather(x, rows, src)
    assert y.numel() > 1 << 32
    ends = torch.cat([torch.arange(300), torch.arange(T - 300, T)]).to(DEV)
    for j in range(k):
        assert torch.equal(y[rows[ends, j].long()], x[ends])
    q, e = lpq.lpq_route_gather_mxfp8(x, rows, src)
    want, scale = lpq.lpq_quantize_mxfp8(x[ends].contiguous())
    u8 = lambda t: t.view(torch.uint8)
    for j in range(k):
        r = rows[ends, j].long()
        assert torch.equal(u8(q)[r], u8(want)) and torch.equal(e[r], scale)
    del q, e
    out = lpq.lpq_route_combine(y, rows)   # exact: x + x
    assert torch.equal(out[ends], 2 * x[ends])
    del out
    dy, dw = lpq.lpq_route_combine_backward(x, rows, src, None, y)
    for j in range(k):
        assert torch.equal(dy[rows[ends, j].long()], x[ends])
    exact = x[ends].double().square().sum(1)   # N products of one sign, N + 12 roundings
    assert bool(((dw[ends].double() - exact[:, None]).abs() <= (N + 12) * 2.0 ** -24 * exact[:, None]).all())

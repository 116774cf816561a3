"""Low-rank adapters against the formula in 64 bits.

Tolerances.  u = x A^T is an FP32 sum of K exact products: off by K 2^-24 of U, the sum of
their magnitudes.  It is scaled (2^-24) and taken as two BF16 numbers, which leave at most 2^-16 of it (half a
step of each: 2^-8 2^-8), then summed over the rank: with S = |s| (|x| |A|^T) |B|^T the
low-rank part is off by (K + rank + 2) 2^-24 S + 2^-16 S.  y adds the base (2^-24 of the sum) and is rounded to
BF16 (2^-8).  dx likewise, with N for K.  The FP32 gradients take u and du as three BF16 numbers
(2^-24): with M tokens, (K + M + 3 + parts) 2^-24 of the sum of their terms' magnitudes; parts, of
the rows and of k, at most 32 + 16."""
import numpy as np
import pytest
import torch

from tests import routed_ref as R
from tests.gpu_util import DEV
from tests.test_gpu_rmsnorm import bf16, f64

pytestmark = pytest.mark.gpu

# tokens, groups, rank, N, K
SHAPES = [(1, 1, 8, 8, 8), (1, 4, 16, 64, 128), (5, 3, 8, 72, 520), (16, 1, 64, 256, 256), (40, 32, 16, 4096, 2560), (33, 70, 24, 136, 1032),
          (77, 5, 40, 200, 64), (130, 2, 128, 320, 1056), (300, 9, 72, 1000, 136), (700, 3, 64, 264, 2560), (1030, 4, 32, 96, 5128),
          (2000, 1, 16, 8, 24), (1500, 1000, 8, 40, 48)]


@pytest.fixture(scope="module")
def lpq():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import precision_weight_quantization_amd as m
    return m


class Case:
    def __init__(self, lpq, shape, seed=0, spread=None):
        T, L, r, N, K = shape
        rng = np.random.default_rng(seed)
        self.ids = rng.integers(0, L, T) if spread is None else spread
        if spread is None:
            self.ids[rng.random(T) < 0.15] = rng.choice([-1, L])
        self.plan = lpq.lpq_route_plan(torch.from_numpy(self.ids.astype(np.int32)).to(DEV), L)
        self.x, self.base = bf16((T, K), 1, outliers=1e-3).to(DEV), bf16((T, N), 2).to(DEV)
        self.A, self.B = bf16((L, r, K), 3, K ** -0.5).to(DEV), bf16((L, N, r), 4, 0.3).to(DEV)
        self.scale = torch.from_numpy(rng.uniform(-2, 2, L).astype(np.float32)).to(DEV)
        self.dy, self.dres = bf16((T, N), 5, 1e-3).to(DEV), bf16((T, K), 6, 1e-3).to(DEV)

    def forward(self, lpq, scale=True, base=True, **kw):
        return lpq.lpq_adapters(self.x, self.A, self.B, *self.plan, scale=self.scale if scale else None,
                                base=self.base if base else None, **kw)

    def backward(self, lpq, scale=True, dres=True, **kw):
        return lpq.lpq_adapters_backward(self.dy, self.x, self.A, self.B, *self.plan, scale=self.scale if scale else None,
                                         dres=self.dres if dres else None, **kw)


def same(a, b):
    return all(torch.equal(s.contiguous().view(torch.uint8), t.contiguous().view(torch.uint8)) for s, t in zip(a, b))


def rounded(exact, low, part):
    """Tolerance of a BF16 result: part is off by low, then added and rounded."""
    tol = low + 2.0 ** -24 * (np.abs(exact) + part)
    return tol + 2.0 ** -8 * (np.abs(exact) + tol) + 2.0 ** -134


def check_forward(lpq, c, shape, scale, base):
    T, L, r, N, K = shape
    s, b = f64(c.scale) if scale else np.ones(L), f64(c.base) if base else np.zeros((T, N))
    exact, size = R.adapters(f64(c.x), f64(c.A), f64(c.B), c.ids, s, b)
    err = np.abs(f64(c.forward(lpq, scale, base)) - exact)
    tol = rounded(exact, ((K + r + 18) * 2.0 ** -24 + 2.0 ** -16) * size, size)
    assert (err <= tol).all(), (err.max(), (err / tol).max())


def check_backward(lpq, c, shape, scale, dres):
    T, L, r, N, K = shape
    s, d = f64(c.scale) if scale else np.ones(L), f64(c.dres) if dres else np.zeros((T, K))
    (dx, dA, dB), (sx, sA, sB) = R.adapters_grad(f64(c.dy), f64(c.x), f64(c.A), f64(c.B), c.ids, s, d)
    gx, gA, gB = c.backward(lpq, scale, dres)
    tol = rounded(dx, ((N + r + 18) * 2.0 ** -24 + 2.0 ** -16) * sx, sx)
    err = np.abs(f64(gx) - dx)
    assert (err <= tol).all(), (err.max(), (err / tol).max())
    most = np.bincount(c.ids[(c.ids >= 0) & (c.ids < L)], minlength=1).max(initial=0)
    assert (np.abs(f64(gA) - dA) <= (N + most + 51) * 2.0 ** -24 * sA).all()
    assert (np.abs(f64(gB) - dB) <= (K + most + 51) * 2.0 ** -24 * sB).all()
    for g, e in ((gA, dA), (gB, dB)):   # far nearer than the worst case over many results
        assert e.size < 256 or np.linalg.norm(f64(g) - e) <= 2e-6 * np.linalg.norm(e)
    assert same(c.backward(lpq, scale, dres), (gx, gA, gB))


@pytest.mark.parametrize("shape", SHAPES)
def test_forward(lpq, shape):
    c = Case(lpq, shape)
    print(f"  {shape}", flush=True)
    for scale, base in ((True, True), (False, False)):
        check_forward(lpq, c, shape, scale, base)
    y = c.forward(lpq)
    assert same([y], [c.forward(lpq)])
    T, N = y.shape
    buf = torch.full((T * N + 128,), 5.0, dtype=torch.bfloat16, device=DEV)   # in place, and nothing behind it
    buf[:T * N] = c.base.view(-1)
    at = buf[:T * N].view(T, N)
    lpq.lpq_adapters(c.x, c.A, c.B, *c.plan, scale=c.scale, base=at, y=at)
    assert same([at], [y]) and bool((buf[T * N:] == 5).all())


@pytest.mark.parametrize("shape", SHAPES)
def test_backward(lpq, shape):
    c = Case(lpq, shape)
    print(f"  {shape}", flush=True)
    for scale, dres in ((True, True), (False, False)):
        check_backward(lpq, c, shape, scale, dres)
    gx, gA, gB = c.backward(lpq)
    T, K = gx.shape
    bufs = [torch.full((n + 128,), 5.0, dtype=t, device=DEV) for n, t in ((T * K, torch.bfloat16), (gA.numel(), torch.float32),
                                                                          (gB.numel(), torch.float32))]
    bufs[0][:T * K] = c.dres.view(-1)
    outs = [b[:g.numel()].view(g.shape) for b, g in zip(bufs, (gx, gA, gB))]
    lpq.lpq_adapters_backward(c.dy, c.x, c.A, c.B, *c.plan, scale=c.scale, dres=outs[0], dx=outs[0], dA=outs[1], dB=outs[2])
    assert same(outs, (gx, gA, gB)) and all(bool((b[-128:] == 5).all()) for b in bufs)
    # accumulated: one FP32 addition to what is there
    more = [torch.randn(g.shape, device=DEV) for g in (gA, gB)]
    _, sA, sB = c.backward(lpq, dA=more[0].clone(), dB=more[1].clone(), accumulate=True)
    for s, m, g in ((sA, more[0], gA), (sB, more[1], gB)):
        assert bool(((s.double() - m.double() - g.double()).abs() <= 2.0 ** -24 * s.abs().double()).all())


@pytest.mark.parametrize("ids", [[-1] * 50, [3] * 50, [0, 3] * 25, [5] + [-1] * 48 + [0]])
def test_uneven(lpq, ids):
    """No token with an adapter, all with one, groups without tokens."""
    shape = (50, 6, 16, 80, 544)
    c = Case(lpq, shape, spread=np.array(ids))
    check_forward(lpq, c, shape, True, True)
    check_backward(lpq, c, shape, True, True)
    none = torch.from_numpy(c.ids < 0).to(DEV)
    assert same([c.forward(lpq)[none]], [c.base[none]]) and same([c.backward(lpq)[0][none]], [c.dres[none]])
    _, gA, gB = c.backward(lpq)
    for g in range(6):
        if g not in ids:
            assert bool((gA[g] == 0).all()) and bool((gB[g] == 0).all())


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("shape", [(100, 7, 16, 264, 520), (400, 5, 72, 136, 1032)])
def test_not_finite(lpq, shape, value):
    """What one adapter's tokens or factors hold shows in no other adapter's results."""
    T, L = shape[:2]
    ids = np.random.default_rng(9).integers(-1, L, T)
    for where in ("x", "dy", "A", "B", "scale"):
        c = Case(lpq, shape, spread=ids)
        want, (wx, wA, wB) = c.forward(lpq), c.backward(lpq)
        bad = torch.from_numpy(ids == 3).to(DEV)
        t = getattr(c, where)
        if where in ("x", "dy"):
            t[bad] = value
        else:
            t[3] = value
        got, (gx, gA, gB) = c.forward(lpq), c.backward(lpq)
        others = [g for g in range(L) if g != 3]
        assert same((got[~bad], gx[~bad], gA[others], gB[others]), (want[~bad], wx[~bad], wA[others], wB[others])), where
        assert where == "dy" or not bool(got[bad].isfinite().any()), where


def test_padded_plans(lpq):
    """A plan whose groups are padded, and one in a larger buffer, give the same results."""
    shape = (100, 7, 32, 264, 520)
    c = Case(lpq, shape)
    want, grads = c.forward(lpq), c.backward(lpq)
    ids = torch.from_numpy(c.ids.astype(np.int64)).to(DEV)
    for align, more in ((1, 1000), (32, 0), (5, 3)):
        src = torch.empty(lpq.lpq_route_capacity(100, 7, align) + more, dtype=torch.int32, device=DEV)
        c.plan = lpq.lpq_route_plan(ids, 7, align, src=src)
        check_forward(lpq, c, shape, True, True)
        check_backward(lpq, c, shape, True, True)
    assert torch.allclose(want.float(), c.forward(lpq).float(), rtol=2.0 ** -6, atol=1e-2) and grads[0].shape == c.x.shape


def test_a_plan_of_other_tokens(lpq):
    """A plan that was not made for these tokens: nothing outside the buffers is touched."""
    c = Case(lpq, (60, 4, 16, 136, 264))
    off, rows, src = (t.clone() for t in c.plan)
    off[1], off[3] = 1 << 30, -7
    src[:30:3], rows[:20:2] = 1 << 30, 1 << 29
    src[1], rows[1] = -5, -(1 << 31)
    c.plan = off, rows, src
    buf = torch.full((60 * 136 + 512,), 5.0, dtype=torch.bfloat16, device=DEV)
    c.forward(lpq, y=buf)
    assert bool((buf[60 * 136:] == 5).all())
    c.backward(lpq)

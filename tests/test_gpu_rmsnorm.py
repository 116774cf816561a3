"""The root-mean-square norm and its gradients against 64-bit references.

Tolerances, from the order of the FP32 operations (u = 2^-24, half a step of FP32;
2^-8 is half a step of BF16, relative):
 * sum of squares: a thread adds at most 64 terms in turn (8 vectors of 8), then at
   most 10 exchanges and 16 waves' sums: relative error below 90 u, all terms being
   positive; rstd takes half of it and 4 more roundings: 50 u;
 * y: rstd, two products and the BF16 rounding: |y| (2^-8 + 52 u);
 * dx: the mean of g n is off by at most 96 u times the mean of |g n|; the other
   terms take 8 roundings of what they are made of; then the BF16 rounding;
 * dgamma: a thread adds the rows it walks in turn (M / 256 at most, rounded up, as
   there are at least 256 workgroups or one for each row), then 4 exchanges, 4 waves,
   32 partials and 32 slices: (M / 256 + 75) u times the sum of |dy n|, each term with
   2 roundings of its own.
"""
import numpy as np
import pytest
import torch

from tests import mx_ref as R
from tests.gpu_util import DEV, host_u8, host_u16, report

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
EPS = 1e-6
SHAPES = [(1, 32), (1, 64), (5, 96), (3, 128), (1000, 128), (7, 160), (9, 256), (2, 512), (5, 544), (3, 1056), (4, 1568),
          (4, 2048), (300, 2560), (5, 2592), (3, 4096), (5, 4128), (2, 7168), (2, 8192), (2, 8224), (1, 16416), (2, 32768)]


@pytest.fixture(scope="module")
def lpq():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import precision_weight_quantization_amd as m
    return m


def bf16(shape, seed, scale=1.0, outliers=0.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(shape, generator=g) * scale
    if outliers:
        x = torch.where(torch.rand(shape, generator=g) < outliers, x * 100, x)
    return x.to(torch.bfloat16)


def f64(t):
    return t.detach().cpu().double().numpy()


def forward_ref(x, res, gamma):
    h = f64(x) + (0 if res is None else f64(res))
    h = R.bf16_to_f64(R.f64_to_bf16(h))
    rstd = 1 / np.sqrt((h * h).mean(1) + np.float64(np.float32(EPS)))
    return h, rstd, h * rstd[:, None] * f64(gamma)


@pytest.mark.parametrize("with_residual", [False, True])
@pytest.mark.parametrize("shape", SHAPES)
def test_forward(lpq, shape, with_residual):
    M, N = shape
    x, gamma = bf16(shape, 1, outliers=1e-3).to(DEV), (1 + 0.2 * bf16((N,), 2).float()).to(torch.bfloat16).to(DEV)
    res = bf16(shape, 3, 3.0).to(DEV) if with_residual else None
    if M > 2:
        x[1] = 0
        if res is not None:
            res[1] = 0
    h_ref, r_ref, y_ref = forward_ref(x, res, gamma)
    y, h, rstd = lpq.lpq_rmsnorm(x, gamma, EPS, residual=res)
    assert np.array_equal(f64(h), h_ref)
    assert (np.abs(f64(rstd) - r_ref) <= 50 * U * r_ref).all()
    assert (np.abs(f64(y) - y_ref) <= np.abs(y_ref) * (2.0 ** -8 + 52 * U)).all()
    y2 = torch.empty_like(y)
    q, e, h2, rstd2 = lpq.lpq_rmsnorm_mxfp8(x, gamma, EPS, residual=res, y=y2)
    qr, er = lpq.lpq_quantize_mxfp8(y)
    assert torch.equal(y.view(torch.int16), y2.view(torch.int16)) and torch.equal(rstd, rstd2)
    assert report("codes", host_u8(q), host_u8(qr)) + report("scales", host_u8(e), host_u8(er)) == 0
    q, e, _, _ = lpq.lpq_rmsnorm_mxfp8(x, gamma, EPS, residual=res)   # without y
    assert report("codes", host_u8(q), host_u8(qr)) + report("scales", host_u8(e), host_u8(er)) == 0
    if res is not None:   # in place on the residual stream, then on x
        for a, src, other in ((res.clone(), x, None), (x.clone(), None, res)):
            _, h3, _ = lpq.lpq_rmsnorm(a if src is None else src, gamma, EPS, residual=a if other is None else other, h=a)
            assert h3 is a and torch.equal(a.view(torch.int16), h.view(torch.int16))


def grad_ref(dy, h, gamma, rstd, dres):
    dy, h, gamma, r = f64(dy), f64(h), f64(gamma), f64(rstd)[:, None]
    g, n = dy * gamma, h * r
    s = (g * n).mean(1, keepdims=True)
    d = 0 if dres is None else f64(dres)
    dx = r * (g - n * s) + d
    size = np.abs(r * g) + np.abs(r * n * s) + np.abs(d)
    tol_dx = 2.0 ** -8 * np.abs(dx) + U * (8 * size + 96 * np.abs(r * n) * np.abs(g * n).mean(1, keepdims=True)) * 1.01
    tol_dg = U * (dy.shape[0] / 256 + 77) * np.abs(dy * n).sum(0)
    return dx, (dy * n).sum(0), tol_dx, tol_dg


def grad_inputs(shape, with_dres):
    M, N = shape
    h, dy = bf16(shape, 4, outliers=1e-3).to(DEV), bf16(shape, 5, 1e-3).to(DEV)
    gamma = (1 + 0.2 * bf16((N,), 6).float()).to(torch.bfloat16).to(DEV)
    rstd = (h.double().square().mean(1) + EPS).rsqrt().float()
    return dy, h, gamma, rstd, bf16(shape, 7, 1e-3).to(DEV) if with_dres else None


@pytest.mark.parametrize("with_dres", [False, True])
@pytest.mark.parametrize("shape", SHAPES + [(5000, 128), (40000, 32), (2200, 2560), (600, 8192)])
def test_backward(lpq, shape, with_dres):
    dy, h, gamma, rstd, dres = grad_inputs(shape, with_dres)
    dx_ref, dg_ref, tol_dx, tol_dg = grad_ref(dy, h, gamma, rstd, dres)
    dx, dg = lpq.lpq_rmsnorm_backward(dy, h, gamma, rstd, dres=dres)
    assert (np.abs(f64(dx) - dx_ref) <= tol_dx).all()
    assert (np.abs(f64(dg) - dg_ref) <= tol_dg).all()
    # the same bits every time, without dgamma, with a workspace of the caller's, and in place
    dx2, none = lpq.lpq_rmsnorm_backward(dy, h, gamma, rstd, dres=dres, want_dgamma=False)
    assert none is None and torch.equal(dx.view(torch.int16), dx2.view(torch.int16))
    need = lpq.lpq_rmsnorm_backward_workspace(*shape)
    work = torch.full((need + 64,), 0xFF, dtype=torch.uint8, device=DEV)
    start = torch.ones(shape[1], device=DEV)
    for target in (dy.clone(),) if dres is None else (dy.clone(), dres.clone()):
        acc = start.clone()
        mine = dict(dres=dres) if dres is None or not torch.equal(target, dres) else dict(dres=target)
        src = target if mine["dres"] is not target else dy
        dx3, dg3 = lpq.lpq_rmsnorm_backward(src, h, gamma, rstd, dx=target, dgamma=acc, accumulate=True, workspace=work, **mine)
        assert dx3 is target and torch.equal(dx3.view(torch.int16), dx.view(torch.int16))
        assert dg3 is acc and torch.equal(dg3, start + dg)
    assert (work[need:] == 0xFF).all()


@pytest.mark.parametrize("shape", [(6, 64), (5, 2560), (3, 4128)])
def test_gradients_against_differences(lpq, shape):
    """The slope of sum(w y) along a random direction, by central differences of the 64-bit
    forward formula, against the kernel's gradients; off by their BF16 and FP32 roundings
    and the difference's own error (step 1e-4: curvature below 1e-6 of the slope's terms)."""
    dy, h, gamma, _, _ = grad_inputs(shape, False)
    y, _, rstd = lpq.lpq_rmsnorm(h, gamma, EPS)
    dx, dg = lpq.lpq_rmsnorm_backward(dy, h, gamma, rstd)
    rng = np.random.default_rng(8)
    hh, ga, w = f64(h), f64(gamma), f64(dy)

    def loss(a, b):
        return (w * a / np.sqrt((a * a).mean(1, keepdims=True) + EPS) * b).sum()

    for _ in range(3):
        u, v = rng.standard_normal(hh.shape), rng.standard_normal(ga.shape)
        t = 1e-4
        num = (loss(hh + t * u, ga) - loss(hh - t * u, ga)) / (2 * t)
        terms = np.abs(f64(dx) * u).sum()
        assert abs(num - (f64(dx) * u).sum()) <= (2.0 ** -8 + 1e-4) * terms
        num = (loss(hh, ga + t * v) - loss(hh, ga - t * v)) / (2 * t)
        assert abs(num - (f64(dg) * v).sum()) <= 1e-4 * np.abs(f64(dg) * v).sum() + 1e-9


def test_side_stream(lpq):
    """Outputs and workspace of a call on another stream are made on that stream."""
    dy, h, gamma, rstd, dres = grad_inputs((700, 2560), True)
    want = lpq.lpq_rmsnorm_backward(dy, h, gamma, rstd, dres=dres)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = []
    for _ in range(4):
        got.append(lpq.lpq_rmsnorm_backward(dy, h, gamma, rstd, dres=dres, stream=s))
        torch.full((8 << 20,), 7.0, device=DEV)   # the current stream takes memory as it becomes free
    torch.cuda.synchronize()
    for dx, dg in got:
        assert torch.equal(dx.view(torch.int16), want[0].view(torch.int16)) and torch.equal(dg, want[1])

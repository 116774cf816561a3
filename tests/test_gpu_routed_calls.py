"""The routed layers' calls as the documentation allows them beside the ordinary run: plans in larger buffers,
plans that lpq_route_plan did not write, and the backward pass of a step down to its tokens."""
import numpy as np
import pytest
import torch

from tests import mx_ref as M
from tests import routed_ref as R
from tests.gpu_util import DEV
from tests.test_gpu_adapters import Case, rounded
from tests.test_gpu_mx_matmul import bound
from tests.test_gpu_mx_routed import many
from tests.test_gpu_rmsnorm import f64
from tests.test_gpu_routed_layer import DIMS, Step, products_ok

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lpq():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import precision_weight_quantization_amd as m
    return m


def test_a_plan_in_larger_buffers(lpq):
    """Its part of them is returned, so that the weight gradients are of its groups and the tokens of its rows."""
    T, k, E = 50, 2, 6
    ids = np.random.default_rng(1).integers(-1, E, (T, k)).astype(np.int32)
    d = torch.from_numpy(ids).to(DEV)
    offsets, rows = (torch.full((n,), 77, dtype=torch.int32, device=DEV) for n in (40, 300))
    off, at, src = lpq.lpq_route_plan(d, E, 32, offsets=offsets, rows=rows)
    for got, want in zip((off, at, src), R.plan(ids, E, 32)):
        assert np.array_equal(got.cpu().numpy(), want)
    assert bool((offsets[E + 1:] == 77).all()) and bool((rows[T * k:] == 77).all())
    (a, ae, va), (b, be, vb) = many(48, src.numel(), M.FP8, 3), many(80, src.numel(), M.FP8, 4)
    y = lpq.lpq_mx_matmul_routed_dw(a, ae, b, be, off)
    assert y.shape == (E, 48, 80)
    for g in range(E):
        r = slice(int(off[g]), int(off[g + 1]))
        exact = va[:, r] @ vb[:, r].T
        assert bool(((y[g].double() - exact).abs() <= bound(va[:, r], vb[:, r], exact, (M.FP8, M.FP8), False)).all())
    x = torch.randn((src.numel(), 64), device=DEV).to(torch.bfloat16)
    assert torch.equal(lpq.lpq_route_combine(x, at), lpq.lpq_route_combine(x, lpq.lpq_route_plan(d, E, 32)[1]))


def test_groups_that_overlap(lpq):
    """Offsets of no plan, every other group with all the rows: their tiles together are more than 2^32, and no place
    that a workgroup finds may lie outside the buffers.  The launch has a tile for every row and one for each group
    more; those beyond the first group's go over the first rows again."""
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GiB of device memory")
    R, N, K, E = 5 << 26, 16, 32, 1024
    assert R // 32 * (E // 2) > 1 << 32
    (a, ae, va), (b, be, vb) = many(64, K, M.FP4, 5), many(E * N, K, M.FP4, 6)
    a, ae = a.repeat(R // 64, 1), ae.repeat(R // 64, 1)
    offsets = torch.tensor([0, R] * (E // 2) + [0], dtype=torch.int32, device=DEV)
    buf = torch.full((R * N + 512,), 5.0, dtype=torch.bfloat16, device=DEV)
    lpq.lpq_mx_matmul_routed(a, ae, b.view(E, N, -1), be.view(E, N, -1), offsets, y=buf)
    assert bool((buf[R * N:] == 5).all())
    exact = va @ vb[:N].T
    y = buf[:R * N].view(-1, 64, N)
    first = y[E * 32 // 64]   # behind what the second group goes over
    assert bool(((first.double() - exact).abs() <= bound(va, vb[:N], exact, (M.FP4, M.FP4), False)).all())
    assert bool((y[E * 32 // 64:] == first).all())


def guarded(shape, dtype):
    """A buffer with 512 elements behind it, and the part in front of them."""
    n = int(np.prod(shape))
    b = torch.full((n + 512,), 5, dtype=dtype, device=DEV)
    return b, b[:n].view(shape)


@pytest.mark.parametrize("shape", [(60, 4, 16, 136, 264), (500, 3, 72, 264, 136)])
def test_adapters_keep_to_their_buffers(lpq, shape):
    """Offsets, rows and tokens that no plan holds: nothing behind any output or the workspace is written."""
    T, L, r, N, K = shape
    c = Case(lpq, shape)
    off, rows, src = (t.clone() for t in c.plan)
    for change in range(3):
        if change == 0:
            off[1], off[3] = 1 << 30, -7
        elif change == 1:
            src[:T // 2:3], rows[:T // 3:2] = 1 << 30, 1 << 29
            src[1], rows[1] = -5, -(1 << 31)
        else:   # every group has all the rows, every row the same token
            off[:] = torch.tensor([0, T] * L, device=DEV)[:L + 1]
            src[:] = T - 1
        c.plan = off, rows, src
        y, at = guarded((T, N), torch.bfloat16)
        dims = T, T, L, r, N, K
        ws, w = guarded((lpq.raw().lpq_adapters_workspace(*dims),), torch.uint8)
        c.forward(lpq, y=at, workspace=w)
        assert bool((y[-512:] == 5).all()) and bool((ws[-512:] == 5).all())
        outs = [guarded(s, t) for s, t in (((T, K), torch.bfloat16), ((L, r, K), torch.float32), ((L, N, r), torch.float32),
                                           ((lpq.raw().lpq_adapters_backward_workspace(*dims),), torch.uint8))]
        (_, dx), (_, dA), (_, dB), (_, w) = outs
        for more in (False, True):
            c.backward(lpq, dx=dx, dA=dA, dB=dB, workspace=w, accumulate=more)
            assert all(bool((b[-512:] == 5).all()) for b, _ in outs)


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_not_finite_in_the_adapters_own_results(lpq, value):
    """What an adapter's dy, tokens or factors hold does show in its own gradients."""
    T, L, r, N, K = shape = (100, 7, 16, 264, 520)
    ids = np.random.default_rng(9).integers(-1, L, T)
    bad = torch.from_numpy(ids == 3).to(DEV)
    # an input that is not finite in all of a group, and the gradients that every element of it is a term of
    for where, shows in (("x", "AB"), ("dy", "xAB"), ("A", "xB"), ("B", "xA"), ("scale", "xAB")):
        c = Case(lpq, shape, spread=ids)
        if where in ("x", "dy"):
            getattr(c, where)[bad] = value
        else:
            getattr(c, where)[3] = value
        gx, gA, gB = c.backward(lpq)
        for name, g in (("x", gx[bad]), ("A", gA[3]), ("B", gB[3])):
            assert bool(g.isfinite().any()) == (name not in shows), (where, name)
            assert bool(g.isfinite().all()) == (name not in shows), (where, name)


@pytest.mark.parametrize("dims", DIMS)
def test_a_steps_backward_pass_to_its_tokens(lpq, dims):
    """The gradients of the gate and up projections: through the activation (torch), dx and the weight gradients of the
    grouped product, the gather's gradient into the tokens'; and of the adapters beside the shared projection."""
    T, k, E, D, F, L, r = dims
    s = Step(lpq, dims, 700, known=E + 2)
    o = s.run()
    n = o["src"].numel()
    h = o["h"].float().requires_grad_()
    gate, lin = h.chunk(2, 1)
    (torch.nn.functional.silu(gate) * lin).backward(o["dact"].float())
    dh = h.grad.to(torch.bfloat16)
    o["dht"], o["dhte"], o["dhq"], o["dhqe"] = lpq.lpq_quantize_mxfp8_transposed(dh, rows=True)
    ups = [lpq.lpq_quantize_mxfp8_transposed(w) for w in s.up.view(E, 2 * F, D)]
    o["upt"], o["upte"] = (torch.stack([u[i].view(torch.uint8) for u in ups]) for i in (0, 1))
    o["dxr"] = torch.zeros((n, D), dtype=torch.bfloat16, device=DEV)
    lpq.lpq_mx_matmul_routed(o["dhq"], o["dhqe"], o["upt"], o["upte"], o["offsets"], y=o["dxr"], b_format="mxfp8")
    x = lpq.lpq_route_gather(s.x, o["rows"], o["src"])
    rows, src = o["rows"].cpu().numpy(), o["src"].cpu().numpy()
    assert np.array_equal(f64(x), np.where((src >= 0)[:, None], f64(s.x)[np.maximum(src, 0) // k], 0.0))
    o["xt"], o["xte"], _, _ = lpq.lpq_quantize_mxfp8_transposed(x)
    o["dup"] = lpq.lpq_mx_matmul_routed_dw(o["dht"], o["dhte"], o["xt"], o["xte"], o["offsets"])
    products_ok(o, "dhq", "upt", "dxr", (M.FP8, M.FP8), E)
    products_ok(o, "dht", "xt", "dup", (M.FP8, M.FP8), E, sums=True)
    dx = lpq.lpq_route_combine(o["dxr"], o["rows"], residual=s.dout)   # and the residual stream's own
    exact, size = R.combine(f64(o["dxr"]), rows, np.ones(rows.shape), f64(s.dout))
    tol = (k + 1) * 2.0 ** -24 * size
    assert (np.abs(f64(dx) - exact) <= tol + 2.0 ** -8 * (np.abs(exact) + tol)).all() and np.abs(exact).max() > 0
    ids = s.adapter.cpu().numpy()[:, 0]
    (dx, dA, dB), (sx, sA, sB) = R.adapters_grad(f64(s.dy), f64(s.x), f64(s.A), f64(s.B), ids, f64(s.scale), np.zeros((T, D)))
    most = np.bincount(ids[ids >= 0], minlength=1).max(initial=0)
    assert (np.abs(f64(o["adx"]) - dx) <= rounded(dx, ((F + r + 18) * 2.0 ** -24 + 2.0 ** -16) * sx, sx)).all()
    assert (np.abs(f64(o["dA"]) - dA) <= (F + most + 51) * 2.0 ** -24 * sA).all()
    assert (np.abs(f64(o["dB"]) - dB) <= (D + most + 51) * 2.0 ** -24 * sB).all()

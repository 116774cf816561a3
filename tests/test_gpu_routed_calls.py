"""The routed layers' calls as the documentation allows them beside the ordinary run: plans in larger buffers,
plans that lpq_route_plan did not write."""
import numpy as np
import pytest
import torch

from tests import mx_ref as M
from tests import routed_ref as R
from tests.gpu_util import DEV
from tests.test_gpu_mx_matmul import bound
from tests.test_gpu_mx_routed import many

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

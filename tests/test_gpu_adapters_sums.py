"""Adapters' sums in between: the bits that u and du carry into the second product, and what infinities
and NaN make of them.

Where a test asks for equality every sum in between is exact in FP32, so that the result is the 64-bit one
rounded once; the others take test_gpu_adapters' tolerances."""
import numpy as np
import pytest
import torch

from tests.gpu_util import DEV
from tests.test_gpu_rmsnorm import bf16

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

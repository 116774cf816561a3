"""Calls whose workgroups one launch does not hold (2^32 threads), so that the call makes
two: rows that repeat give results that repeat, past the border between the launches too."""
import pytest
import torch

pytestmark = pytest.mark.gpu

PERIOD = 4096


@pytest.fixture(scope="module")
def lpq():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import precision_weight_quantization_amd as m
    yield m
    torch.cuda.empty_cache()


def room(gib):
    if torch.cuda.mem_get_info()[0] < gib << 30:
        pytest.skip(f"needs {gib} GiB of device memory")


def test_product_of_one_row_and_many_columns(lpq):
    room(12)
    g = torch.Generator(device="cuda").manual_seed(1)
    a, b = (torch.randn((rows, 32), generator=g, device="cuda").bfloat16() for rows in (1, PERIOD))
    a, ae = lpq.lpq_quantize_mxfp8(a)
    b, be = lpq.lpq_quantize_mxfp8(b)
    want = lpq.lpq_mx_matmul(a, ae, b, be).view(-1)
    times = 2 ** 27 // PERIOD + 1   # 2^23 workgroups of 512 threads and more
    b = b.view(torch.uint8).repeat(times, 1).view(torch.float8_e4m3fn)
    y = lpq.lpq_mx_matmul(a, ae, b, be.repeat(times, 1)).view(times, PERIOD)
    assert bool((y == want).all())


def test_norm_of_very_many_rows(lpq):
    room(80)
    g = torch.Generator(device="cuda").manual_seed(2)
    N, times = 288, 2 ** 26 // PERIOD + 1   # 2^24 workgroups of 256 threads and more, 4 rows each
    x = torch.randn((PERIOD, N), generator=g, device="cuda").bfloat16()
    gamma = torch.randn(N, generator=g, device="cuda").bfloat16()
    q, e, _, rstd = lpq.lpq_rmsnorm_mxfp8(x, gamma)
    Q, E, _, R = lpq.lpq_rmsnorm_mxfp8(x.repeat(times, 1), gamma)
    assert bool((R.view(times, PERIOD) == rstd).all())
    assert bool((E.view(times, PERIOD, -1) == e).all())
    assert all(torch.equal(part, q.view(torch.uint8)) for part in Q.view(torch.uint8).view(times, PERIOD, N)[::64])
    assert torch.equal(Q.view(torch.uint8)[-PERIOD:], q.view(torch.uint8))

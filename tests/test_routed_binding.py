"""What lpq_route_plan returns of the buffers that it is given (CPU: the runtime's and the library's calls are replaced)."""
import pytest
import torch

import precision_weight_quantization_amd as lpq
from tests.test_launch_device import runtime  # noqa: F401  (fixture)
from tests.test_routed_abi import I32, on1


class Library:
    def __getattr__(self, fn):
        return lambda *args: 12 if fn == "lpq_route_capacity" else 0


@pytest.mark.parametrize("offsets,rows", [((5,), (6, 2)), ((9,), (12,)), ((1024,), (7, 2)), ((3, 2), (4, 4)), ((5,), (2, 6)), ((8,), (40,))])
@pytest.mark.parametrize("ids", [(6, 2), (12,)])
def test_the_plans_part_of_larger_buffers(runtime, monkeypatch, offsets, rows, ids):  # noqa: F811
    """Calls that read a plan take groups, tokens and slots from its shapes."""
    monkeypatch.setattr(lpq, "_L", Library())
    o, r, s = on1(I32, *offsets), on1(I32, *rows), on1(I32, 12)
    got = lpq.lpq_route_plan(on1(I32, *ids), 4, offsets=o, rows=r, src=s)
    assert got[0].shape == (5,) and got[1].shape == ids and got[2] is s
    assert got[0].data_ptr() == o.data_ptr() and got[1].data_ptr() == r.data_ptr()
    assert got[0].is_contiguous() and got[1].is_contiguous()
    if offsets == (5,):
        assert got[0] is o
    if rows == ids:
        assert got[1] is r


@pytest.mark.parametrize("pairs,groups,align", [(8, (1 << 32) + 4, 1), (8, 4 - (1 << 32), 1), (8, 4, (1 << 32) + 1), (8, 4, 1 - (1 << 32)),
                                                ((1 << 64) + 8, 4, 1), (8, 1 << 31, 1)])
def test_sizes_beyond_their_c_types(pairs, groups, align):
    """They are refused, not taken by their low bits."""
    with pytest.raises(ValueError):
        lpq.lpq_route_capacity(pairs, groups, align)
    if pairs < 1 << 40:
        with pytest.raises(ValueError):
            lpq.lpq_route_plan(on1(I32, 4, 2), groups, align)

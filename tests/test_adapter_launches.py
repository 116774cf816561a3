"""The launches of the adapters' calls at the largest shapes: all of a call's below 2^32 threads along each
axis, or the call refused before any of them (CPU: the runtime's launch functions are replaced by a recorder)."""
import json
import subprocess
import sys

import pytest

from tests.test_launch_limits import CHILD, LIBRARY, RECORDER, at


@pytest.fixture(scope="module")
def run(tmp_path_factory):
    so = str(tmp_path_factory.mktemp("record") / "librecord.so")
    subprocess.check_call(["gcc", "-O1", "-Wall", "-Wextra", "-shared", "-fPIC", "-o", so, RECORDER])

    def go(*calls):
        r = subprocess.run([sys.executable, "-c", CHILD, so, LIBRARY, json.dumps(calls)], capture_output=True, text=True, timeout=300)
        assert r.returncode == 0, r.stderr
        return json.loads(r.stdout)

    return go


def forward(T, R, groups, rank, N, K, in_place=False):
    base = at(7)
    return ["lpq_adapters", [at(0), at(1), at(2), at(3), at(4), at(5), at(6), ["i64", T], ["i64", R], ["i", groups], ["i", rank], ["i64", N],
                             ["i64", K], base, base if in_place else at(8), at(9), ["i64", 1 << 43], ["p", 0]], []]


def backward(T, R, groups, rank, N, K):
    return ["lpq_adapters_backward", [at(10), at(0), at(1), at(2), at(3), at(4), at(5), at(6), ["i64", T], ["i64", R], ["i", groups], ["i", rank],
                                      ["i64", N], ["i64", K], at(7), at(8), at(9), at(11), ["i", 0], at(12), ["i64", 1 << 43], ["p", 0]], []]


TOP = 1 << 24
# tokens, capacity, groups, rank, N, K
FIT = [(1, 1, 1, 8, 8, 8), (1 << 17, 1 << 17, 1024, 128, 1 << 18, 1 << 18), (TOP, TOP, 1024, 128, 2048, 2048), (TOP, TOP, 1, 8, 8, 8),
       (1 << 17, 60000, 1024, 64, 1 << 18, 64), (1, TOP, 1, 8, 16384, 16384), (1 << 17, 1 << 17, 1024, 64, 1 << 18, 1 << 18)]
BEYOND = [(1, TOP, 1, 8, 32768, 64), (64, TOP, 1024, 16, 1 << 18, 64), (1 << 17, TOP, 8, 64, 1 << 18, 64), (1, 1 << 23, 1, 8, 1 << 17, 8)]


def launched(o):
    for l in o["launches"]:
        assert all(0 < g < 2 ** 31 and g * b < 2 ** 32 for g, b in zip(l["grid"], l["block"])), l
    return len(o["launches"])


@pytest.mark.parametrize("shape", FIT)
def test_all_launches_hold(run, shape):
    T, R, groups, rank, N, K = shape
    f, g, b = run(forward(*shape), forward(*shape, in_place=True), backward(*shape))
    assert [f["status"], launched(f)] == [0, 2] and [g["status"], launched(g)] == [0, 2]
    if (rank, N, K) == (128, 1 << 18, 1 << 18):   # both factors' transposes: 2^24 workgroups of 256
        assert b["status"] == 2 and b["launches"] == []
    else:
        assert b["status"] == 0 and launched(b) >= 5


@pytest.mark.parametrize("shape", BEYOND)
def test_a_call_that_no_launch_holds_is_refused(run, shape):
    """y's rows by columns; in the backward pass dx's."""
    T, R, groups, rank, N, K = shape
    f, b = run(forward(*shape), backward(T, R, groups, rank, K, N))
    assert f["status"] == 2 and f["launches"] == []
    assert b["status"] == 2 and b["launches"] == []
    import precision_weight_quantization_amd as lpq
    L = lpq.raw()
    assert L.lpq_adapters_workspace(*shape) == 0 and L.lpq_adapters_backward_workspace(T, R, groups, rank, K, N) == 0
    # the other factor's side has no rows of that many columns
    f, = run(forward(T, R, groups, rank, K, N))
    assert f["status"] == 0 and launched(f) == 2

"""The launches of calls at and beyond what one launch may hold: workgroups times threads
stay below 2^32, the runtime's limit along a grid's axis, and what a call covers is covered
once (CPU: the runtime's launch functions are replaced by a recorder)."""
import json
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
RECORDER = os.path.join(ROOT, "tests", "launch_record", "record.c")
LIBRARY = os.path.join(ROOT, "precision_weight_quantization_amd", "liblpq.so")

# In a process of its own: the recorder's names have to be found before the runtime's.
CHILD = r"""
import ctypes, json, struct, sys
rec = ctypes.CDLL(sys.argv[1], mode=ctypes.RTLD_GLOBAL)
lib = ctypes.CDLL(sys.argv[2])

class Launch(ctypes.Structure):
    _fields_ = [("grid", ctypes.c_uint * 3), ("block", ctypes.c_uint * 3), ("args", ctypes.c_ubyte * 256)]

class Tensor(ctypes.Structure):
    _fields_ = [("src", ctypes.c_void_p), ("dst", ctypes.c_void_p), ("scale", ctypes.c_void_p),
                ("rows", ctypes.c_int64), ("cols", ctypes.c_int64), ("group", ctypes.c_int32), ("reserved", ctypes.c_int32)]

launches = (Launch * 4096).in_dll(rec, "record_list")
count = ctypes.c_int.in_dll(rec, "record_count")
sizes = (ctypes.c_int * 8).in_dll(rec, "record_sizes")
i64, vp, i32, f32 = ctypes.c_int64, ctypes.c_void_p, ctypes.c_int, ctypes.c_float
out = []
for name, args, keep in json.loads(sys.argv[3]):
    count.value = 0
    for i in range(8):
        sizes[i] = struct.calcsize(keep[i]) if i < len(keep) else 0
    c = []
    for kind, value in args:
        if kind == "table":
            t = (Tensor * len(value))(*[Tensor(*e) for e in value])
            c.append(t)
        else:
            c.append({"i64": i64, "p": vp, "i": i32, "f": f32}[kind](value))
    fn = getattr(lib, name)
    fn.restype = ctypes.c_int
    status = fn(*c)
    got = []
    for l in launches[:count.value]:
        at, vals = 0, []
        for k in keep:
            vals.append(struct.unpack_from(k, bytes(l.args), at))
            at += struct.calcsize(k)
        got.append({"grid": list(l.grid), "block": list(l.block), "args": vals})
    out.append({"status": status, "launches": got})
print(json.dumps(out))
"""

NORM = "<8Qqif"          # x, residual, gamma, h, y, rstd, q, e; M, N, eps
TRANSPOSE = "<5Q5q"      # w, q, e, qt, et; M, N, Mp, tiles along N, first tile
MATMUL = "<5Q4i"         # a, ae, b, be, y; M, N, K, FP32


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    so = str(tmp_path_factory.mktemp("record") / "librecord.so")
    subprocess.check_call(["gcc", "-O1", "-Wall", "-Wextra", "-shared", "-fPIC", "-o", so, RECORDER])

    def run(*calls):
        r = subprocess.run([sys.executable, "-c", CHILD, so, LIBRARY, json.dumps(calls)], capture_output=True, text=True, timeout=300)
        assert r.returncode == 0, r.stderr
        out = json.loads(r.stdout)
        for o in out:
            for l in o["launches"]:
                assert l["grid"][1:] == [1, 1] and l["block"][1:] == [1, 1]
                assert 0 < l["grid"][0] < 2 ** 31 and l["grid"][0] * l["block"][0] < 2 ** 32, l
        return out

    return run


def at(i):
    """Addresses 2^44 apart: arrays that never overlap, in one order."""
    return ["p", (i + 1) << 44]


def norm_call(M, N, residual=True):
    return ["lpq_rmsnorm_mxfp8",
            [at(0), at(1) if residual else ["p", 0], at(2), ["f", 1e-6], ["i64", M], ["i64", N],
             at(3) if residual else ["p", 0], at(4), at(5), at(6), at(7), ["p", 0]], [NORM]]


# rows of 288 take one wave each, 4 to a workgroup; of 32 four threads, 64 to a workgroup; of 32768 a workgroup
@pytest.mark.parametrize("N,rows,threads", [(288, 4, 256), (32, 64, 256), (32768, 1, 1024)])
def test_norm(plan, N, rows, threads):
    most = (2 ** 32 - 1) // threads * rows
    top = 2 ** 40 // N
    Ms = [M for M in (1, most, most + 1, 2 * most + 5) if M <= top]
    for M, o in zip(Ms, plan(*[norm_call(M, N) for M in Ms])):
        assert o["status"] == 0
        row = 0
        for l in o["launches"]:
            x, res, gamma, h, y, rstd, q, e, m, n, _ = l["args"][0]
            base = [(i + 1) << 44 for i in range(8)]
            assert (n, l["block"][0]) == (N, threads) and l["grid"][0] == -(-m // rows)
            assert [x, res, gamma] == [base[0] + 2 * N * row, base[1] + 2 * N * row, base[2]]
            assert [h, rstd, y] == [base[3] + 2 * N * row, base[4] + 4 * row, base[5] + 2 * N * row]
            assert [q, e] == [base[6] + N * row, base[7] + N // 32 * row]
            row += m
        assert row == M and len(o["launches"]) == -(-M // most)
    # arrays that are not there stay away in every launch
    if most + 1 <= top:
        for l in plan(norm_call(most + 1, N, residual=False))[0]["launches"]:
            assert l["args"][0][1] == 0 and l["args"][0][3] == 0


@pytest.mark.parametrize("name", ["lpq_quantize_mxfp8_transposed", "lpq_quantize_mxfp4_transposed"])
def test_transpose(plan, name):
    most = (2 ** 32 - 1) // 256   # tiles of 128 x 128 a launch
    for M, N, rows in ((1, 32, True), (128 * most, 32, True), (128 * most + 1, 32, True), (128 * most + 1, 32, False), (2 ** 32, 256, True)):
        o, = plan([name, [at(0), ["i64", M], ["i64", N], ["i", 0], at(1) if rows else ["p", 0], at(2) if rows else ["p", 0],
                          at(3), at(4), ["p", 0]], [TRANSPOSE]])
        assert o["status"] == 0
        tile = 0
        for l in o["launches"]:
            v = l["args"][0]
            assert v[0] == 1 << 44 and v[5:8] == [M, N, -(-M // 32) * 32] and v[9] == tile
            tile += l["grid"][0]
        assert tile == -(-M // 128) * -(-N // 128) and len(o["launches"]) == -(-tile // most)


def matmul_call(M, N, K, a=0, b=0):
    return ["lpq_mx_matmul", [at(0), at(1), ["i", a], at(2), at(3), ["i", b], ["i64", M], ["i64", N], ["i64", K], at(4), ["i", 0],
                              ["p", 0]], [MATMUL, "<i", "<i"]]


@pytest.mark.parametrize("a,b", [(0, 0), (0, 1), (1, 0), (1, 1)])
def test_few_rows_product(plan, a, b):
    """Results of 16 columns a workgroup of 512 threads: 2^27 columns are 2^23 workgroups."""
    most = (2 ** 32 - 1) // 512
    for M, N, K, groups in ((1, 16 * most, 32, most), (1, 2 ** 27, 32, 2 ** 23), (16, 2 ** 30, 64, 2 ** 26), (40, 2 ** 30, 32, 2 ** 24),
                            (2 ** 29, 48, 32, 2 ** 23)):
        o, = plan(matmul_call(M, N, K, a, b))
        assert o["status"] == 0, (M, N, K)
        first = 0
        for l in o["launches"]:
            assert l["block"][0] == 512 and l["args"][0][5:8] == [M, N, K] and l["args"][2] == [first]
            first += l["grid"][0]
        assert first == groups and len(o["launches"]) == -(-groups // most)


def test_tile_product_walks_its_tiles(plan):
    """The tile kernel's workgroups go on from tile to tile: one launch of what runs at one time."""
    for call in (matmul_call(2 ** 28, 256, 512), matmul_call(2 ** 18, 2 ** 22, 512)):
        o, = plan(call)
        assert o["status"] == 0 and len(o["launches"]) == 1 and o["launches"][0]["grid"][0] <= 512


FLAT = [("lpq_quantize_mxfp4", 128, 4), ("lpq_quantize_mxfp4_floor", 128, 4), ("lpq_dequantize_mxfp4", 128, 4),
        ("lpq_quantize_mxfp8", 128, 2), ("lpq_dequantize_mxfp8", 256, 2)]


@pytest.mark.parametrize("name,threads,vectors", FLAT)
def test_a_codec_call_that_no_launch_holds_is_refused(plan, name, threads, vectors):
    most = (2 ** 32 - 1) // threads * threads * vectors * 8   # elements of one launch
    call = lambda n: [name, [at(0), *([at(1)] if "dequantize" in name else []), ["i64", n // 32], ["i64", 32],
                             *([] if "dequantize" in name else [at(1)]), at(2), ["p", 0]], []]
    fits, beyond = plan(call(most), call(most + 32))
    assert fits["status"] == 0 and len(fits["launches"]) == 1
    assert beyond["status"] == 2 and beyond["launches"] == []


def test_block_fp8_of_one_column(plan):
    """A column vector has a tile for every 128 elements, with a workgroup of 256 threads or more to it."""
    call = lambda M: ["lpq_quantize_fp8blk", [at(0), ["i64", M], ["i64", 1], at(1), at(2), ["p", 0]], []]
    fits, beyond = plan(call(2 ** 29), call(2 ** 32))
    assert fits["status"] == 0 and len(fits["launches"]) == 1
    assert beyond["status"] == 2 and beyond["launches"] == []


def test_block_fp8_of_narrow_rows(plan):
    """Decoded flat where the layout allows it, whatever the count of tiles."""
    call = lambda M, off=0: ["lpq_dequantize_fp8blk", [["p", (1 << 44) + off], at(1), ["i64", M], ["i64", 64], at(2), ["p", 0]], []]
    flat, unaligned, beyond = plan(call(2 ** 29 + 128), call(2 ** 29 - 128, 1), call(2 ** 29 + 128, 1))
    assert flat["status"] == 0 and len(flat["launches"]) == 1 and flat["launches"][0]["block"][0] == 128
    assert unaligned["status"] == 0 and unaligned["launches"][0]["block"][0] == 1024
    assert beyond["status"] == 2 and beyond["launches"] == []


def test_nothing_is_enqueued_before_a_refusal(plan):
    """An amax pass holds more of a tensor than the encoder behind it; a table's last tensor may be too large."""
    n = 2 ** 39
    o, = plan(["lpq_quantize_nvfp4", [at(0), ["i64", n // 32], ["i64", 32], ["p", 0], at(1), at(2), at(3), ["p", 0]], []])
    assert o["status"] == 2 and o["launches"] == []
    each = [(i + 1) << 44 for i in range(6)]
    table = [[*each[:3], 64, 32, 0, 0], [*each[3:], 2 ** 34, 32, 0, 0]]
    o, = plan(["lpq_quantize_mxfp4_grouped", [["table", table], ["p", 1 << 20], ["i", 2], ["p", 0]], []])
    assert o["status"] == 2 and o["launches"] == []


@pytest.mark.parametrize("name", ["lpq_quantize_mxfp4_grouped", "lpq_mxfp4_qdq_grouped", "lpq_quantize_mxfp8_grouped"])
def test_grouped_calls_split_at_the_limit(plan, name):
    """Six tensors of a third of a launch each: two launches or more, none beyond the limit."""
    rows = 2 ** 36 // 3 // 32
    each = [(i + 1) << 44 for i in range(18)]
    table = [[each[3 * i], each[3 * i + 1], each[3 * i + 2], rows, 32, 0, 0] for i in range(6)]
    o, = plan([name, [["table", table], ["p", 1 << 20], ["i", 6], ["p", 0]], []])
    units = -(-rows * 32 // (2048 if "mxfp8" in name else 4096))
    assert o["status"] == 0 and len(o["launches"]) >= 2 and sum(l["grid"][0] for l in o["launches"]) == 6 * units

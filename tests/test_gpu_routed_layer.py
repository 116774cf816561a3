"""The routed layers' calls together, as a mixture-of-experts layer and a projection with adapters run
them, and under the callers' conditions.

A step: tokens to their experts in MXFP8, gate and up products with MXFP4 weights, the gated
activation (torch), the down product, the weighted combination into the residual stream; the backward pass down to
the tokens' gradient and the experts' weight gradients; and adapters beside a shared projection.
Each call's result is held to the 64-bit formula on the numbers that it was given (the tolerances
of test_gpu_mx_matmul, test_gpu_route and test_gpu_adapters).  Then the step captured into a HIP graph and replayed
with other routings, on side streams, two at once, and from two host threads."""
import threading

import numpy as np
import pytest
import torch

from tests import mx_ref as M
from tests import routed_ref as R
from tests.gpu_util import DEV, host_u8
from tests.test_gpu_adapters import rounded
from tests.test_gpu_mx_matmul import bound
from tests.test_gpu_rmsnorm import bf16, f64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lpq():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import precision_weight_quantization_amd as m
    return m


class Step:
    """Inputs of a step; run() is the step, on the current stream."""

    def __init__(self, lpq, dims, seed, known=None):
        T, k, E, D, F, L, r = self.dims = dims
        self.lpq, self.known = lpq, known or E   # experts that the router knows; E of them are here
        mk = lambda *s: torch.empty(s, dtype=torch.bfloat16, device=DEV)
        self.x, self.res, self.dout, self.dy = mk(T, D), mk(T, D), mk(T, D), mk(T, F)
        self.ids, self.adapter = (torch.empty((T, n), dtype=torch.int32, device=DEV) for n in (k, 1))
        self.weights = torch.empty((T, k), device=DEV)
        self.up, self.down = bf16((E * 2 * F, D), 90, 0.05).to(DEV), bf16((E * D, F), 91, 0.05).to(DEV)
        self.A, self.B = bf16((L, r, D), 92, 0.05).to(DEV), bf16((L, F, r), 93, 0.3).to(DEV)
        self.w = bf16((F, D), 94, 0.05).to(DEV)
        self.scale = torch.linspace(0.5, 2, L, device=DEV)
        self.fill(seed)

    def fill(self, seed):
        T, k, E, D, F, L, r = self.dims
        rng = np.random.default_rng(seed)
        for t, scale in ((self.x, 1.0), (self.res, 2.0), (self.dout, 1e-3), (self.dy, 1e-3)):
            t.copy_(bf16(tuple(t.shape), seed, scale))
            seed += 1
        order = np.argsort(rng.random((T, self.known)) + 0.5 * rng.random(self.known), axis=1)[:, :k]
        self.ids.copy_(torch.from_numpy(order.astype(np.int32)))
        self.adapter.copy_(torch.from_numpy(rng.integers(-1, L, (T, 1)).astype(np.int32)))
        self.weights.copy_(torch.from_numpy(rng.dirichlet(np.ones(k), T).astype(np.float32)))

    def run(self):
        q, (T, k, E, D, F, L, r), o = self.lpq, self.dims, {}
        plan = o["offsets"], o["rows"], o["src"] = q.lpq_route_plan(self.ids, E, 32)
        n = plan[2].numel()
        o["a"], o["ae"] = q.lpq_route_gather_mxfp8(self.x, *plan[1:])
        o["up"], o["upe"] = q.lpq_quantize_mxfp4(self.up)
        o["h"] = torch.zeros((n, 2 * F), dtype=torch.bfloat16, device=DEV)
        q.lpq_mx_matmul_routed(o["a"], o["ae"], o["up"].view(E, 2 * F, -1), o["upe"].view(E, 2 * F, -1), plan[0], y=o["h"])
        gate, lin = o["h"].float().chunk(2, 1)
        act = (torch.nn.functional.silu(gate) * lin).to(torch.bfloat16)
        o["act"], o["acte"] = q.lpq_quantize_mxfp8(act)
        o["down"], o["downe"] = q.lpq_quantize_mxfp4(self.down)
        o["y"] = torch.zeros((n, D), dtype=torch.bfloat16, device=DEV)
        q.lpq_mx_matmul_routed(o["act"], o["acte"], o["down"].view(E, D, -1), o["downe"].view(E, D, -1), plan[0], y=o["y"])
        o["out"] = q.lpq_route_combine(o["y"], plan[1], self.weights, residual=self.res)
        # backward: dy, dweights; d act = dy down; d down = dy^T act; the gradient of a gather
        o["dyr"], o["dw"] = q.lpq_route_combine_backward(self.dout, *plan[1:], self.weights, y=o["y"])
        o["dyt"], o["dyte"], o["dyq"], o["dyqe"] = q.lpq_quantize_mxfp8_transposed(o["dyr"], rows=True)
        o["actt"], o["actte"], _, _ = q.lpq_quantize_mxfp8_transposed(act)
        dt = [q.lpq_quantize_mxfp8_transposed(w) for w in self.down.view(E, D, F)]
        o["downt"], o["downte"] = (torch.stack([d[i].view(torch.uint8) for d in dt]) for i in (0, 1))
        o["dact"] = torch.zeros((n, F), dtype=torch.bfloat16, device=DEV)
        q.lpq_mx_matmul_routed(o["dyq"], o["dyqe"], o["downt"], o["downte"], plan[0], y=o["dact"], b_format="mxfp8")
        o["ddown"] = q.lpq_mx_matmul_routed_dw(o["dyt"], o["dyte"], o["actt"], o["actte"], plan[0])
        o["dx"] = q.lpq_route_combine(o["y"], plan[1])
        # a shared projection with adapters
        aplan = q.lpq_route_plan(self.adapter, L)
        o["base"] = q.lpq_mx_matmul(*q.lpq_quantize_mxfp8(self.x), *q.lpq_quantize_mxfp4(self.w))
        o["proj"] = q.lpq_adapters(self.x, self.A, self.B, *aplan, scale=self.scale, base=o["base"])
        o["adx"], o["dA"], o["dB"] = q.lpq_adapters_backward(self.dy, self.x, self.A, self.B, *aplan, scale=self.scale)
        return o


def held(codes, scales, fmt):
    c, e = host_u8(codes), host_u8(scales)
    c, e = c.reshape(-1, c.shape[-1]), e.reshape(-1, e.shape[-1])
    return M.values(M.unpack(c) if fmt == M.FP4 else c, e, fmt)


def products_ok(o, a, b, y, fmts, groups, sums=False):
    """Each group's product against the 64-bit one of its operands."""
    va, vb = held(o[a], o[a + "e"], fmts[0]), held(o[b], o[b + "e"], fmts[1])
    off, out = o["offsets"].tolist(), f64(o[y])
    rows = len(vb) // groups
    for g in range(groups):
        r = slice(off[g], off[g + 1])
        pa, pb = (va[:, r], vb[:, r]) if sums else (va[r], vb[g * rows:(g + 1) * rows])
        exact = pa @ pb.T
        if exact.size and pa.shape[1]:
            assert (np.abs((out[g] if sums else out[r]) - exact) <= bound(pa, pb, exact, fmts, False).numpy()).all(), (y, g)


def same(a, b):
    return [k for k in a if not torch.equal(a[k].contiguous().view(torch.uint8), b[k].contiguous().view(torch.uint8))]


# tokens, slots, experts, width, hidden width, adapters, rank
DIMS = [(40, 2, 6, 96, 64, 3, 8), (300, 4, 16, 544, 288, 5, 16), (1, 2, 8, 256, 160, 2, 16), (900, 2, 4, 512, 256, 2, 32)]


@pytest.mark.parametrize("dims", DIMS)
def test_layer(lpq, dims):
    T, k, E, D, F, L, r = dims
    s = Step(lpq, dims, 100, known=E + 2)
    o = s.run()
    for g, w in zip((o["offsets"], o["rows"], o["src"]), R.plan(s.ids.cpu().numpy(), E, 32)):
        assert np.array_equal(g.cpu().numpy(), w)
    products_ok(o, "a", "up", "h", (M.FP8, M.FP4), E)
    products_ok(o, "act", "down", "y", (M.FP8, M.FP4), E)
    products_ok(o, "dyq", "downt", "dact", (M.FP8, M.FP8), E)
    products_ok(o, "dyt", "actt", "ddown", (M.FP8, M.FP8), E, sums=True)
    rows, src, w = o["rows"].cpu().numpy(), o["src"].cpu().numpy(), f64(s.weights)
    for got, weights, res in ((o["out"], w, f64(s.res)), (o["dx"], np.ones_like(w), np.zeros((T, D)))):
        exact, size = R.combine(f64(o["y"]), rows, weights, res)
        tol = (k + 1) * 2.0 ** -24 * size
        assert (np.abs(f64(got) - exact) <= tol + 2.0 ** -8 * (np.abs(exact) + tol)).all()
    dy, dw, size = R.combine_grad(f64(s.dout), f64(o["y"]), rows, src, w)
    assert (np.abs(f64(o["dyr"]) - dy) <= (2.0 ** -24 + 2.0 ** -8) * np.abs(dy) + 2.0 ** -134).all()
    assert (np.abs(f64(o["dw"]) - dw) <= D * 2.0 ** -24 * size).all()
    exact, size = R.adapters(f64(s.x), f64(s.A), f64(s.B), s.adapter.cpu().numpy()[:, 0], f64(s.scale), f64(o["base"]))
    assert (np.abs(f64(o["proj"]) - exact) <= rounded(exact, ((D + r + 18) * 2.0 ** -24 + 2.0 ** -16) * size, size)).all()


@pytest.mark.parametrize("dims", DIMS[:3])
def test_graph(lpq, dims):
    """One capture, replayed with other tokens and other routings, other eager work in between."""
    s = Step(lpq, dims, 200)
    s.run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = s.run()
    for t in range(4):
        s.fill(210 + 10 * t)
        torch.zeros(1 << 16, device=DEV).sum().item()
        graph.replay()
        torch.cuda.synchronize()
        got = {k: v.clone() for k, v in captured.items()}
        assert same(got, s.run()) == [], t


def test_two_graphs_of_one_workspace(lpq):
    """Plans and adapters' gradients that share a workspace, captured apart and replayed in turn."""
    dims = [(9000, 3, 8, 64, 64, 4, 16), (700, 2, 8, 64, 64, 4, 16)]
    steps = [Step(lpq, d, 300 + 10 * i) for i, d in enumerate(dims)]
    work = torch.empty(1 << 26, dtype=torch.uint8, device=DEV)

    def run(s, workspace):
        plan = lpq.lpq_route_plan(s.ids, s.dims[2], workspace=workspace)
        aplan = lpq.lpq_route_plan(s.adapter, s.dims[5], workspace=workspace)
        y = lpq.lpq_adapters(s.x, s.A, s.B, *aplan, workspace=workspace)
        return [*plan, y, *lpq.lpq_adapters_backward(s.dy, s.x, s.A, s.B, *aplan, workspace=workspace)]

    wants = [run(s, None) for s in steps]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for s in steps:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(run(s, work))
        graphs.append(g)
    for _ in range(3):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    for want, out in zip(wants, outs):
        assert all(torch.equal(a, b) for a, b in zip(want, out))


def test_two_streams_at_once(lpq):
    steps = [Step(lpq, DIMS[1], 400), Step(lpq, DIMS[3], 410)]
    want = [s.run() for s in steps]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in steps]
    got = [None, None]
    for _ in range(3):
        for i, s in enumerate(steps):
            with torch.cuda.stream(streams[i]):
                got[i] = s.run()
        torch.cuda.synchronize()
        for w, g in zip(want, got):
            assert same(w, g) == []


def test_two_host_threads(lpq):
    steps = [Step(lpq, DIMS[0], 500), Step(lpq, DIMS[1], 510)]
    want = [s.run() for s in steps]
    torch.cuda.synchronize()
    bad = []

    def work(i):
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(4):
                o = steps[i].run()
                torch.cuda.current_stream().synchronize()
                bad.extend(same(want[i], o))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert bad == []


def test_stream_argument(lpq):
    """A call given a stream by object or by handle runs and allocates there."""
    s = Step(lpq, DIMS[1], 600)
    want = s.run()
    T, k, E, D, F, L, r = s.dims
    b, be = want["up"].view(E, 2 * F, -1), want["upe"].view(E, 2 * F, -1)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream, 0):
        off, rows, src = lpq.lpq_route_plan(s.ids, E, 32, stream=stream)
        a, ae = lpq.lpq_route_gather_mxfp8(s.x, rows, src, stream=stream)
        h = lpq.lpq_mx_matmul_routed(a, ae, b, be, off, stream=stream)
        out = lpq.lpq_route_combine(want["y"], rows, s.weights, residual=s.res, stream=stream)
        dyr, dw = lpq.lpq_route_combine_backward(s.dout, rows, src, s.weights, y=want["y"], stream=stream)
        dd = lpq.lpq_mx_matmul_routed_dw(want["dyt"], want["dyte"], want["actt"], want["actte"], off, stream=stream)
        torch.cuda.synchronize()
        last = int(off[-1])
        assert torch.equal(off, want["offsets"]) and torch.equal(src, want["src"]) and torch.equal(ae, want["ae"])
        assert torch.equal(h[:last], want["h"][:last]) and torch.equal(out, want["out"])
        assert torch.equal(dyr, want["dyr"]) and torch.equal(dw, want["dw"]) and torch.equal(dd, want["ddown"])

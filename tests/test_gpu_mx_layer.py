"""The microscaled operators together, as a layer runs them, and under the callers' conditions.

A layer's step: the norm of the residual stream with MXFP8 output, the product with MXFP4
weights, and the backward pass: both gradient products from the two-way quantizer's forms, then
the norm's gradients.  Each product is held to the 64-bit product of the numbers that its own
quantized operands stand for (the tolerance of one product, as derived in test_gpu_mx_matmul),
the norm's gradients to the formula's.  Then the same step captured once into a HIP graph and
replayed with new inputs, other eager work between the replays; on side streams, two at once; and
from two host threads."""
import threading

import numpy as np
import pytest
import torch

from tests import mx_ref as R
from tests.gpu_util import DEV, host_u8
from tests.test_gpu_mx_matmul import bound
from tests.test_gpu_rmsnorm import EPS, bf16, f64, grad_ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lpq():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import precision_weight_quantization_amd as m
    return m


class Step:
    """Inputs of one layer's step; run() is the step, on the current stream."""

    def __init__(self, lpq, M, N, K, seed):
        self.lpq, self.dims = lpq, (M, N, K)
        self.x, self.res, self.dy = (torch.empty((M, w), dtype=torch.bfloat16, device=DEV) for w in (K, K, N))
        self.gamma = (1 + 0.2 * bf16((K,), 90).float()).to(torch.bfloat16).to(DEV)
        self.w = bf16((N, K), 91, 0.02).to(DEV)
        self.fill(seed)

    def fill(self, seed):
        M, N, K = self.dims
        self.x.copy_(bf16((M, K), seed, outliers=1e-3))
        self.res.copy_(bf16((M, K), seed + 1, 2.0))
        self.dy.copy_(bf16((M, N), seed + 2, 1e-3))

    def run(self):
        L, y = self.lpq, torch.empty_like(self.x)
        wp, we = L.lpq_quantize_mxfp4(self.w)
        q, e, h, rstd = L.lpq_rmsnorm_mxfp8(self.x, self.gamma, EPS, residual=self.res, y=y)
        out = L.lpq_mx_matmul(q, e, wp, we)
        # backward: dx = dy w, dw = dy^T y, contracted over N and over the tokens
        wt, wte, _, _ = L.lpq_quantize_mxfp8_transposed(self.w)
        dyt, dyte, dyq, dye = L.lpq_quantize_mxfp8_transposed(self.dy, rows=True)
        yt, yte, _, _ = L.lpq_quantize_mxfp8_transposed(y)
        dnorm = L.lpq_mx_matmul(dyq, dye, wt, wte)
        dw = L.lpq_mx_matmul(dyt, dyte, yt, yte)
        dh, dgamma = L.lpq_rmsnorm_backward(dnorm, h, self.gamma, rstd)
        return dict(q=q, e=e, h=h, rstd=rstd, wp=wp, we=we, out=out, wt=wt, wte=wte, dyt=dyt, dyte=dyte, dyq=dyq, dye=dye,
                    yt=yt, yte=yte, dnorm=dnorm, dw=dw, dh=dh, dgamma=dgamma)


def held(codes, scales, fmt):
    c = host_u8(codes)
    return R.values(R.unpack(c) if fmt == R.FP4 else c, host_u8(scales), fmt)


def product_ok(r, a, ae, b, be, out, fmts):
    va, vb = held(r[a], r[ae], fmts[0]), held(r[b], r[be], fmts[1])
    exact = va @ vb.T
    err = np.abs(r[out].double().cpu().numpy() - exact)
    assert (err <= bound(va, vb, exact, fmts, False).numpy()).all(), out


def same(a, b):
    return [k for k in a if not torch.equal(a[k].contiguous().view(torch.uint8), b[k].contiguous().view(torch.uint8))]


@pytest.mark.parametrize("dims", [(40, 96, 64), (77, 160, 2560), (300, 512, 1056), (768, 1024, 768), (1100, 1280, 1056)])
def test_layer(lpq, dims):
    s = Step(lpq, *dims, 100)
    r = s.run()
    product_ok(r, "q", "e", "wp", "we", "out", (R.FP8, R.FP4))
    product_ok(r, "dyq", "dye", "wt", "wte", "dnorm", (R.FP8, R.FP8))
    product_ok(r, "dyt", "dyte", "yt", "yte", "dw", (R.FP8, R.FP8))
    dx, dg, tol_dx, tol_dg = grad_ref(r["dnorm"], r["h"], s.gamma, r["rstd"], None)
    assert (np.abs(f64(r["dh"]) - dx) <= tol_dx).all() and (np.abs(f64(r["dgamma"]) - dg) <= tol_dg).all()


@pytest.mark.parametrize("dims", [(77, 160, 2560), (1100, 1280, 1056)])
def test_graph(lpq, dims):
    s = Step(lpq, *dims, 200)
    s.run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = s.run()
    for t in range(4):
        s.fill(210 + 10 * t)
        torch.zeros(1 << 16, device=DEV).sum().item()   # other eager work and a synchronisation
        graph.replay()
        torch.cuda.synchronize()
        got = {k: v.clone() for k, v in captured.items()}
        assert same(got, s.run()) == [], t


def test_two_graphs_of_one_workspace(lpq):
    """Two captured gradients that were given the same workspace, replayed in turn on one stream."""
    dims = [(700, 2560), (3000, 128)]
    need = max(lpq.lpq_rmsnorm_backward_workspace(*d) for d in dims)
    work = torch.empty(need, dtype=torch.uint8, device=DEV)
    graphs, wants, outs = [], [], []
    for i, (M, K) in enumerate(dims):
        dy, h = bf16((M, K), 300 + i, 1e-3).to(DEV), bf16((M, K), 310 + i).to(DEV)
        gamma, rstd = torch.ones(K, dtype=torch.bfloat16, device=DEV), torch.rand(M, device=DEV) + 0.5
        wants.append(lpq.lpq_rmsnorm_backward(dy, h, gamma, rstd))
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(lpq.lpq_rmsnorm_backward(dy, h, gamma, rstd, workspace=work) + (dy, h, gamma, rstd))
        graphs.append(g)
    for _ in range(3):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    for (dx, dg), o in zip(wants, outs):
        assert torch.equal(dx.view(torch.int16), o[0].view(torch.int16)) and torch.equal(dg, o[1])


def test_two_streams_at_once(lpq):
    steps = [Step(lpq, 77, 160, 2560, 400), Step(lpq, 1100, 1280, 1056, 410)]
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
    steps = [Step(lpq, 1030, 1120, 320, 500), Step(lpq, 300, 512, 1056, 510)]
    want = [s.run() for s in steps]
    torch.cuda.synchronize()
    bad = []

    def work(i):
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(5):
                r = steps[i].run()
                torch.cuda.current_stream().synchronize()
                bad.extend(same(want[i], r))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert bad == []


def test_stream_argument(lpq):
    """A call given a stream by object or by handle runs and allocates there."""
    s = Step(lpq, 130, 256, 1056, 600)
    a = lpq.lpq_quantize_mxfp8(s.x)
    b = lpq.lpq_quantize_mxfp4(s.w)
    want = lpq.lpq_mx_matmul(*a, *b)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream, 0):   # 0: the default stream
        b2 = lpq.lpq_quantize_mxfp4(s.w, stream=stream)
        q2 = lpq.lpq_rmsnorm_mxfp8(s.x, s.gamma, stream=stream)
        y2 = lpq.lpq_mx_matmul(*a, *b2, stream=stream)
        t2 = lpq.lpq_quantize_mxfp4_transposed(s.w, rows=True, stream=stream)
        d2 = lpq.lpq_dequantize_mxfp4(*b2, stream=stream)
        torch.cuda.synchronize()
        assert torch.equal(y2.view(torch.int16), want.view(torch.int16))
        assert torch.equal(t2[2], b[0]) and torch.equal(t2[3], b[1])
        assert torch.equal(d2, lpq.lpq_mxfp4_qdq(s.w))
        ref = lpq.lpq_rmsnorm_mxfp8(s.x, s.gamma)
        assert torch.equal(q2[0].view(torch.uint8), ref[0].view(torch.uint8))

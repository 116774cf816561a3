"""Operators of layers whose rows go to different weights, as workloads to time and compare.

A mixture-of-experts layer in microscaled formats, and low-rank adapters beside a shared
projection.  Both order the tokens by the weight that each goes to and run one product per
run of rows:

* ``dispatch``   expert indexes -> the rows of each expert (offsets, places), and the tokens'
                 MXFP8 or MXFP4 form in that order;
* ``experts``    products grouped by expert, y[r] = a[r] b[expert of r]^T, ragged row counts;
* ``experts_grad``  their weight gradients, dw[e] = sum over the expert's rows of dy^T x;
* ``combine``    the weighted sum of each token's expert outputs, and its backward pass;
* ``adapters``   y = base + s_g (x A_g^T) B_g^T, g the adapter of the token, and its backward pass.

``run`` computes each from elementary torch operations in 32 bits, or, where ``own`` is true,
by the framework's calls.  Values held in 8 or 4 bits come back as the BF16 numbers that they
stand for.
"""
import math

import torch

own = False

DEV = "cuda"
FP8, FP4 = "mxfp8", "mxfp4"

# ----------------------------------------------------------------------------- cases


def listed():
    return [
        # the tokens of a training batch in front of the experts' products; an expert's rows are
        # padded to whole blocks, as the weight gradient needs them
        {"name": "dispatch 8192x8 of 128 fp8 2048", "op": "dispatch", "t": 8192, "k": 8, "groups": 128, "n": 2048, "align": 32,
         "format": FP8, "drop": False},
        # one decoded token on a rank that holds half of the experts, 4-bit activations
        {"name": "dispatch 1x8 of 64 fp4 2048", "op": "dispatch", "t": 1, "k": 8, "groups": 64, "n": 2048, "align": 1,
         "format": FP4, "drop": True},
        # gate and up projections of a training batch or a long prompt, 8-bit operands
        {"name": "experts fp8 8192x8 of 128 1536x2048", "op": "experts", "t": 8192, "k": 8, "groups": 128, "n": 1536, "K": 2048,
         "align": 32, "a": FP8, "b": FP8, "out": "bf16"},
        # the down projection of a decoding batch: few rows an expert, 4-bit weights
        {"name": "experts fp8 fp4 24x8 of 128 2048x768", "op": "experts", "t": 24, "k": 8, "groups": 128, "n": 2048, "K": 768,
         "align": 1, "a": FP8, "b": FP4, "out": "bf16"},
        # a short prompt, sizes that fill no tile, 4-bit operands and an FP32 result
        {"name": "experts fp4 701x6 of 60 1021x1056", "op": "experts", "t": 701, "k": 6, "groups": 60, "n": 1021, "K": 1056,
         "align": 1, "a": FP4, "b": FP4, "out": "f32"},
        # the weight gradient of the gate and up projections over a training batch
        {"name": "experts grad fp8 8192x8 of 128 1536x2048", "op": "experts_grad", "t": 8192, "k": 8, "groups": 128, "n": 1536,
         "K": 2048, "a": FP8, "b": FP8, "out": "bf16"},
        # a small batch over many experts, some without a token; 4-bit operands, FP32 gradients
        {"name": "experts grad fp4 157x4 of 96 520x776", "op": "experts_grad", "t": 157, "k": 4, "groups": 96, "n": 520, "K": 776,
         "a": FP4, "b": FP4, "out": "f32"},
        # the experts' outputs of a training batch back into the residual stream
        {"name": "combine 8192x8 2048", "op": "combine", "t": 8192, "k": 8, "groups": 128, "n": 2048, "align": 1,
         "residual": True, "drop": False, "backward": False},
        # its backward pass on a rank that holds half of the experts: gradients of the outputs and weights
        {"name": "combine grad 1237x6 7168", "op": "combine", "t": 1237, "k": 6, "groups": 64, "n": 7168, "align": 32,
         "residual": False, "drop": True, "backward": True},
        # prompts of a few requests, each with its own adapter, through a gate projection
        {"name": "adapters 8192 of 8 9728x2560 rank 64", "op": "adapters", "t": 8192, "groups": 8, "n": 9728, "K": 2560, "rank": 64,
         "backward": False},
        # one decoding step of many requests, nearly every one with another adapter
        {"name": "adapters 40 of 32 4096x2560 rank 16", "op": "adapters", "t": 40, "groups": 32, "n": 4096, "K": 2560, "rank": 16,
         "backward": False},
        # fine-tuning several adapters in one batch: gradients of the input and of both factors
        {"name": "adapters grad 4099 of 4 1024x2560 rank 24", "op": "adapters", "t": 4099, "groups": 4, "n": 1024, "K": 2560,
         "rank": 24, "backward": True},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["dispatch", "experts", "experts", "experts_grad", "combine", "adapters", "adapters"])
    groups = _log_int(rng, 2, 256)
    k = rng.randint(1, min(8, groups))
    if op == "dispatch":
        n = 32 * _log_int(rng, 2, 224)
        return {"op": op, "t": _log_int(rng, 1, min(16384, 8192 * 8 * 2048 // (k * n))), "k": k, "groups": groups, "n": n,
                "align": rng.choice([1, 32]), "format": rng.choice([FP8, FP4]), "drop": rng.random() < 0.3}
    if op == "combine":
        n, backward = 32 * _log_int(rng, 2, 224), rng.random() < 0.5
        return {"op": op, "t": _log_int(rng, 1, min(16384, 8192 * 8 * 2048 // (k * n * (2 if backward else 1)))), "k": k,
                "groups": groups, "n": n, "align": rng.choice([1, 32]), "residual": not backward and rng.random() < 0.5,
                "drop": rng.random() < 0.3, "backward": backward}
    if op == "adapters":
        n, K, rank = 8 * _log_int(rng, 8, 1216), 8 * _log_int(rng, 8, 1024), 8 * _log_int(rng, 1, 16)
        backward, groups = rng.random() < 0.4, _log_int(rng, 1, 64)
        most = 8192 * (9728 + 2560) * 64 // (3 if backward else 1)
        return {"op": op, "t": _log_int(rng, 1, max(1, min(8192, most // ((n + K) * rank)))), "groups": groups, "n": n, "K": K,
                "rank": rank, "backward": backward}
    n, K = _log_int(rng, 64, 2048), 32 * _log_int(rng, 2, 64)
    groups = min(groups, 128 * 1536 * 2048 // (n * K))
    a, b = rng.choice([(FP8, FP8), (FP8, FP4), (FP4, FP4), (FP4, FP8)])
    case = {"op": op, "t": _log_int(rng, 1, max(1, min(8192, 8192 * 8 * 1536 * 2048 // (k * n * K)))), "k": k, "groups": groups,
            "n": n, "K": K, "a": a, "b": b, "out": rng.choice(["bf16", "f32"]) if a == b == FP4 else "bf16"}
    if op == "experts":
        case["align"] = rng.choice([1, 32])
    else:
        case["n"], case["K"] = -(-n // 8) * 8, K - rng.choice([0, 8, 24])
    return case


def _active(groups, pairs):
    """Groups that an even routing of so many pairs reaches, on average."""
    return groups * (1 - (1 - 1 / groups) ** pairs)


def work(case):
    op, t, n = case["op"], case["t"], case["n"]
    size = {FP8: 1 + 1 / 32, FP4: 1 / 2 + 1 / 32}
    if op == "adapters":
        K, rank = case["K"], case["rank"]
        factors = _active(case["groups"], t) * rank * (n + K)
        if case["backward"]:
            return {"bytes": 2 * t * (n + 3 * K) + (2 + 4) * factors, "flops": 2 * t * rank * (3 * n + 3 * K)}
        return {"bytes": 2 * t * (2 * n + K) + 2 * factors, "flops": 2 * t * rank * (n + K)}
    pairs = t * case["k"]
    if op == "dispatch":
        pairs /= 2 if case["drop"] else 1
        return {"bytes": 2 * t * n + pairs * n * size[case["format"]] + 2 * pairs * n + 16 * t * case["k"], "flops": 4 * t * n}
    if op == "combine":
        pairs /= 2 if case["drop"] else 1
        if case["backward"]:
            return {"bytes": 2 * t * n + 4 * pairs * n + 12 * t * case["k"], "flops": 3 * pairs * n}
        return {"bytes": 2 * t * n * (2 if case["residual"] else 1) + 2 * pairs * n + 8 * t * case["k"], "flops": 2 * pairs * n}
    K, out = case["K"], 2 if case["out"] == "bf16" else 4
    if op == "experts":
        return {"bytes": pairs * K * size[case["a"]] + _active(case["groups"], pairs) * n * K * size[case["b"]] + pairs * n * out,
                "flops": 2 * pairs * n * K}
    return {"bytes": pairs * (n * size[case["a"]] + K * size[case["b"]]) + case["groups"] * n * K * out, "flops": 2 * pairs * n * K}


# ----------------------------------------------------------------------------- inputs


def _activations(g, m, n):
    """Unit-variance activations with one value in a few thousand far out, and a few strong channels."""
    x = torch.randn((m, n), generator=g, device=DEV)
    x = torch.where(torch.rand((m, n), generator=g, device=DEV) < 3e-4, x * 30, x)
    return (x * torch.exp(0.3 * torch.randn((n,), generator=g, device=DEV))).to(torch.bfloat16)


def _routing(g, t, k, groups, drop):
    """Expert indexes of k experts a token, some experts liked more than others, and the router's
    weights.  ``drop``: the router knows twice as many experts as this rank holds."""
    known = 2 * groups if drop else groups
    logits = torch.randn((t, known), generator=g, device=DEV) + 0.7 * torch.randn((known,), generator=g, device=DEV)
    top, ids = torch.topk(logits, k, dim=1)
    return ids.to(torch.int32), torch.softmax(top, 1)


def _capacity(pairs, groups, align):
    """Rows that hold any routing of so many pairs with each group's rows padded."""
    return -(-(pairs + min(groups, pairs) * (align - 1)) // align) * align


def _plan(ids, groups, align):
    """(offsets [groups + 1], rows like ids, src [capacity]): the rows of each group, padded to
    ``align``, its pairs in their order; the row of each pair (-1: no such group); the pair of each
    row (-1: padding)."""
    flat = ids.reshape(-1).long()
    pairs = flat.numel()
    kept = (flat >= 0) & (flat < groups)
    key = torch.where(kept, flat, groups)
    order = torch.argsort(key, stable=True)
    counts = torch.zeros(groups + 1, dtype=torch.int64, device=DEV).index_add_(0, key, torch.ones_like(key))
    padded = (counts[:groups] + align - 1) // align * align
    zero = torch.zeros(1, dtype=torch.int64, device=DEV)
    offsets = torch.cat([zero, padded.cumsum(0)])
    before = torch.cat([zero, counts.cumsum(0)])   # in sorted order
    rank = torch.empty_like(key)
    rank[order] = torch.arange(pairs, device=DEV) - before[key[order]]
    rows = torch.where(kept, offsets[key] + rank, -1)
    capacity = _capacity(pairs, groups, align)
    src = torch.full((capacity + 1,), -1, dtype=torch.int64, device=DEV)
    src[torch.where(kept, rows, capacity)] = torch.arange(pairs, device=DEV)   # dropped pairs: the place behind
    return offsets.to(torch.int32), rows.reshape(ids.shape).to(torch.int32), src[:capacity].to(torch.int32)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    op, t, groups, n = case["op"], case["t"], case["groups"], case["n"]
    s = {"case": case}
    if op == "adapters":
        K, rank = case["K"], case["rank"]
        ids = torch.randint(0, groups, (t, 1), generator=g, device=DEV, dtype=torch.int32)
        ids = torch.where(torch.rand((t, 1), generator=g, device=DEV) < 0.1, -1, ids)   # requests without an adapter
        s["offsets"], s["rows"], s["src"] = _plan(ids, groups, 1)
        s["bounds"] = s["offsets"].tolist()
        s["x"] = _activations(g, t, K)
        s["A"] = (torch.randn((groups, rank, K), generator=g, device=DEV) / math.sqrt(K)).to(torch.bfloat16)
        s["B"] = (0.3 * torch.randn((groups, n, rank), generator=g, device=DEV)).to(torch.bfloat16)
        s["scale"] = 0.5 + 1.5 * torch.rand((groups,), generator=g, device=DEV)
        if case["backward"]:
            s["dy"] = (1e-3 * torch.randn((t, n), generator=g, device=DEV)).to(torch.bfloat16)
            s["dres"] = (1e-3 * torch.randn((t, K), generator=g, device=DEV)).to(torch.bfloat16)
        else:
            s["base"] = torch.randn((t, n), generator=g, device=DEV).to(torch.bfloat16)
        return s
    drop = case.get("drop", False)
    ids, weights = _routing(g, t, case["k"], groups, drop)
    if op == "dispatch":
        s["ids"], s["x"] = ids, _activations(g, t, n)
        return s
    align = case.get("align", 32)
    s["offsets"], s["rows"], s["src"] = _plan(ids, groups, align)
    capacity, real = s["src"].numel(), (s["src"] >= 0)[:, None]
    if op == "combine":
        s["weights"] = weights
        s["y"] = torch.where(real, _activations(g, capacity, n), 0.0)
        if case["backward"]:
            s["dout"] = (1e-3 * torch.randn((t, n), generator=g, device=DEV)).to(torch.bfloat16)
        else:
            s["residual"] = _activations(g, t, n) if case["residual"] else None
        return s
    K = case["K"]
    s["bounds"] = s["offsets"].tolist()
    out = torch.bfloat16 if case["out"] == "bf16" else torch.float32
    if op == "experts":
        x = torch.where(real, _activations(g, capacity, K), 0.0)
        s["a"], s["ae"] = _codes(x.float(), case["a"])
        w = (0.02 * torch.randn((groups * n, K), generator=g, device=DEV)).to(torch.bfloat16)
        b, be = _codes(w.float(), case["b"])
        s["b"], s["be"] = b.reshape(groups, n, -1), be.reshape(groups, n, -1)
        s["y"] = torch.zeros((capacity, n), dtype=out, device=DEV)   # rows behind the last expert's stay as they are
        return s
    for name, width, scale in (("a", n, 1e-3), ("b", K, 1.0)):
        v = torch.where(real, (scale * _activations(g, capacity, width).float()), 0.0)
        s[name], s[name + "e"] = _codes(v.t().contiguous().to(torch.bfloat16).float(), case[name])
    return s


# ----------------------------------------------------------------------------- the formats, in 32 bits


def _pow2(e):
    """2^e exactly, e an int32 tensor in [-127, 127]: the bits of a binary32 number (2^-127 is subnormal)."""
    return torch.where(e > -127, (e + 127) << 23, 1 << 22).to(torch.int32).view(torch.float32)


def _quantize(v, fmt):
    """(E4M3 values or E2M1 codes [rows, cols], exponents [rows, cols/32]) of 1x32 blocks."""
    b = v.reshape(v.shape[0], -1, 32)
    m, ex = torch.frexp(b.abs().amax(-1))   # amax = m * 2^ex, m in [0.5, 1): the smallest e with amax <= 448 * 2^e or 6 * 2^e
    e = ex - 9 + (m > 0.875) if fmt == FP8 else ex - 3 + (m > 0.75)
    e = torch.where(m == 0, -127, e.clamp(min=-127))
    u = (b * _pow2(-e)[..., None]).reshape(v.shape)
    if fmt == FP8:
        return u.clamp(-448, 448).to(torch.float8_e4m3fn), e
    a = u.abs()   # nearest value, ties to the even code
    c = (a > 0.25).int() + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5)
    return c + 8 * torch.signbit(u), e


def _dequantize(q, e, fmt):
    if fmt == FP8:
        v = q.float()
    else:
        k = q & 7
        v = torch.where(k < 4, 0.5 * k, torch.where(k < 6, k - 2.0, 2.0 * k - 8.0))
        v = torch.where(q >= 8, -v, v)
    return (v.reshape(*e.shape, 32) * _pow2(e)[..., None]).reshape(v.shape)


def _codes(v, fmt):
    """As a program holds them: E4M3 codes or two E2M1 codes to a byte, and the scale bytes."""
    q, e = _quantize(v, fmt)
    if fmt == FP4:
        q = (q[:, 0::2] | (q[:, 1::2] << 4)).to(torch.uint8)
    return q, (e + 127).to(torch.uint8)


def _values(q, e, fmt):
    if fmt == FP4:
        q = q.int()
        q = torch.stack([q & 15, q >> 4], -1).reshape(q.shape[0], -1)
    return _dequantize(q, e.int() - 127, fmt)


# ----------------------------------------------------------------------------- one pass


def run(state):
    if own:
        return _run_own(state)
    case = state["case"]
    op = case["op"]
    if op == "dispatch":
        offsets, rows, src = _plan(state["ids"], case["groups"], case["align"])
        v = _dequantize(*_quantize(state["x"].float(), case["format"]), case["format"])
        token = src.clamp(min=0).long() // case["k"]
        return {"offsets": offsets, "rows": rows, "src": src,
                "x": torch.where((src >= 0)[:, None], v[token], 0.0).to(torch.bfloat16)}
    if op == "combine":
        rows, weights = state["rows"], state["weights"]
        kept = rows >= 0
        if not case["backward"]:
            y = state["y"].float()
            out = state["residual"].float() if case["residual"] else torch.zeros((case["t"], case["n"]), device=DEV)
            for j in range(case["k"]):
                part = weights[:, j, None] * y[rows[:, j].clamp(min=0).long()]
                out = out + torch.where(kept[:, j, None], part, 0.0)
            return {"out": out.to(torch.bfloat16)}
        dout, src = state["dout"].float(), state["src"]
        pair = src.clamp(min=0).long()
        dy = weights.reshape(-1)[pair][:, None] * dout[pair // case["k"]]
        dw = [(dout * state["y"][rows[:, j].clamp(min=0).long()].float()).sum(1) for j in range(case["k"])]
        return {"dy": torch.where((src >= 0)[:, None], dy, 0.0).to(torch.bfloat16),
                "dweights": torch.where(kept, torch.stack(dw, 1), 0.0)}
    if op == "adapters":
        x, A, B, src, bounds = state["x"].float(), state["A"].float(), state["B"].float(), state["src"].long(), state["bounds"]
        runs = [(e, src[bounds[e]:bounds[e + 1]]) for e in range(case["groups"])]
        if not case["backward"]:
            y = state["base"].float()
            for e, token in runs:
                y[token] = y[token] + state["scale"][e] * ((x[token] @ A[e].t()) @ B[e].t())
            return {"y": y.to(torch.bfloat16)}
        dy, dx = state["dy"].float(), state["dres"].float()
        dA, dB = torch.zeros_like(A), torch.zeros_like(B)
        for e, token in runs:
            d = state["scale"][e] * dy[token]
            u, du = x[token] @ A[e].t(), d @ B[e]
            dx[token] = dx[token] + du @ A[e]
            dA[e], dB[e] = du.t() @ x[token], d.t() @ u
        return {"dx": dx.to(torch.bfloat16), "dA": dA, "dB": dB}
    bounds, out = state["bounds"], torch.bfloat16 if case["out"] == "bf16" else torch.float32
    a, ae, b, be = (state[x] for x in ("a", "ae", "b", "be"))
    if op == "experts":
        va = _values(a, ae, case["a"])
        y = torch.zeros((a.shape[0], case["n"]), device=DEV)
        for e in range(case["groups"]):
            lo, hi = bounds[e], bounds[e + 1]
            if hi > lo:
                y[lo:hi] = va[lo:hi] @ _values(b[e], be[e], case["b"]).t()
        return {"y": y.to(out)}
    va, vb = _values(a, ae, case["a"]), _values(b, be, case["b"])
    dw = torch.empty((case["groups"], case["n"], case["K"]), dtype=out, device=DEV)
    for e in range(case["groups"]):
        lo, hi = bounds[e], bounds[e + 1]
        dw[e] = (va[:, lo:hi] @ vb[:, lo:hi].t()).to(out)
    return {"dw": dw}


def _run_own(state):
    import precision_weight_quantization_amd as lpq
    case = state["case"]
    op = case["op"]
    if op == "dispatch":
        offsets, rows, src = lpq.lpq_route_plan(state["ids"], case["groups"], case["align"])
        gather, dequantize = {FP8: (lpq.lpq_route_gather_mxfp8, lpq.lpq_dequantize_mxfp8),
                              FP4: (lpq.lpq_route_gather_mxfp4, lpq.lpq_dequantize_mxfp4)}[case["format"]]
        return {"offsets": offsets, "rows": rows, "src": src, "x": dequantize(*gather(state["x"], rows, src))}
    if op == "combine":
        if not case["backward"]:
            return {"out": lpq.lpq_route_combine(state["y"], state["rows"], state["weights"], residual=state["residual"])}
        dy, dweights = lpq.lpq_route_combine_backward(state["dout"], state["rows"], state["src"], state["weights"], y=state["y"])
        return {"dy": dy, "dweights": dweights}
    if op == "adapters":
        plan = state["offsets"], state["rows"], state["src"]
        if not case["backward"]:
            return {"y": lpq.lpq_adapters(state["x"], state["A"], state["B"], *plan, scale=state["scale"], base=state["base"])}
        dx, dA, dB = lpq.lpq_adapters_backward(state["dy"], state["x"], state["A"], state["B"], *plan, scale=state["scale"],
                                               dres=state["dres"])
        return {"dx": dx, "dA": dA, "dB": dB}
    out = torch.bfloat16 if case["out"] == "bf16" else torch.float32
    operands = state["a"], state["ae"], state["b"], state["be"], state["offsets"]
    if op == "experts":
        return {"y": lpq.lpq_mx_matmul_routed(*operands, out_dtype=out, y=state["y"])}
    return {"dw": lpq.lpq_mx_matmul_routed_dw(*operands, out_dtype=out)}


# ----------------------------------------------------------------------------- the definition, in 64 bits


def _grid(fmt):
    """The non-negative finite values of the format in order of their codes."""
    bits, bias, last = (3, 7, 126) if fmt == FP8 else (1, 1, 7)
    one = 1 << bits
    return [(c % one + one * (c >= one)) / one * 2.0 ** (max(c // one, 1) - bias) for c in range(last + 1)]


def _exact_pow2(e):
    """2^e exactly, e whole numbers in 64 bits: the bits of a binary64 number."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _exact_quantized(v, fmt):
    """The value each element is stored as, from the definition, in 64 bits."""
    grid = torch.tensor(_grid(fmt), dtype=torch.float64, device=DEV)
    b = v.reshape(v.shape[0], -1, 32)
    top = b.abs().amax(-1)
    safe = torch.where(top > 0, top, 1.0)
    e = torch.ceil(torch.log2(safe / grid[-1]))
    e = e + (grid[-1] * _exact_pow2(e) < safe).double()
    e = e - (grid[-1] * _exact_pow2(e - 1) >= safe).double()
    scale = _exact_pow2(torch.where(top > 0, e.clamp(min=-127), -127.0))[..., None]
    u = (b / scale).abs().clamp(max=grid[-1].item())
    lo = (torch.bucketize(u, grid, right=True) - 1).clamp(max=len(grid) - 2)
    below, above = u - grid[lo], grid[lo + 1] - u
    up = (above < below) | ((above == below) & (lo % 2 == 1))
    r = torch.where(up, grid[lo + 1], grid[lo]) * scale
    return torch.where(b < 0, -r, r).reshape(v.shape)


def _exact_values(q, e, fmt):
    grid = torch.tensor(_grid(fmt), dtype=torch.float64, device=DEV)
    if fmt == FP8:
        c = q.view(torch.uint8).long()
        v = grid[c & 127] * (1 - 2 * (c >> 7)).double()
    else:
        c = torch.stack([q & 15, q >> 4], -1).reshape(q.shape[0], -1).long()
        v = grid[c & 7] * (1 - 2 * (c >> 3)).double()
    return v * _exact_pow2(e.long() - 127).repeat_interleave(32, 1)


def exact(case, seed):
    s = prepare(case, seed)
    op, t, groups, n = case["op"], case["t"], case["groups"], case["n"]
    if op == "dispatch":
        # a pair's place from how many pairs before it go to the same expert
        k, align = case["k"], case["align"]
        onehot = (s["ids"].reshape(-1, 1) == torch.arange(groups, device=DEV)).long()
        earlier = ((onehot.cumsum(0) - onehot) * onehot).sum(1)
        padded = -(-onehot.sum(0) // align) * align
        start = padded.cumsum(0) - padded
        row = torch.where(onehot.sum(1) > 0, (onehot * start).sum(1) + earlier, -1)
        capacity = _capacity(t * k, groups, align)
        src = torch.full((capacity,), -1, dtype=torch.int64, device=DEV)
        x = torch.zeros((capacity, n), dtype=torch.float64, device=DEV)
        stored = _exact_quantized(s["x"].double(), case["format"])
        pairs = torch.nonzero(row >= 0)[:, 0]
        src[row[pairs]] = pairs
        x[row[pairs]] = stored[pairs // k]
        return {"offsets": torch.cat([start, padded.sum()[None]]), "rows": row.reshape(t, k), "src": src, "x": x}
    if op == "combine":
        rows, w = s["rows"].reshape(-1).long(), s["weights"].double().reshape(-1)
        pairs = torch.nonzero(rows >= 0)[:, 0]
        token = pairs // case["k"]
        if not case["backward"]:
            out = s["residual"].double() if case["residual"] else torch.zeros((t, n), dtype=torch.float64, device=DEV)
            for j in range(case["k"]):   # a token at most once a slot
                p = pairs[pairs % case["k"] == j]
                out[p // case["k"]] += w[p, None] * s["y"][rows[p]].double()
            return {"out": out}
        dy = torch.zeros((s["src"].numel(), n), dtype=torch.float64, device=DEV)
        dy[rows[pairs]] = w[pairs, None] * s["dout"][token].double()
        dw = torch.zeros_like(w)
        dw[pairs] = (s["dout"][token].double() * s["y"][rows[pairs]].double()).sum(1)
        return {"dy": dy, "dweights": dw.reshape(t, -1)}
    bounds = s["bounds"]
    if op == "adapters":
        x, A, B, scale = s["x"].double(), s["A"].double(), s["B"].double(), s["scale"].double()
        if case["backward"]:
            dx, dA, dB = s["dres"].double(), torch.zeros_like(A), torch.zeros_like(B)
        else:
            y = s["base"].double()
        for e in range(groups):
            token = torch.nonzero((s["rows"][:, 0] >= bounds[e]) & (s["rows"][:, 0] < bounds[e + 1]))[:, 0]
            xe, factor = x[token], scale[e]
            if not case["backward"]:
                y[token] += torch.matmul(xe, (factor * A[e]).t()) @ B[e].t()
                continue
            d = s["dy"][token].double()
            dx[token] += factor * torch.matmul(torch.matmul(d, B[e]), A[e])
            dA[e] = factor * torch.matmul(B[e].t(), torch.matmul(d.t(), xe))
            dB[e] = factor * torch.matmul(torch.matmul(d.t(), xe), A[e].t())
        return {"dx": dx, "dA": dA, "dB": dB} if case["backward"] else {"y": y}
    va = _exact_values(s["a"], s["ae"], case["a"])
    if op == "experts":
        y = torch.zeros((va.shape[0], n), dtype=torch.float64, device=DEV)
        for e in range(groups):
            r = slice(bounds[e], bounds[e + 1])
            y[r] = torch.matmul(va[r], _exact_values(s["b"][e], s["be"][e], case["b"]).t())
        return {"y": y}
    vb = _exact_values(s["b"], s["be"], case["b"])
    return {"dw": torch.stack([torch.matmul(va[:, bounds[e]:bounds[e + 1]], vb[:, bounds[e]:bounds[e + 1]].t()) for e in range(groups)])}

"""Binding of the routed layers' calls: rows that go to different weights.

A plan orders tokens by their group (an expert, an adapter) on the device; the gather,
the products, the combination and the adapters read it there.  The functions are found in
the package under the same names, and follow its manner: device tensors in, outputs
allocated when not passed (on ``stream`` if one is given), launches on the device of the
data.  Indexes are ``torch.int32``.
"""
from __future__ import annotations

import math

import torch

import precision_weight_quantization_amd as _p
from precision_weight_quantization_amd import _bf16_in, _empty, _launch, _on, _ptr

_I32 = (torch.int32,)


def _arg(t, name, like=None, nbytes=0, esize=None, dtypes=None, dims=None):
    """The package's check of an argument, which words the refusal; this one finds out whether there is one
    (lpq_adapters has nine arrays: 17.7 us of the host's time a call, 18.8 without)."""
    if (isinstance(t, torch.Tensor) and t.is_cuda and t.is_contiguous() and (dtypes is None or t.dtype in dtypes)
            and (like is None or t.device == like.device) and (nbytes == 0 or t.nbytes >= nbytes)
            and (esize is None or t.element_size() == esize) and (dims is None or t.dim() == dims)):
        return t
    return _p._arg(t, name, like, nbytes, esize, dtypes, dims)


def _outs(like, *specs):
    """Outputs as the package's _outs makes them."""
    device = like.device
    for t, name, nbytes, _, _, esize in specs:
        if t is not None:
            _arg(t, name, like, nbytes, esize)
    return [t if t is not None else torch.empty(shape, dtype=dtype, device=device) for t, _, _, shape, dtype, _ in specs]


# --------------------------------------------------------------------------- plan

def lpq_route_capacity(pairs: int, groups: int, align: int = 1) -> int:
    """Rows that hold every routing of so many pairs, each group's rows padded to ``align``."""
    # the C call's 32-bit arguments would be the low bits of larger numbers
    n = _p._L.lpq_route_capacity(pairs, groups, align) if 0 < pairs <= 1 << 30 and 0 < groups <= 1024 and 0 < align <= 1024 else 0
    if n == 0:
        raise ValueError(f"no plan of {pairs} pairs over {groups} groups with rows padded to {align}: 1 to 1024 groups, "
                         "1 to 1024 rows, up to 2^30 rows in all")
    return n


def _part(t, shape):
    """The first elements of a buffer that was passed in, in the shape of what the call wrote there."""
    return t if t.shape == shape else t.view(-1)[:math.prod(shape)].view(shape)


def lpq_route_plan(ids, groups, align=1, offsets=None, rows=None, src=None, workspace=None, stream=None):
    """The rows of each group: ids (int32 or int64, [tokens, k] or [tokens]; outside [0, groups): no row) ->
    (offsets [groups+1], rows like ids (-1: none), src [capacity], the pair of each row (-1: padding)), all int32.
    offsets and rows passed in may be larger: what is returned is the part of them that holds the plan.
    A src passed in sets the capacity, at least ``lpq_route_capacity(ids.numel(), groups, align)`` rows."""
    _arg(ids, "ids", dtypes=(torch.int32, torch.int64))
    pairs = ids.numel()
    capacity = lpq_route_capacity(pairs, groups, align)
    need = _p._L.lpq_route_plan_workspace(pairs, groups)
    if src is not None:
        _arg(src, "src", ids, 4 * capacity, dtypes=_I32)
        capacity = src.numel()
    if workspace is not None:
        _arg(workspace, "workspace", ids, need)
    for t, name in ((offsets, "offsets"), (rows, "rows")):
        if t is not None:
            _arg(t, name, ids, dtypes=_I32)
    with _on(stream, ids):
        offsets, rows, src = _outs(ids, (offsets, "offsets", 4 * (groups + 1), (groups + 1,), torch.int32, 4),
                                   (rows, "rows", 4 * pairs, ids.shape, torch.int32, 4),
                                   (src, "src", 4 * capacity, (capacity,), torch.int32, 4))
        if need and workspace is None:
            workspace = _empty((need,), torch.uint8, ids)
    _launch(_p._L.lpq_route_plan, "lpq_route_plan", ids, stream, ids.data_ptr(), ids.element_size(), pairs, groups, align,
            offsets.data_ptr(), rows.data_ptr(), src.data_ptr(), capacity, _ptr(workspace),
            0 if workspace is None else workspace.nbytes)
    # of larger buffers the plan's part: the calls that read a plan take its sizes from these
    return _part(offsets, (groups + 1,)), _part(rows, ids.shape), src


def _tokens(rows, like, tokens=None):
    """(tokens, k) of the rows of a plan, [tokens, k] or [tokens]."""
    _arg(rows, "rows", like, dtypes=_I32)
    if rows.dim() not in (1, 2):
        raise ValueError(f"rows must be [tokens, k] or [tokens], got shape {tuple(rows.shape)}")
    if tokens is not None and rows.shape[0] != tokens:
        raise ValueError(f"rows is of {rows.shape[0]} tokens, the call's data of {tokens}")
    return rows.shape[0], rows.shape[1] if rows.dim() == 2 else 1


# --------------------------------------------------------------------------- gather

def lpq_route_gather(x, rows, src, y=None, stream=None):
    """x [tokens,N] BF16 (N % 32 == 0) in a plan's order: [src.numel(), N] BF16, zeros in rows without a token."""
    x = _bf16_in(x, "x")
    T, N = x.shape
    _, k = _tokens(rows, x, T)
    R = _arg(src, "src", x, dtypes=_I32).numel()
    with _on(stream, x):
        y, = _outs(x, (y, "y", 2 * R * N, (R, N), torch.bfloat16, 2))
    _launch(_p._L.lpq_route_gather, "lpq_route_gather", x, stream, x.data_ptr(), T, N, rows.data_ptr(), k, src.data_ptr(), R,
            y.data_ptr())
    return y


def lpq_route_gather_mxfp8(x, rows, src, q=None, e=None, stream=None):
    """As lpq_route_gather, quantized: (codes [R,N] float8_e4m3fn, UE8M0 bytes [R,N/32] uint8)."""
    x = _bf16_in(x, "x")
    T, N = x.shape
    _, k = _tokens(rows, x, T)
    R = _arg(src, "src", x, dtypes=_I32).numel()
    with _on(stream, x):
        q, e = _outs(x, (q, "q", R * N, (R, N), torch.float8_e4m3fn, 1),
                     (e, "e", R * (N // 32), (R, max(N // 32, 1)), torch.uint8, 1))
    _launch(_p._L.lpq_route_gather_mxfp8, "lpq_route_gather_mxfp8", x, stream, x.data_ptr(), T, N, rows.data_ptr(), k,
            src.data_ptr(), R, q.data_ptr(), e.data_ptr())
    return q, e


def lpq_route_gather_mxfp4(x, rows, src, p=None, e=None, stream=None):
    """As lpq_route_gather, quantized: (packed E2M1 codes [R,N/2] uint8, UE8M0 bytes [R,N/32] uint8)."""
    x = _bf16_in(x, "x")
    T, N = x.shape
    _, k = _tokens(rows, x, T)
    R = _arg(src, "src", x, dtypes=_I32).numel()
    with _on(stream, x):
        p, e = _outs(x, (p, "p", R * (N // 2), (R, max(N // 2, 1)), torch.uint8, 1),
                     (e, "e", R * (N // 32), (R, max(N // 32, 1)), torch.uint8, 1))
    _launch(_p._L.lpq_route_gather_mxfp4, "lpq_route_gather_mxfp4", x, stream, x.data_ptr(), T, N, rows.data_ptr(), k,
            src.data_ptr(), R, p.data_ptr(), e.data_ptr())
    return p, e


# --------------------------------------------------------------------------- products

def _offsets(offsets, like):
    groups = _arg(offsets, "offsets", like, dtypes=_I32, dims=1).numel() - 1
    if groups < 1:
        raise ValueError("offsets holds groups + 1 numbers")
    return groups


def _out_type(out_dtype):
    if out_dtype not in _p._MX_OUT:
        raise TypeError(f"out_dtype must be one of {[str(d) for d in _p._MX_OUT]}, got {out_dtype}")
    return _p._MX_OUT[out_dtype], 4 if out_dtype == torch.float32 else 2


def lpq_mx_matmul_routed(a, ae, b, be, offsets, out_dtype=torch.bfloat16, y=None, a_format=None, b_format=None, stream=None):
    """y [R,N], y[r] = a[r] b[group of r]^T: a [R,K] codes in a plan's order with scale bytes ae, b [groups,N,K] the
    groups' weights with be [groups,N,K/32], offsets [groups+1] the plan's.  Rows of no group are left as they were
    (not set in a y that is allocated here).  Formats and types as in lpq_mx_matmul."""
    fa, R, K = _p._mx_operand(a, ae, a_format, "a")
    groups = _offsets(offsets, a)
    _arg(b, "b", a, esize=1, dims=3)
    if b.shape[0] != groups:
        raise ValueError(f"b holds {b.shape[0]} groups' weights, offsets are of {groups}")
    fb, rows, Kb = _p._mx_operand(b.view(-1, b.shape[2]), be, b_format, "b", a)
    if K != Kb:
        raise ValueError(f"a has {K} columns, b {Kb}")
    N = rows // groups
    kind, size = _out_type(out_dtype)
    with _on(stream, a):
        y, = _outs(a, (y, "y", size * R * N, (R, N), out_dtype, size))
    _launch(_p._L.lpq_mx_matmul_routed, "lpq_mx_matmul_routed", a, stream, a.data_ptr(), ae.data_ptr(), fa, b.data_ptr(),
            be.data_ptr(), fb, offsets.data_ptr(), groups, R, N, K, y.data_ptr(), kind)
    return y


def lpq_mx_matmul_routed_dw(a, ae, b, be, offsets, out_dtype=torch.bfloat16, y=None, a_format=None, b_format=None, stream=None):
    """y [groups,M,N], y[g] = a[:, rows of g] b[:, rows of g]^T: a [M,R] and b [N,R] the transposed forms of gathered
    rows (a plan with align 32), offsets [groups+1] the plan's.  Zeros for a group without rows."""
    fa, M, R = _p._mx_operand(a, ae, a_format, "a")
    fb, N, Rb = _p._mx_operand(b, be, b_format, "b", a)
    if R != Rb:
        raise ValueError(f"a has {R} columns, b {Rb}")
    groups = _offsets(offsets, a)
    kind, size = _out_type(out_dtype)
    with _on(stream, a):
        y, = _outs(a, (y, "y", size * groups * M * N, (groups, M, N), out_dtype, size))
    _launch(_p._L.lpq_mx_matmul_routed_dw, "lpq_mx_matmul_routed_dw", a, stream, a.data_ptr(), ae.data_ptr(), fa, b.data_ptr(),
            be.data_ptr(), fb, offsets.data_ptr(), groups, M, N, R, y.data_ptr(), kind)
    return y


# --------------------------------------------------------------------------- combination

def lpq_route_combine(y, rows, weights=None, residual=None, out=None, stream=None):
    """out [tokens,N] = BF16(residual + sum over j of weights[:, j] * y[rows[:, j]]): y [R,N] BF16, weights like rows
    FP32 (None: ones, the gradient of a gather), residual [tokens,N] BF16 or None (``out`` may be it)."""
    y = _bf16_in(y, "y")
    R, N = y.shape
    T, k = _tokens(rows, y)
    if weights is not None:
        _arg(weights, "weights", y, 4 * T * k, dtypes=(torch.float32,))
    if residual is not None:
        _arg(residual, "residual", y, 2 * T * N, dtypes=_p._BF16)
    with _on(stream, y):
        out, = _outs(y, (out, "out", 2 * T * N, (T, N), torch.bfloat16, 2))
    _launch(_p._L.lpq_route_combine, "lpq_route_combine", y, stream, y.data_ptr(), R, N, rows.data_ptr(), T, k, _ptr(weights),
            _ptr(residual), out.data_ptr())
    return out


def lpq_route_combine_backward(dout, rows, src, weights=None, y=None, dy=None, dweights=None, want_dweights=True, stream=None):
    """Gradients of lpq_route_combine from dout [tokens,N] BF16: (dy [R,N] BF16, zeros in rows without a token;
    dweights like rows FP32, or None with ``want_dweights`` False, which needs no y)."""
    dout = _bf16_in(dout, "dout")
    T, N = dout.shape
    _, k = _tokens(rows, dout, T)
    R = _arg(src, "src", dout, dtypes=_I32).numel()
    if want_dweights:
        if y is None:
            raise ValueError("the gradient of the weights needs y")
        _arg(y, "y", dout, 2 * R * N, dtypes=_p._BF16)
    elif dweights is not None:
        raise ValueError("dweights was passed in, and want_dweights is False")
    if weights is not None:
        _arg(weights, "weights", dout, 4 * T * k, dtypes=(torch.float32,))
    specs = [(dy, "dy", 2 * R * N, (R, N), torch.bfloat16, 2)]
    if want_dweights:
        specs.append((dweights, "dweights", 4 * T * k, rows.shape, torch.float32, 4))
    with _on(stream, dout):
        dy, dweights = (_outs(dout, *specs) + [None])[:2]
    _launch(_p._L.lpq_route_combine_backward, "lpq_route_combine_backward", dout, stream, dout.data_ptr(),
            _ptr(y) if want_dweights else 0, R, N, rows.data_ptr(), src.data_ptr(), T, k, _ptr(weights), dy.data_ptr(),
            _ptr(dweights))
    return dy, dweights


# --------------------------------------------------------------------------- adapters

def _adapters(x, A, B, offsets, rows, src, scale):
    """(tokens, capacity, groups, rank, N, K), every input checked."""
    x = _bf16_in(x, "x")
    T, K = x.shape
    _arg(A, "A", x, dtypes=_p._BF16, dims=3)
    _arg(B, "B", x, dtypes=_p._BF16, dims=3)
    L, r, KA = A.shape
    if KA != K or B.shape[0] != L or B.shape[2] != r:
        raise ValueError(f"A must be [groups, rank, {K}] and B [groups, N, rank], got {tuple(A.shape)} and {tuple(B.shape)}")
    if _offsets(offsets, x) != L:
        raise ValueError(f"offsets is of {offsets.numel() - 1} groups, the adapters are {L}")
    _, k = _tokens(rows, x, T)
    if k != 1:
        raise ValueError(f"a token has one adapter, the plan {k} slots a token")
    R = _arg(src, "src", x, dtypes=_I32).numel()
    if scale is not None:
        _arg(scale, "scale", x, 4 * L, dtypes=(torch.float32,))
    return T, R, L, r, B.shape[1], K


def lpq_adapters(x, A, B, offsets, rows, src, scale=None, base=None, y=None, workspace=None, stream=None):
    """y [tokens,N] = BF16(base + scale[g] (x A[g]^T) B[g]^T), g each token's adapter in a plan of one slot a token:
    x [tokens,K], A [groups,rank,K], B [groups,N,rank] BF16 (K, N and rank multiples of 8, rank up to 128), scale
    [groups] FP32 (None: ones), base [tokens,N] BF16 (None: zeros; ``y`` may be it)."""
    T, R, L, r, N, K = dims = _adapters(x, A, B, offsets, rows, src, scale)
    if base is not None:
        _arg(base, "base", x, 2 * T * N, dtypes=_p._BF16)
    need = _p._L.lpq_adapters_workspace(*dims)
    if workspace is not None:
        _arg(workspace, "workspace", x, need)
    with _on(stream, x):
        y, = _outs(x, (y, "y", 2 * T * N, (T, N), torch.bfloat16, 2))
        if workspace is None:
            workspace = _empty((need,), torch.uint8, x)
    _launch(_p._L.lpq_adapters, "lpq_adapters", x, stream, x.data_ptr(), A.data_ptr(), B.data_ptr(), _ptr(scale),
            offsets.data_ptr(), rows.data_ptr(), src.data_ptr(), *dims, _ptr(base), y.data_ptr(), workspace.data_ptr(),
            workspace.nbytes)
    return y


def lpq_adapters_backward(dy, x, A, B, offsets, rows, src, scale=None, dres=None, dx=None, dA=None, dB=None, accumulate=False,
                          workspace=None, stream=None):
    """Gradients of lpq_adapters from dy [tokens,N] BF16: (dx [tokens,K] BF16 = dres + ..., dA and dB like A and B in
    FP32).  ``accumulate``: dA and dB, passed in, are added to."""
    T, R, L, r, N, K = dims = _adapters(x, A, B, offsets, rows, src, scale)
    _arg(dy, "dy", x, 2 * T * N, dtypes=_p._BF16)
    if dres is not None:
        _arg(dres, "dres", x, 2 * T * K, dtypes=_p._BF16)
    if accumulate and (dA is None or dB is None):
        raise ValueError("accumulate adds to the dA and dB that are passed in")
    need = _p._L.lpq_adapters_backward_workspace(*dims)
    if workspace is not None:
        _arg(workspace, "workspace", x, need)
    with _on(stream, x):
        dx, dA, dB = _outs(x, (dx, "dx", 2 * T * K, (T, K), torch.bfloat16, 2), (dA, "dA", 4 * L * r * K, (L, r, K), torch.float32, 4),
                           (dB, "dB", 4 * L * N * r, (L, N, r), torch.float32, 4))
        if workspace is None:
            workspace = _empty((need,), torch.uint8, x)
    _launch(_p._L.lpq_adapters_backward, "lpq_adapters_backward", x, stream, dy.data_ptr(), x.data_ptr(), A.data_ptr(), B.data_ptr(),
            _ptr(scale), offsets.data_ptr(), rows.data_ptr(), src.data_ptr(), *dims, _ptr(dres), dx.data_ptr(), dA.data_ptr(),
            dB.data_ptr(), int(bool(accumulate)), workspace.data_ptr(), workspace.nbytes)
    return dx, dA, dB

"""The two ends of a block: the residual's addition with the norm in front of a projection, and projections in 8 bits.

8-bit tensors are ``torch.float8_e4m3fn`` with an fp32 scale for each block of 128 consecutive values of a row, or of 128
rows and columns (weights); a value stands for code times scale.  scale = max(largest magnitude of the block, 2^-100) / 448
and value / scale are fp32, and the code is the nearest to that quotient, halves to the even one: ``(x / scale).to(
torch.float8_e4m3fn)`` of finite fp32 tensors, bit for bit.  Rows of 8-bit tensors that are made here have their length rounded
up to a multiple of 16, with zeros behind the end, so that any of them can go into a product, and begin at a multiple of 128
bytes where they are long.  A block that holds a NaN or an infinity makes every result of its row (its rows and columns) that
it meets NaN.

A projection y = x W^T and its gradients are

    xq = quantize_fp8(x);  wq = quantize_fp8_blocks(W, columns=True)
    y  = matmul_fp8(xq["q"], xq["scale"], wq["q"], wq["scale"])
    gq = quantize_fp8(dy, columns=True);  xt = quantize_fp8(x, rows=False, columns=True)
    dx = matmul_fp8(gq["q"], gq["scale"], wq["qt"], wq["scale_t"])
    dW = matmul_fp8(gq["qt"], gq["scale_t"], xt["qt"], xt["scale_t"], out_dtype=torch.float32)

``add_norm_fwd`` with an 8-bit output takes the place of a norm and the quantisation behind it.

Rows may lie further apart than they are long; the other axes are dense.  Work runs on the current stream of the tensors'
device, or on ``stream``; what a call allocates belongs to that stream.  Nothing is read on the host, so a call can be
captured into a graph.  A given workspace serves one call at a time.
"""
from __future__ import annotations

import ctypes

from . import _abi
from .packed import _apart, _dtype_code, _launch, _on_gpu, _ptr, _rows, _space, _whole

BLOCK = 128


def _up16(n):
    return (n + 15) // 16 * 16


def _codes(rows, cols, device):
    """Memory for codes (rows, cols rounded up to 16).  Rows of several cache lines begin with one: the product of rows that
    do not reads every line twice (8191 x 2560 x 10576: 320 and 287 us)."""
    import torch
    n = (cols + 15) // 16 * 16
    if n % 128 == 0 or n < 512:
        return torch.empty(rows, n, dtype=torch.float8_e4m3fn, device=device)
    return torch.empty(rows, (n + 127) // 128 * 128, dtype=torch.float8_e4m3fn, device=device)[:, :n]


def _blocks(n):
    return (n + BLOCK - 1) // BLOCK


def _alias(out, *ins):
    """The names of the tensors that ``out`` may be itself: those of its type."""
    return tuple(name for name, t in ins if t is not None and out is not None and t.dtype == out.dtype)


# ---------------------------------------------------------------------------------------------------------------
# norm

def add_norm_fwd(x, weight, residual=None, *, eps=1e-5, y_dtype=None, residual_dtype=None, y=None, y_scale=None,
                 residual_out=None, stream=None):
    """Residual addition and root mean square norm of each row: h = x + residual, y = h weight / sqrt(mean(h^2) + eps).

    x (T, D) float32 or bfloat16, D <= 16384; weight (D,) float32; residual (T, D) float32 or bfloat16.  Returns
    (y, residual_out, y_scale).  y has x's type, or with ``y_dtype`` (or a given y of) float8_e4m3fn it holds codes
    (T, D rounded up to 16) and y_scale (T, ceil(D / 128)) their scales; without, y_scale is None.  residual_out is h in the
    residual's type; without a residual it is kept (h = x) when ``residual_dtype`` or ``residual_out`` is given, else None.
    The norm is that of the fp32 sum, of rows of any finite size.  residual_out may be the residual or x, y may be x (of one
    type with it)."""
    import torch
    T, D = x.shape
    dev = _on_gpu(x, "x")
    io = _dtype_code(x, "x")
    f8 = torch.float8_e4m3fn
    if y is not None:
        if y_dtype is not None and y_dtype != y.dtype:
            raise TypeError("y_dtype %s does not match the given y (%s)" % (y_dtype, y.dtype))
        y_dtype = y.dtype
    elif y_dtype is None:
        y_dtype = x.dtype
    if y_dtype != x.dtype and y_dtype != f8:
        raise TypeError("y: unsupported dtype %s (x's, or float8_e4m3fn)" % y_dtype)
    eight = y_dtype == f8
    for t in (residual, residual_out):
        if t is not None:
            if residual_dtype is not None and residual_dtype != t.dtype:
                raise TypeError("residual and residual_out: expected one dtype, got %s and %s" % (residual_dtype, t.dtype))
            residual_dtype = t.dtype
    if residual_dtype is None or residual_dtype == x.dtype:
        rio = io
    elif residual_dtype == torch.float32:
        rio = _abi.SSM_F32
    elif residual_dtype == torch.bfloat16:
        rio = _abi.SSM_BF16
    else:
        raise TypeError("residual: unsupported dtype %s (float32 or bfloat16)" % residual_dtype)
    keep = residual_dtype is not None
    _whole("weight", weight, (D,), torch.float32, dev, optional=False)
    xs = _rows("x", x, (T, D), x.dtype, dev)
    rs = hs = ys = ss = 0
    if residual is not None:
        rs = _rows("residual", residual, (T, D), residual_dtype, dev)
    if y_scale is not None:
        if not eight:
            raise ValueError("y_scale without an 8-bit y")
        ss = _rows("y_scale", y_scale, (T, _blocks(D)), torch.float32, dev)
    if y is not None:
        ys = _rows("y", y, (T, _up16(D) if eight else D), y_dtype, dev)
    if residual_out is not None:
        hs = _rows("residual_out", residual_out, (T, D), residual_dtype, dev)
        ins = (("x", x), ("residual", residual))
        _apart(residual_out, "residual_out", ("weight", weight), *ins, may_be=_alias(residual_out, *ins))
    if y is not None:
        _apart(y, "y", ("x", x), ("weight", weight), ("residual", residual), ("residual_out", residual_out),
               may_be=_alias(y, ("x", x)))
    if y_scale is not None:
        _apart(y_scale, "y_scale", ("x", x), ("weight", weight), ("residual", residual), ("residual_out", residual_out), ("y", y))
    with _launch(dev, stream, x, weight, residual, y, y_scale, residual_out) as st:
        if y is None:
            y = _codes(T, D, dev) if eight else torch.empty(T, D, dtype=y_dtype, device=dev)
            ys = y.stride(0)
        if eight and y_scale is None:
            y_scale = torch.empty(T, _blocks(D), dtype=torch.float32, device=dev)
        if keep and residual_out is None:
            residual_out = torch.empty(T, D, dtype=residual_dtype, device=dev)
        p = _abi.AddNormParams(T, D, xs, rs, hs, ys, ss, 0, 0, 0, 0, float(eps), io, rio, _abi.SSM_E4M3 if eight else io, 0)
        _abi.check(_abi.lib().ssm_add_norm_fwd(ctypes.byref(p), _ptr(x), _ptr(residual), _ptr(weight), _ptr(residual_out),
                                               _ptr(y), _ptr(y_scale), st))
    return y, residual_out, y_scale


def add_norm_bwd(h, weight, dy, dh=None, *, eps=1e-5, dx=None, dresidual=None, workspace=None, stream=None):
    """Backward of add_norm_fwd for dy = dL/dy (T, D) and optionally dh = dL/d(residual_out): h (T, D) is the sum that the
    forward kept (x itself where there was no residual).  Returns dict dx (T, D) of dy's type and dresidual (T, D) of h's,
    both the gradient of the sum (one tensor where the types are the same), and dweight (D,) float32.  The rounding of an
    8-bit y counts as the identity.  ``dx`` and ``dresidual`` may be given; dx may be dy, dresidual may be h or dh."""
    import torch
    T, D = h.shape
    dev = _on_gpu(h, "h")
    rio = _dtype_code(h, "h")
    if dy is None:
        raise ValueError("dy is required")
    io = _dtype_code(dy, "dy")
    _whole("weight", weight, (D,), torch.float32, dev, optional=False)
    hs = _rows("h", h, (T, D), h.dtype, dev)
    dys = _rows("dy", dy, (T, D), dy.dtype, dev)
    dhs = _rows("dh", dh, (T, D), h.dtype, dev, optional=True)
    dxs = drs = 0
    ins = (("h", h), ("dy", dy), ("dh", dh))
    if dx is not None:
        dxs = _rows("dx", dx, (T, D), dy.dtype, dev)
        _apart(dx, "dx", *ins, ("weight", weight), ("dresidual", dresidual), may_be=_alias(dx, *ins))
    if dresidual is not None:
        drs = _rows("dresidual", dresidual, (T, D), h.dtype, dev)
        _apart(dresidual, "dresidual", *ins, ("weight", weight), may_be=_alias(dresidual, *ins))
    if workspace is not None:
        _apart(workspace, "workspace", *ins, ("weight", weight), ("dx", dx), ("dresidual", dresidual))
    with _launch(dev, stream, h, weight, dy, dh, dx, dresidual, workspace) as st:
        one = io == rio and (dx is None or dresidual is None)
        if one:
            dx = dresidual = dx if dx is not None else dresidual if dresidual is not None else torch.empty(
                T, D, dtype=h.dtype, device=dev)
            dxs = drs = dxs or drs
        else:
            dx = torch.empty(T, D, dtype=dy.dtype, device=dev) if dx is None else dx
            dresidual = torch.empty(T, D, dtype=h.dtype, device=dev) if dresidual is None else dresidual
        dweight = torch.empty(D, dtype=torch.float32, device=dev)
        p = _abi.AddNormParams(T, D, 0, 0, hs, 0, 0, dys, dhs, dxs, drs, float(eps), io, rio, io, 0)
        if workspace is None:
            need = int(_abi.lib().ssm_add_norm_bwd_workspace_bytes(ctypes.byref(p)))
            workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=dev)
        _abi.check(_abi.lib().ssm_add_norm_bwd(ctypes.byref(p), _ptr(h), _ptr(weight), _ptr(dy), _ptr(dh),
                                               0 if one else _ptr(dx), _ptr(dresidual), _ptr(dweight), _ptr(workspace),
                                               _space(workspace, dev), st))
    return {"dx": dx, "dresidual": dresidual, "dweight": dweight}


# ---------------------------------------------------------------------------------------------------------------
# quantisation

def _output(name, t, shape, dtype, dev, *ins):
    """Checks an output, which may not overlap ``ins``, and returns the stride between its rows."""
    stride = _rows(name, t, shape, dtype, dev)
    _apart(t, name, *ins)
    return stride


def _quantize(x, square, rows, columns, q, scale, qt, scale_t, stream):
    import torch
    T, D = x.shape
    dev = _on_gpu(x, "x")
    io = _dtype_code(x, "x")
    f8, f32 = torch.float8_e4m3fn, torch.float32
    if not rows and not columns:
        raise ValueError("rows or columns: at least one is required")
    if not rows and (q is not None or scale is not None):
        raise ValueError("q and scale: no output of this call without rows")
    if not columns and (qt is not None or scale_t is not None):
        raise ValueError("qt and scale_t: no output of this call without columns")
    tb, db = (T + 127) // 128, (D + 127) // 128
    of_rows, of_columns = ((tb, db), (db, tb)) if square else ((T, db), (D, tb))
    xs = _rows("x", x, (T, D), x.dtype, dev)
    qs = ss = qts = sts = 0
    if q is not None:
        qs = _output("q", q, (T, _up16(D)), f8, dev, ("x", x))
    if scale is not None:
        ss = _output("scale", scale, of_rows, f32, dev, ("x", x), ("q", q))
    if qt is not None:
        qts = _output("qt", qt, (D, _up16(T)), f8, dev, ("x", x), ("q", q), ("scale", scale))
    if scale_t is not None:
        sts = _output("scale_t", scale_t, of_columns, f32, dev, ("x", x), ("q", q), ("scale", scale), ("qt", qt))
    with _launch(dev, stream, x, q, scale, qt, scale_t) as st:
        if rows:
            if q is None:
                q = _codes(T, D, dev)
                qs = q.stride(0)
            if scale is None:
                scale = torch.empty(*of_rows, dtype=f32, device=dev)
        if columns:
            if qt is None:
                qt = _codes(D, T, dev)
                qts = qt.stride(0)
            if scale_t is None:
                scale_t = torch.empty(*of_columns, dtype=f32, device=dev)
        p = _abi.QuantizeFp8Params(T, D, xs, qs, ss, qts, sts, io, square)
        _abi.check(_abi.lib().ssm_quantize_fp8(ctypes.byref(p), _ptr(x), _ptr(q), _ptr(scale), _ptr(qt), _ptr(scale_t), st))
    return {"q": q, "scale": scale, "qt": qt, "scale_t": scale_t}


def quantize_fp8(x, *, rows=True, columns=False, q=None, scale=None, qt=None, scale_t=None, stream=None):
    """x (T, D) float32 or bfloat16 to 8 bits with a scale for each block of 128 along the rows, the columns or both.
    Returns dict q (T, D rounded up to 16) and scale (T, ceil(D / 128)) with ``rows``, qt (D, T rounded up to 16), the codes
    of the transposed matrix, and scale_t (D, ceil(T / 128)) with ``columns``; the others are None.  Outputs may be given."""
    return _quantize(x, 0, rows, columns, q, scale, qt, scale_t, stream)


def quantize_fp8_blocks(w, *, rows=True, columns=False, q=None, scale=None, qt=None, scale_t=None, stream=None):
    """w (N, K) float32 or bfloat16 to 8 bits with a scale for each block of 128 rows and 128 columns: the form of a
    weight.  Returns dict as quantize_fp8, with scale (ceil(N / 128), ceil(K / 128)) and scale_t its transposed."""
    return _quantize(w, 1, rows, columns, q, scale, qt, scale_t, stream)


# ---------------------------------------------------------------------------------------------------------------
# product

def matmul_fp8(a, a_scale, b, b_scale, *, out_dtype=None, out=None, stream=None):
    """Matrix product of 8-bit operands: out (M, N) = a b^T for a (M, K), b (N, K) float8_e4m3fn, K a multiple of 16, with
    a_scale (M, ceil(K / 128)) and b_scale (ceil(N / 128), ceil(K / 128)), or (N, ceil(K / 128)) with a scale for each row,
    float32.  out is bfloat16 (default) or float32, rounded once.  Two scales are multiplied in fp32: their product has to be
    finite, and below 2^-126 it is rounded to a multiple of 2^-149.
    float32 results are sums in fp32.  For bfloat16 ones the matrix cores drop what lies below about 2^-12 of the largest
    product of a block (1e-5 to 5e-5 of the results' 2-norm, whose rounding is 1.7e-3); where large products of a block cancel,
    float32 results keep what is left below that."""
    import torch
    M, K = a.shape
    dev = _on_gpu(a, "a")
    f8, f32 = torch.float8_e4m3fn, torch.float32
    if b is None or b.dim() != 2:
        raise ValueError("b: expected shape (N, %d)" % K)
    N = b.shape[0]
    sa = _rows("a", a, (M, K), f8, dev)
    sb = _rows("b", b, (N, K), f8, dev)
    kb = (K + 127) // 128
    sas = _rows("a_scale", a_scale, (M, kb), f32, dev)
    if b_scale is None or b_scale.dim() != 2:
        raise ValueError("b_scale: expected shape (%d, %d) or (%d, %d)" % (_blocks(N), kb, N, kb))
    b_rows = 1 if b_scale.shape[0] == N and N > 1 else BLOCK
    sbs = _rows("b_scale", b_scale, (N if b_rows == 1 else (N + 127) // 128, kb), f32, dev)
    if out is not None:
        if out_dtype is not None and out_dtype != out.dtype:
            raise TypeError("out_dtype %s does not match the given out (%s)" % (out_dtype, out.dtype))
        out_dtype = out.dtype
    elif out_dtype is None:
        out_dtype = torch.bfloat16
    if out_dtype != torch.bfloat16 and out_dtype != f32:
        raise TypeError("out: unsupported dtype %s (float32 or bfloat16)" % out_dtype)
    os_ = 0
    if out is not None:
        os_ = _rows("out", out, (M, N), out_dtype, dev)
        _apart(out, "out", ("a", a), ("a_scale", a_scale), ("b", b), ("b_scale", b_scale))
    with _launch(dev, stream, a, a_scale, b, b_scale, out) as st:
        if out is None:
            out = torch.empty(M, N, dtype=out_dtype, device=dev)
        p = _abi.MatmulFp8Params(M, N, K, sa, sb, os_, sas, sbs, b_rows, _abi.SSM_F32 if out_dtype == f32 else _abi.SSM_BF16)
        _abi.check(_abi.lib().ssm_matmul_fp8(ctypes.byref(p), _ptr(a), _ptr(a_scale), _ptr(b), _ptr(b_scale), _ptr(out), st))
    return out

"""The Mamba-2 block's operators over packed tokens: the causal convolution, the SSD layer and the gated group norm.

Rows are tokens; the sequences of a batch lie one behind the other, and ``cu_seqlens`` (S + 1,) int32, on the device,
holds where each begins and the last one ends.  Rows may lie further apart than they are long (slices of a wider
projection are taken as they are); the other axes are dense.  Rows outside every sequence are not used and not written.

Recurrent states live in a pool whose first axis is slots.  ``state_idx`` (S,) int32, on the device, names the slot of
each sequence or row (None: sequence s uses slot s); an index outside the pool means that it has none, so it starts
from zeros and its last state is not kept.  Each slot may be named once per call.  ``has_state`` (S,) bool, on the
device: which sequences start from their slot (None: all, when ``state`` is given).  ``state_out`` receives the last
states and may be ``state`` itself.  Nothing is read on the host, so a call can be captured into a graph.

Work runs on the current stream of the tensors' device, or on ``stream``; what a call allocates belongs to that stream.
A given workspace serves one call at a time: calls that overlap, and graphs replayed side by side, take one each.
Rows outside every sequence are left as they are in outputs too: unset where the call allocates the output.
"""
from __future__ import annotations

import ctypes

from . import _abi
from ._abi import EULER_B


def _ptr(t):
    return 0 if t is None else t.data_ptr()


def _dtype_code(t, name):
    import torch
    if t.dtype == torch.float32:
        return _abi.SSM_F32
    if t.dtype == torch.bfloat16:
        return _abi.SSM_BF16
    raise TypeError("%s: unsupported dtype %s (float32 or bfloat16)" % (name, t.dtype))


def _rows(name, t, shape, dtype, device, optional=False):
    """Checks a tensor of rows and returns the stride between them (0 for an absent tensor)."""
    if t is not None and t.shape == shape and t.dtype == dtype and t.device == device and t.is_contiguous():
        return shape[1] if len(shape) == 2 else t.numel() // max(shape[0], 1)
    if t is None:
        if not optional:
            raise ValueError("%s is required" % name)
        return 0
    if tuple(t.shape) != tuple(shape):
        raise ValueError("%s: expected shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))
    if t.dtype != dtype:
        raise TypeError("%s: expected dtype %s, got %s" % (name, dtype, t.dtype))
    if t.device != device:
        raise ValueError("%s: expected device %s, got %s" % (name, device, t.device))
    dense = 1
    for d in range(t.dim() - 1, 0, -1):
        if t.shape[d] != 1 and t.stride(d) != dense:
            raise ValueError("%s: only the rows may lie apart (strides %s)" % (name, tuple(t.stride())))
        dense *= t.shape[d]
    if t.shape[0] == 1:
        return dense
    if t.stride(0) < dense:
        raise ValueError("%s: rows overlap (strides %s)" % (name, tuple(t.stride())))
    return t.stride(0)


def _whole(name, t, shape, dtype, device, optional=True):
    """Checks a contiguous tensor."""
    if t is not None and t.shape == shape and t.dtype == dtype and t.device == device and t.is_contiguous():
        return
    if t is None:
        if not optional:
            raise ValueError("%s is required" % name)
        return
    if tuple(t.shape) != tuple(shape):
        raise ValueError("%s: expected shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))
    if t.dtype != dtype:
        raise TypeError("%s: expected dtype %s, got %s" % (name, dtype, t.dtype))
    if t.device != device:
        raise ValueError("%s: expected device %s, got %s" % (name, device, t.device))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)


def _space(t, device):
    """Checks a given workspace and returns its bytes."""
    if t is None:
        return 0
    if t.device != device or not t.is_contiguous():
        raise ValueError("workspace: expected a contiguous tensor on %s" % device)
    return t.numel() * t.element_size()


def _on_gpu(t, name):
    if not t.is_cuda:
        raise ValueError("%s: expected a tensor on the GPU, got %s" % (name, t.device))
    return t.device


class _launch:
    """The device made current and the stream's handle; tensors made inside belong to that stream, and the memory of
    ``tensors`` is not given away before a given stream has used it."""
    __slots__ = ("device", "stream", "tensors", "inside")

    def __init__(self, device, stream, *tensors):
        self.device, self.stream, self.tensors, self.inside = device, stream, tensors, ()

    def __enter__(self):
        import torch
        if self.stream is None:
            if self.device.index != torch._C._cuda_getDevice():
                self._enter(torch.cuda.device(self.device))
            # (the handle alone: torch.cuda.current_stream makes an object around it, 1.9 of a call's 10 us)
            return torch._C._cuda_getCurrentRawStream(self.device.index)
        if self.stream.device != self.device:
            raise ValueError("stream: expected one of %s, got %s" % (self.device, self.stream.device))
        self._enter(torch.cuda.device(self.device))
        self._enter(torch.cuda.stream(self.stream))
        return self.stream.cuda_stream

    def _enter(self, context):
        context.__enter__()
        self.inside = (context,) + self.inside

    def __exit__(self, *error):
        for context in self.inside:
            context.__exit__(*error)
        if self.stream is not None and error[0] is None:
            for t in self.tensors:
                if t is not None:
                    t.record_stream(self.stream)


def _apart(out, name, *ins, may_be=()):
    """Refuses an output that shares memory with another tensor of the call, unless it is one of ``may_be`` itself."""
    def span(t):
        return t.data_ptr(), t.data_ptr() + (sum((n - 1) * s for n, s in zip(t.shape, t.stride())) + 1) * t.element_size()

    def row(t):
        return (sum((n - 1) * s for n, s in zip(t.shape[1:], t.stride()[1:])) + 1) * t.element_size()

    if out is None:
        return
    for other, t in ins:
        if t is None or out.untyped_storage().data_ptr() != t.untyped_storage().data_ptr():
            continue
        if other in may_be and t.data_ptr() == out.data_ptr() and t.stride() == out.stride():
            continue
        (a0, a1), (b0, b1) = span(out), span(t)
        if a1 <= b0 or b1 <= a0:
            continue
        # slices of one wider row lie side by side
        width = out.stride(0) * out.element_size()
        if out.shape[0] > 1 and t.shape[0] > 1 and t.stride(0) * t.element_size() == width:
            gap = (b0 - a0) % width
            if gap >= row(out) and gap + row(t) <= width:
                continue
        raise ValueError("%s must not overlap %s" % (name, other))


def _sequences(cu_seqlens, device):
    import torch
    if cu_seqlens is None or cu_seqlens.dim() != 1 or cu_seqlens.shape[0] < 2:
        raise ValueError("cu_seqlens: expected shape (sequences + 1,)")
    _whole("cu_seqlens", cu_seqlens, tuple(cu_seqlens.shape), torch.int32, device, optional=False)
    return cu_seqlens.shape[0] - 1


def _pool(state, state_out, state_idx, has_state, tail, S, device):
    """Checks the pools and their indices and returns the number of slots."""
    import torch
    slots = None
    for name, t in (("state", state), ("state_out", state_out)):
        if t is None:
            continue
        if t.dim() != 1 + len(tail):
            raise ValueError("%s: expected shape (slots,) + %s" % (name, tuple(tail)))
        if slots is not None and t.shape[0] != slots:
            raise ValueError("state and state_out must have the same number of slots")
        slots = t.shape[0]
        _whole(name, t, (slots,) + tuple(tail), torch.float32, device)
    _whole("state_idx", state_idx, (S,), torch.int32, device)
    _whole("has_state", has_state, (S,), torch.bool, device)
    if slots is not None and state_idx is None and slots < S:
        raise ValueError("%d slots for %d sequences: state_idx is required" % (slots, S))
    if state is not None and state_out is not None and state.data_ptr() != state_out.data_ptr():
        _apart(state_out, "state_out", ("state", state))
    return slots or 0


# ---------------------------------------------------------------------------------------------------------------
# convolution

def _conv_weights(conv_w, conv_bias, D, device):
    import torch
    if conv_w is None or conv_w.dim() != 2 or conv_w.shape[0] != D:
        raise ValueError("conv_w: expected shape (%d, width)" % D)
    _whole("conv_w", conv_w, (D, conv_w.shape[1]), torch.float32, device, optional=False)
    _whole("conv_bias", conv_bias, (D,), torch.float32, device)
    return conv_w.shape[1]


def conv1d_packed_fwd(x, conv_w, cu_seqlens, conv_bias=None, *, state=None, state_out=None, state_idx=None,
                      has_state=None, activation=True, u=None, stream=None):
    """Causal depthwise convolution (+ SiLU) over packed tokens: x (T, D) float32 or bfloat16 -> u (T, D).

    conv_w (D, width <= 4), conv_bias (D,) float32.  state / state_out (slots, D, width - 1) float32: the width - 1
    inputs before a sequence, oldest first, and its last ones.  Rows of u outside every sequence are left as they are.
    """
    import torch
    T, D = x.shape
    dev = _on_gpu(x, "x")
    io = _dtype_code(x, "x")
    K = _conv_weights(conv_w, conv_bias, D, dev)
    S = _sequences(cu_seqlens, dev)
    slots = _pool(state, state_out, state_idx, has_state, (D, K - 1), S, dev)
    xs = _rows("x", x, (T, D), x.dtype, dev)
    us = _rows("u", u, (T, D), x.dtype, dev, optional=True)
    _apart(u, "u", ("x", x))
    with _launch(dev, stream, x, conv_w, cu_seqlens, conv_bias, state, state_out, state_idx, has_state, u) as st:
        if u is None:
            u = torch.empty((T, D), dtype=x.dtype, device=dev)
            us = D
        p = _abi.ConvPackedParams(T, S, D, slots, xs, us, 0, 0, K, int(bool(activation)), io, 0)
        _abi.check(_abi.lib().ssm_conv1d_packed_fwd(ctypes.byref(p), _ptr(x), _ptr(conv_w), _ptr(conv_bias),
                                                    _ptr(cu_seqlens), _ptr(state), _ptr(state_idx), _ptr(has_state),
                                                    _ptr(state_out), _ptr(u), st))
    return u


def conv1d_slot_update(state, x, conv_w, conv_bias=None, *, state_idx=None, activation=True, u=None, stream=None):
    """One token per row through the convolution: x (b, D); the window of row r in state (slots, D, width - 1), slot
    state_idx[r], is shifted in place.  Returns u (b, D)."""
    import torch
    b, D = x.shape
    dev = _on_gpu(x, "x")
    io = _dtype_code(x, "x")
    K = _conv_weights(conv_w, conv_bias, D, dev)
    if state is None:
        raise ValueError("state is required")
    slots = _pool(state, None, state_idx, None, (D, K - 1), b, dev)
    xs = _rows("x", x, (b, D), x.dtype, dev)
    us = _rows("u", u, (b, D), x.dtype, dev, optional=True)
    _apart(u, "u", ("x", x))
    with _launch(dev, stream, state, x, conv_w, conv_bias, state_idx, u) as st:
        if u is None:
            u = torch.empty((b, D), dtype=x.dtype, device=dev)
            us = D
        p = _abi.ConvPackedParams(b, b, D, slots, xs, us, 0, 0, K, int(bool(activation)), io, 0)
        _abi.check(_abi.lib().ssm_conv1d_slot_update(ctypes.byref(p), _ptr(x), _ptr(conv_w), _ptr(conv_bias),
                                                     _ptr(state), _ptr(state_idx), _ptr(u), st))
    return u


def conv1d_packed_bwd(x, conv_w, du, cu_seqlens, conv_bias=None, *, state=None, state_idx=None, has_state=None,
                      dstate_out=None, activation=True, want_dstate=False, dx=None, workspace=None, stream=None):
    """Backward of conv1d_packed_fwd for du = dL/du (T, D) and optionally dstate_out = dL/d(last window)
    (S, D, width - 1) float32, by sequence.  ``state`` is the pool as it was before the forward.  Returns dict dx (T, D),
    dweight (D, width), dbias (D,) and, with ``want_dstate``, dstate (S, D, width - 1); ``dx`` may be given.  Rows of dx
    outside every sequence are left as they are."""
    import torch
    T, D = x.shape
    dev = _on_gpu(x, "x")
    io = _dtype_code(x, "x")
    f32 = torch.float32
    K = _conv_weights(conv_w, conv_bias, D, dev)
    S = _sequences(cu_seqlens, dev)
    slots = _pool(state, None, state_idx, has_state, (D, K - 1), S, dev)
    _whole("dstate_out", dstate_out, (S, D, K - 1), f32, dev)
    xs = _rows("x", x, (T, D), x.dtype, dev)
    dus = _rows("du", du, (T, D), x.dtype, dev)
    dxs = _rows("dx", dx, (T, D), x.dtype, dev, optional=True)
    _apart(dx, "dx", ("x", x), ("du", du))
    with _launch(dev, stream, x, conv_w, du, cu_seqlens, conv_bias, state, state_idx, has_state, dstate_out, dx,
                 workspace) as st:
        if dx is None:
            dx = torch.empty((T, D), dtype=x.dtype, device=dev)
            dxs = D
        out = {"dx": dx, "dweight": torch.empty((D, K), dtype=f32, device=dev),
               "dbias": torch.empty((D,), dtype=f32, device=dev),
               "dstate": torch.empty((S, D, K - 1), dtype=f32, device=dev) if want_dstate else None}
        p = _abi.ConvPackedParams(T, S, D, slots, xs, 0, dus, dxs, K, int(bool(activation)), io, 0)
        need = int(_abi.lib().ssm_conv1d_packed_bwd_workspace_bytes(ctypes.byref(p)))
        if workspace is None:
            workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=dev)
        _abi.check(_abi.lib().ssm_conv1d_packed_bwd(
            ctypes.byref(p), _ptr(x), _ptr(conv_w), _ptr(conv_bias), _ptr(cu_seqlens), _ptr(state), _ptr(state_idx),
            _ptr(has_state), _ptr(du), _ptr(dstate_out), _ptr(dx), _ptr(out["dweight"]), _ptr(out["dbias"]),
            _ptr(out["dstate"]) if K > 1 else 0, _ptr(workspace), _space(workspace, dev), st))
    return out


# ---------------------------------------------------------------------------------------------------------------
# scan

def _ssd_inputs(x, dt, A, B, C, dt_bias, Dskip, lead, dev):
    """Checks the inputs both forms share; returns sizes and row strides."""
    import torch
    f32 = torch.float32
    _, H, P = x.shape
    if B is None or B.dim() != 3:
        raise ValueError("B: expected shape (%d, groups, dstate)" % lead)
    G, N = B.shape[1], B.shape[2]
    xs = _rows("x", x, (lead, H, P), x.dtype, dev)
    ds = _rows("dt", dt, (lead, H), x.dtype, dev)
    bs = _rows("B", B, (lead, G, N), x.dtype, dev)
    cs = _rows("C", C, (lead, G, N), x.dtype, dev)
    _whole("A", A, (H,), f32, dev, optional=False)
    _whole("dt_bias", dt_bias, (H,), f32, dev)
    _whole("Dskip", Dskip, (H,), f32, dev)
    return H, P, G, N, xs, ds, bs, cs


def ssd_packed_fwd(x, dt, A, B, C, cu_seqlens, dt_bias=None, Dskip=None, *, state=None, state_out=None, state_idx=None,
                   has_state=None, y=None, disc=EULER_B, softplus=True, segment_chunks=0, workspace=None, stream=None):
    """The Mamba-2 SSD layer over packed tokens, without the gate: x (T, H, 64), dt (T, H), B, C (T, G, N) bfloat16 (rows
    of x, B and C 16-byte aligned); A, dt_bias, Dskip (H,) float32; state / state_out (slots, H, 64, N) float32.  N is 64,
    128 or 256.  segment_chunks: 0 = the library's choice of the 64-step chunks of a sequence that run one after the
    other.  Returns y (T, H, 64); its rows outside every sequence are left as they are.  What is not finite reaches no earlier
    step and no other sequence: an entry of x makes its own column of y and of the state NaN from its step on."""
    import torch
    T = x.shape[0]
    dev = _on_gpu(x, "x")
    io = _dtype_code(x, "x")
    H, P, G, N, xs, ds, bs, cs = _ssd_inputs(x, dt, A, B, C, dt_bias, Dskip, T, dev)
    S = _sequences(cu_seqlens, dev)
    slots = _pool(state, state_out, state_idx, has_state, (H, P, N), S, dev)
    ys = _rows("y", y, (T, H, P), x.dtype, dev, optional=True)
    _apart(y, "y", ("x", x), ("dt", dt), ("B", B), ("C", C))
    with _launch(dev, stream, x, dt, A, B, C, cu_seqlens, dt_bias, Dskip, state, state_out, state_idx, has_state, y,
                 workspace) as st:
        if y is None:
            y = torch.empty((T, H, P), dtype=x.dtype, device=dev)
            ys = H * P
        p = _abi.SsdPackedParams(T, S, H, P, G, N, slots, xs, ds, bs, cs, ys, 0, 0, 0, 0, 0, io, int(disc),
                                 int(bool(softplus)), int(segment_chunks), 0)
        need = int(_abi.lib().ssm_ssd_packed_fwd_workspace_bytes(ctypes.byref(p)))
        if need and workspace is None:
            workspace = torch.empty(need, dtype=torch.uint8, device=dev)
        _abi.check(_abi.lib().ssm_ssd_packed_fwd(
            ctypes.byref(p), _ptr(x), _ptr(dt), _ptr(dt_bias), _ptr(A), _ptr(B), _ptr(C), _ptr(Dskip), _ptr(cu_seqlens),
            _ptr(state), _ptr(state_idx), _ptr(has_state), _ptr(state_out), _ptr(y), _ptr(workspace),
            _space(workspace, dev), st))
    return y


def ssd_slot_update(state, x, dt, A, B, C, dt_bias=None, Dskip=None, *, state_idx=None, y=None, disc=EULER_B,
                    softplus=True, stream=None):
    """One SSD step per row: x (b, H, 64), dt (b, H), B, C (b, G, N) bfloat16; the state of row r in state (slots, H, 64,
    N) float32, slot state_idx[r], is updated in place.  Returns y (b, H, 64)."""
    import torch
    b = x.shape[0]
    dev = _on_gpu(x, "x")
    io = _dtype_code(x, "x")
    H, P, G, N, xs, ds, bs, cs = _ssd_inputs(x, dt, A, B, C, dt_bias, Dskip, b, dev)
    if state is None:
        raise ValueError("state is required")
    slots = _pool(state, None, state_idx, None, (H, P, N), b, dev)
    ys = _rows("y", y, (b, H, P), x.dtype, dev, optional=True)
    _apart(y, "y", ("x", x), ("dt", dt), ("B", B), ("C", C))
    with _launch(dev, stream, state, x, dt, A, B, C, dt_bias, Dskip, state_idx, y) as st:
        if y is None:
            y = torch.empty((b, H, P), dtype=x.dtype, device=dev)
            ys = H * P
        p = _abi.SsdPackedParams(b, b, H, P, G, N, slots, xs, ds, bs, cs, ys, 0, 0, 0, 0, 0, io, int(disc),
                                 int(bool(softplus)), 0, 0)
        _abi.check(_abi.lib().ssm_ssd_slot_update(ctypes.byref(p), _ptr(state), _ptr(x), _ptr(dt), _ptr(dt_bias), _ptr(A),
                                                  _ptr(B), _ptr(C), _ptr(Dskip), _ptr(state_idx), _ptr(y), st))
    return y


def ssd_packed_bwd(x, dt, A, B, C, dy, cu_seqlens, dt_bias=None, Dskip=None, *, state=None, state_idx=None,
                   has_state=None, dstate_out=None, disc=EULER_B, softplus=True, segment_chunks=0, want_dstate=None,
                   out=None, workspace=None, stream=None):
    """Backward of ssd_packed_fwd for dy = dL/dy (T, H, 64) and optionally dstate_out = dL/d(last state) (S, H, 64, N)
    float32, by sequence; the states are recomputed from ``state``, the pool as it was before the forward.  Returns dict
    dx (T, H, 64), ddt (T, H), dB, dC (T, G, N) bfloat16, dA, dDskip, ddt_bias (H,) float32 and dstate (S, H, 64, N)
    float32, the gradient of the state each sequence starts from (want_dstate; by default when ``state`` or
    ``dstate_out`` is given).  ``out`` may hold dx, ddt, dB, dC to write into (rows of dx 16-byte, of dB and dC 8-byte
    aligned).  Rows outside every sequence are left as they are.  What is not finite in a sequence reaches the parameters'
    gradients and may reach any gradient of that sequence, but no other one's.  The workspace holds the states and adjoint
    states of every chunk of 64 steps: 512 H N bytes for each of about T / 64 + S chunks."""
    import torch
    T = x.shape[0]
    dev = _on_gpu(x, "x")
    io = _dtype_code(x, "x")
    f32 = torch.float32
    H, P, G, N, xs, ds, bs, cs = _ssd_inputs(x, dt, A, B, C, dt_bias, Dskip, T, dev)
    S = _sequences(cu_seqlens, dev)
    slots = _pool(state, None, state_idx, has_state, (H, P, N), S, dev)
    dys = _rows("dy", dy, (T, H, P), x.dtype, dev)
    _whole("dstate_out", dstate_out, (S, H, P, N), f32, dev)
    o = dict(out or {})
    shapes = {"dx": (T, H, P), "ddt": (T, H), "dB": (T, G, N), "dC": (T, G, N)}
    if set(o) - set(shapes):
        raise ValueError("out: dx, ddt, dB and dC may be given, got %s" % sorted(o))
    rows = {k: _rows(k, o.get(k), shp, x.dtype, dev, optional=True) for k, shp in shapes.items()}
    ins = [("x", x), ("dt", dt), ("B", B), ("C", C), ("dy", dy)]
    for k in shapes:
        _apart(o.get(k), k, *ins)
        ins.append((k, o.get(k)))
    if want_dstate is None:
        want_dstate = state is not None or dstate_out is not None
    with _launch(dev, stream, x, dt, A, B, C, dy, cu_seqlens, dt_bias, Dskip, state, state_idx, has_state, dstate_out,
                 workspace, *o.values()) as st:
        for k, shp in shapes.items():
            if o.get(k) is None:
                o[k] = torch.empty(shp, dtype=x.dtype, device=dev)
                rows[k] = 0
        for k in ("dA", "dDskip", "ddt_bias"):
            o[k] = torch.empty((H,), dtype=f32, device=dev)
        o["dstate"] = torch.empty((S, H, P, N), dtype=f32, device=dev) if want_dstate else None
        p = _abi.SsdPackedParams(T, S, H, P, G, N, slots, xs, ds, bs, cs, 0, dys, rows["dx"], rows["ddt"], rows["dB"],
                                 rows["dC"], io, int(disc), int(bool(softplus)), int(segment_chunks), 0)
        if workspace is None:
            need = int(_abi.lib().ssm_ssd_packed_bwd_workspace_bytes(ctypes.byref(p)))
            workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=dev)
        _abi.check(_abi.lib().ssm_ssd_packed_bwd(
            ctypes.byref(p), _ptr(x), _ptr(dt), _ptr(dt_bias), _ptr(A), _ptr(B), _ptr(C), _ptr(Dskip), _ptr(cu_seqlens),
            _ptr(state), _ptr(state_idx), _ptr(has_state), _ptr(dy), _ptr(dstate_out), _ptr(o["dx"]), _ptr(o["ddt"]),
            _ptr(o["dA"]), _ptr(o["dB"]), _ptr(o["dC"]), _ptr(o["dDskip"]), _ptr(o["ddt_bias"]), _ptr(o["dstate"]),
            _ptr(workspace), _space(workspace, dev), st))
    return o


# ---------------------------------------------------------------------------------------------------------------
# norm

def _norm_inputs(x, weight, bias, z, groups):
    import torch
    T, D = x.shape
    dev = _on_gpu(x, "x")
    io = _dtype_code(x, "x")
    if groups < 1 or D % groups:
        raise ValueError("groups: %d channels do not divide into %d groups" % (D, groups))
    _whole("weight", weight, (D,), torch.float32, dev, optional=False)
    _whole("bias", bias, (D,), torch.float32, dev)
    return T, D, dev, io, _rows("x", x, (T, D), x.dtype, dev), _rows("z", z, (T, D), x.dtype, dev, optional=True)


def gated_norm_fwd(x, weight, bias=None, z=None, *, groups=1, eps=1e-5, gate_first=True, center=False, y=None,
                   stream=None):
    """Group norm of each row of x (T, D) over ``groups`` groups of channels, with an optional SiLU gate z (T, D):
    norm(x silu(z)) weight + bias (gate_first), or (norm(x) weight + bias) silu(z).  ``center`` takes the mean off; without
    it the norm is the root mean square.  x, z float32 or bfloat16; weight, bias (D,) float32.  ``y`` may be x or z."""
    import torch
    T, D, dev, io, xs, zs = _norm_inputs(x, weight, bias, z, groups)
    ys = _rows("y", y, (T, D), x.dtype, dev, optional=True)
    _apart(y, "y", ("x", x), ("z", z), may_be=("x", "z"))
    with _launch(dev, stream, x, weight, bias, z, y) as st:
        if y is None:
            y = torch.empty((T, D), dtype=x.dtype, device=dev)
            ys = D
        p = _abi.GatedNormParams(T, D, groups, xs, zs, ys, 0, 0, 0, float(eps), io, int(bool(gate_first)),
                                 int(bool(center)), 0)
        _abi.check(_abi.lib().ssm_gated_norm_fwd(ctypes.byref(p), _ptr(x), _ptr(z), _ptr(weight), _ptr(bias), _ptr(y), st))
    return y


def gated_norm_bwd(x, weight, dy, bias=None, z=None, *, groups=1, eps=1e-5, gate_first=True, center=False, dx=None,
                   dz=None, workspace=None, stream=None):
    """Backward of gated_norm_fwd for dy = dL/dy (T, D); the statistics are recomputed.  Returns dict dx, dz (None without
    a gate) (T, D), dweight, dbias (D,) float32.  ``dx`` and ``dz`` may be given; dx may be x or dy, dz may be z."""
    import torch
    T, D, dev, io, xs, zs = _norm_inputs(x, weight, bias, z, groups)
    f32 = torch.float32
    if z is None and dz is not None:
        raise ValueError("dz without z")
    dys = _rows("dy", dy, (T, D), x.dtype, dev)
    dxs = _rows("dx", dx, (T, D), x.dtype, dev, optional=True)
    dzs = _rows("dz", dz, (T, D), x.dtype, dev, optional=True)
    _apart(dx, "dx", ("x", x), ("dy", dy), ("z", z), ("dz", dz), may_be=("x", "dy"))
    _apart(dz, "dz", ("z", z), ("x", x), ("dy", dy), may_be=("z",))
    with _launch(dev, stream, x, weight, dy, bias, z, dx, dz, workspace) as st:
        if dx is None:
            dx = torch.empty((T, D), dtype=x.dtype, device=dev)
            dxs = D
        if z is not None and dz is None:
            dz = torch.empty((T, D), dtype=x.dtype, device=dev)
            dzs = D
        out = {"dx": dx, "dz": dz, "dweight": torch.empty((D,), dtype=f32, device=dev),
               "dbias": torch.empty((D,), dtype=f32, device=dev)}
        p = _abi.GatedNormParams(T, D, groups, xs, zs, 0, dys, dxs, dzs, float(eps), io, int(bool(gate_first)),
                                 int(bool(center)), 0)
        need = int(_abi.lib().ssm_gated_norm_bwd_workspace_bytes(ctypes.byref(p)))
        if workspace is None:
            workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=dev)
        _abi.check(_abi.lib().ssm_gated_norm_bwd(
            ctypes.byref(p), _ptr(x), _ptr(z), _ptr(weight), _ptr(bias), _ptr(dy), _ptr(dx), _ptr(dz), _ptr(out["dweight"]),
            _ptr(out["dbias"]), _ptr(workspace), _space(workspace, dev), st))
    return out

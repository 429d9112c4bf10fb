"""ctypes binding of the block operators of libm3scan with the names of the C ABI (include/m3block.h):
gated scan, RMS norm with residual and 8-bit rows, gradient norm and clipping.

Like m3scan.py it only marshals: it checks placement, dtype, shape and strides, allocates outputs and
workspaces with torch when they are not passed, and turns a non-OK status into an M3Error.  There is
no fallback.  Calls run on the tensors' device, whichever is current, on its current stream or on
``stream``; what they allocate belongs to that stream.

Tensors of rows (gate, x, y, r, dy, ...) may be slices of wider ones: the last dimension has to be
dense, and the rows before it evenly spaced.
"""
from __future__ import annotations

import array
import contextlib
import ctypes

import torch

from . import m3scan
from .m3scan import M3_BF16, M3_F32, M3Error, STATUS_NAMES  # noqa: F401

EXPORTED = ["m3_gated_scan_chunks", "m3_gated_scan_workspace_bytes", "m3_gated_scan", "m3_gated_scan_step",
            "m3_gated_scan_backward_workspace_bytes", "m3_gated_scan_backward", "m3_rmsnorm",
            "m3_rmsnorm_backward_workspace_bytes", "m3_rmsnorm_backward", "m3_grad_workspace_bytes",
            "m3_grad_norm", "m3_grad_clip"]


class M3ScanDims(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int64), ("seqlen", ctypes.c_int64), ("width", ctypes.c_int64),
                ("gate_pitch", ctypes.c_int64), ("x_pitch", ctypes.c_int64), ("y_pitch", ctypes.c_int64),
                ("dgate_pitch", ctypes.c_int64), ("dx_pitch", ctypes.c_int64), ("io", ctypes.c_int32),
                ("flags", ctypes.c_uint32)]


class M3NormDims(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("width", ctypes.c_int64), ("x_pitch", ctypes.c_int64),
                ("res_pitch", ctypes.c_int64), ("r_pitch", ctypes.c_int64), ("y_pitch", ctypes.c_int64),
                ("dx_pitch", ctypes.c_int64), ("group", ctypes.c_int64), ("io", ctypes.c_int32),
                ("flags", ctypes.c_uint32), ("eps", ctypes.c_float)]


class M3GradTensor(ctypes.Structure):
    _fields_ = [("src", ctypes.c_void_p), ("dst", ctypes.c_void_p), ("numel", ctypes.c_int64),
                ("io", ctypes.c_int32), ("pad", ctypes.c_int32)]


_P = ctypes.c_void_p
_Z = ctypes.c_size_t
_lib = None


def load():
    """The library with the signatures of m3block.h declared (see m3scan.load)."""
    global _lib
    if _lib is None:
        lib = m3scan.load()
        scan, norm, grad = ctypes.POINTER(M3ScanDims), ctypes.POINTER(M3NormDims), ctypes.c_void_p
        f32, i64, st = ctypes.c_float, ctypes.c_int64, ctypes.c_int
        for name, res, args in [
                ("m3_gated_scan_chunks", i64, [scan, st]),
                ("m3_gated_scan_workspace_bytes", _Z, [scan, st]),
                ("m3_gated_scan", st, [scan] + [_P] * 9 + [_Z, _P]),
                ("m3_gated_scan_step", st, [scan] + [_P] * 7),
                ("m3_gated_scan_backward_workspace_bytes", _Z, [scan, st]),
                ("m3_gated_scan_backward", st, [scan] + [_P] * 13 + [_Z, _P]),
                ("m3_rmsnorm", st, [norm] + [_P] * 8),
                ("m3_rmsnorm_backward_workspace_bytes", _Z, [norm]),
                ("m3_rmsnorm_backward", st, [norm] + [_P] * 7 + [_Z, _P]),
                ("m3_grad_workspace_bytes", _Z, [grad, i64]),
                ("m3_grad_norm", st, [grad, i64, f32, _P, _P, _Z, _P]),
                ("m3_grad_clip", st, [grad, i64, f32, _P, _P, _Z, _P])]:
            fn = getattr(lib, name)
            fn.restype, fn.argtypes = res, args
        _lib = lib
    return _lib


def _check(status):
    if status:
        raise M3Error(status, m3scan.last_error())


def _io_code(t, name):
    if t.dtype == torch.bfloat16:
        return M3_BF16
    if t.dtype == torch.float32:
        return M3_F32
    raise ValueError("%s must be float32 or bfloat16, got %s" % (name, t.dtype))


def _scope(dev, stream):
    """Makes `dev` current, and `stream` too when one is given."""
    if stream is not None:
        if stream.device != dev:
            raise ValueError("stream is on %s, the tensors on %s" % (stream.device, dev))
        return torch.cuda.stream(stream)
    if dev.type != "cuda":
        raise ValueError("tensors must be on a GPU, got %s" % dev)
    return contextlib.nullcontext() if torch.cuda.current_device() == dev.index else torch.cuda.device(dev)


def _raw_stream(dev):
    return torch.cuda.current_stream(dev).cuda_stream


def _ptr(t):
    return None if t is None else t.data_ptr()


def _dense(t, name, shape, dtype, dev):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if t.device != dev:
        raise ValueError("%s is on %s, expected %s" % (name, t.device, dev))
    if t.dtype != dtype:
        raise ValueError("%s has dtype %s, expected %s" % (name, t.dtype, dtype))
    if t.shape != shape:
        raise ValueError("%s has shape %s, expected %s" % (name, tuple(t.shape), tuple(shape)))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    return t


def _pitch(t, name, shape, dtype, dev):
    """Distance in elements between the rows of `t` (0 when there is at most one)."""
    if t is None:
        return 0
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if t.device != dev:
        raise ValueError("%s is on %s, expected %s" % (name, t.device, dev))
    if t.dtype != dtype:
        raise ValueError("%s has dtype %s, expected %s" % (name, t.dtype, dtype))
    if t.shape != shape:
        raise ValueError("%s has shape %s, expected %s" % (name, tuple(t.shape), tuple(shape)))
    if t.is_contiguous():
        return 0
    *rows, d = shape
    if t.numel() == 0:
        return 0
    stride = t.stride()
    pitch, rest = None, 1   # rows counted from the innermost dimension outwards
    for n, s in zip(reversed(rows), reversed(stride[:-1])):
        if n == 1:
            continue
        pitch = s if pitch is None else pitch
        if s != pitch * rest:
            raise ValueError("%s: rows must be evenly spaced, got strides %s for shape %s" % (name, stride, tuple(shape)))
        rest *= n
    if (d > 1 and stride[-1] != 1) or (pitch is not None and pitch < d):
        raise ValueError("%s: rows must be dense and apart, got strides %s for shape %s" % (name, stride, tuple(shape)))
    return pitch or 0


def _workspace(workspace, need, dev):
    if need == 0:
        return None, 0
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    elif workspace.device != dev or not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous and on %s" % dev)
    return workspace, workspace.numel() * workspace.element_size()


def _scan_shape(x, cu_seqlens, h_in):
    """(batch, seqlen, D) of x [b, L, D], or [T, D] with offsets [b + 1]."""
    if cu_seqlens is None:
        if x.dim() != 3:
            raise ValueError("x must be [b, L, D] (or [T, D] with cu_seqlens), got %s" % (tuple(x.shape),))
        return tuple(x.shape)
    if x.dim() != 2:
        raise ValueError("x must be [T, D] with cu_seqlens, got %s" % (tuple(x.shape),))
    if cu_seqlens.dim() != 1 or cu_seqlens.shape[0] < 1:
        raise ValueError("cu_seqlens must be [b + 1], got %s" % (tuple(cu_seqlens.shape),))
    _dense(cu_seqlens, "cu_seqlens", cu_seqlens.shape, torch.int32, x.device)
    return cu_seqlens.shape[0] - 1, x.shape[0], x.shape[1]


def m3_gated_scan(gate, x, bias=None, h_in=None, cu_seqlens=None, y=None, h_out=None, states=None,
                  save_states=False, workspace=None, stream=None):
    """h_t = (1 - z_t) h_{t-1} + z_t x_t with z_t = sigmoid(gate_t + bias), over [b, L, D] or, with
    cu_seqlens [b + 1] int32, a packed [T, D].  bias [D], h_in [b, D] f32.  Returns (y, h_out), and
    with save_states (or states given) also the states m3_gated_scan_backward reads."""
    lib = load()
    b, L, D = _scan_shape(x, cu_seqlens, h_in)
    dev, io, shape = x.device, x.dtype, x.shape
    dims = M3ScanDims(b, L, D, _pitch(gate, "gate", shape, io, dev), _pitch(x, "x", shape, io, dev), 0, 0, 0,
                      _io_code(x, "x"), 0)
    _dense(bias, "bias", (D,), torch.float32, dev)
    _dense(h_in, "h_in", (b, D), torch.float32, dev)
    packed = cu_seqlens is not None
    with _scope(dev, stream):
        if y is None:
            y = torch.empty(shape, dtype=io, device=dev)
        dims.y_pitch = _pitch(y, "y", shape, io, dev)
        if h_out is None:
            h_out = torch.empty((b, D), dtype=torch.float32, device=dev)
        _dense(h_out, "h_out", (b, D), torch.float32, dev)
        if states is not None or save_states:
            want = (lib.m3_gated_scan_chunks(ctypes.byref(dims), packed), D)
            if states is None:
                states = torch.empty(want, dtype=torch.float32, device=dev)
            _dense(states, "states", want, torch.float32, dev)
        workspace, ws_bytes = _workspace(workspace, lib.m3_gated_scan_workspace_bytes(ctypes.byref(dims), packed), dev)
        _check(lib.m3_gated_scan(ctypes.byref(dims), _ptr(cu_seqlens), _ptr(gate), _ptr(x), _ptr(bias), _ptr(h_in),
                                 _ptr(y), _ptr(h_out), _ptr(states), _ptr(workspace), ws_bytes, _raw_stream(dev)))
    return (y, h_out) if states is None else (y, h_out, states)


def m3_gated_scan_step(gate, x, h, bias=None, y=None, h_out=None, stream=None):
    """One token: gate, x [b, D], state h [b, D] f32, updated in place unless h_out is given.
    Returns y."""
    lib = load()
    if x.dim() != 2:
        raise ValueError("x must be [b, D], got %s" % (tuple(x.shape),))
    dev, io, shape = x.device, x.dtype, x.shape
    b, D = shape
    dims = M3ScanDims(b, 1, D, _pitch(gate, "gate", shape, io, dev), _pitch(x, "x", shape, io, dev), 0, 0, 0,
                      _io_code(x, "x"), 0)
    _dense(bias, "bias", (D,), torch.float32, dev)
    _dense(h, "h", shape, torch.float32, dev)
    _dense(h_out, "h_out", shape, torch.float32, dev)
    with _scope(dev, stream):
        if y is None:
            y = torch.empty(shape, dtype=io, device=dev)
        dims.y_pitch = _pitch(y, "y", shape, io, dev)
        _check(lib.m3_gated_scan_step(ctypes.byref(dims), _ptr(gate), _ptr(x), _ptr(bias), _ptr(h), _ptr(y),
                                      _ptr(h if h_out is None else h_out), _raw_stream(dev)))
    return y


def m3_gated_scan_backward(gate, x, dy, states, bias=None, h_in=None, dh_out=None, cu_seqlens=None, grads=None,
                           workspace=None, stream=None):
    """Gradients of m3_gated_scan, from the states it saved.  dy like x; dh_out [b, D] f32 (None: 0).
    Returns a dict keyed by input name (gate, x, and bias, h_in where they were given); ``grads`` may
    supply preallocated tensors under those names."""
    lib = load()
    b, L, D = _scan_shape(x, cu_seqlens, h_in)
    dev, io, shape = x.device, x.dtype, x.shape
    f32 = torch.float32
    dims = M3ScanDims(b, L, D, _pitch(gate, "gate", shape, io, dev), _pitch(x, "x", shape, io, dev),
                      _pitch(dy, "dy", shape, io, dev), 0, 0, _io_code(x, "x"), 0)
    packed = cu_seqlens is not None
    _dense(bias, "bias", (D,), f32, dev)
    _dense(h_in, "h_in", (b, D), f32, dev)
    _dense(dh_out, "dh_out", (b, D), f32, dev)
    _dense(states, "states", (lib.m3_gated_scan_chunks(ctypes.byref(dims), packed), D), f32, dev)
    g = dict(grads or {})
    with _scope(dev, stream):
        for k in ("gate", "x"):
            if g.get(k) is None:
                g[k] = torch.empty(shape, dtype=io, device=dev)
        for k, given, want in (("bias", bias, (D,)), ("h_in", h_in, (b, D))):
            if g.get(k) is None and given is not None:
                g[k] = torch.empty(want, dtype=f32, device=dev)
            _dense(g.get(k), "grad " + k, want, f32, dev)
        dims.dgate_pitch = _pitch(g["gate"], "grad gate", shape, io, dev)
        dims.dx_pitch = _pitch(g["x"], "grad x", shape, io, dev)
        workspace, ws_bytes = _workspace(
            workspace, lib.m3_gated_scan_backward_workspace_bytes(ctypes.byref(dims), packed), dev)
        _check(lib.m3_gated_scan_backward(
            ctypes.byref(dims), _ptr(cu_seqlens), _ptr(gate), _ptr(x), _ptr(bias), _ptr(h_in), _ptr(states), _ptr(dy),
            _ptr(dh_out), _ptr(g["gate"]), _ptr(g["x"]), _ptr(g.get("bias")), _ptr(g.get("h_in")), _ptr(workspace),
            ws_bytes, _raw_stream(dev)))
    return g


def m3_rmsnorm(x, residual=None, weight=None, eps=1e-5, want_y=True, quant=False, group=0, r_out=None, y=None,
               q=None, scale=None, stream=None):
    """r = x + residual, n = r / sqrt(mean(r^2) + eps) * weight over the last dimension.  Returns (y, r_out,
    q, scale): y = n (None without want_y), r_out = r (None where there is no residual and none was
    passed), q = n / scale in float8_e4m3fn with scale f32 [..., 1] (group 0), or one for each `group`
    elements (both None without quant)."""
    lib = load()
    if x.dim() < 1:
        raise ValueError("x must have at least one dimension")
    dev, io, shape = x.device, x.dtype, x.shape
    D = shape[-1]
    rows = x.numel() // D if D else 0
    dims = M3NormDims(rows, D, _pitch(x, "x", shape, io, dev), _pitch(residual, "residual", shape, io, dev), 0, 0, 0,
                      group, _io_code(x, "x"), 0, eps)
    _dense(weight, "weight", (D,), torch.float32, dev)
    with _scope(dev, stream):
        if r_out is None and residual is not None:
            r_out = torch.empty(shape, dtype=io, device=dev)
        if y is None and want_y:
            y = torch.empty(shape, dtype=io, device=dev)
        if quant or q is not None or scale is not None:
            n = (-(-D // group) if group > 0 else 1) if D else 0
            if q is None:
                q = torch.empty(shape, dtype=torch.float8_e4m3fn, device=dev)
            if scale is None:
                scale = torch.empty((*shape[:-1], n), dtype=torch.float32, device=dev)
            _dense(q, "q", shape, torch.float8_e4m3fn, dev)
            _dense(scale, "scale", (*shape[:-1], n), torch.float32, dev)
        dims.r_pitch = _pitch(r_out, "r_out", shape, io, dev)
        dims.y_pitch = _pitch(y, "y", shape, io, dev)
        _check(lib.m3_rmsnorm(ctypes.byref(dims), _ptr(x), _ptr(residual), _ptr(weight), _ptr(r_out), _ptr(y), _ptr(q),
                              _ptr(scale), _raw_stream(dev)))
    return y, r_out, q, scale


def m3_rmsnorm_backward(r, dy, weight=None, dr_out=None, eps=1e-5, dx=None, dweight=None, workspace=None,
                        stream=None):
    """Gradients of the norm of r (m3_rmsnorm's r_out, or its x where there was no residual): dx, which is
    the gradient of x and of residual alike and takes the residual stream's dr_out in, and dweight
    (None where there is no weight and none was passed)."""
    lib = load()
    if r.dim() < 1:
        raise ValueError("r must have at least one dimension")
    dev, io, shape = r.device, r.dtype, r.shape
    D = shape[-1]
    rows = r.numel() // D if D else 0
    dims = M3NormDims(rows, D, 0, _pitch(dr_out, "dr_out", shape, io, dev), _pitch(r, "r", shape, io, dev),
                      _pitch(dy, "dy", shape, io, dev), 0, 0, _io_code(r, "r"), 0, eps)
    _dense(weight, "weight", (D,), torch.float32, dev)
    with _scope(dev, stream):
        if dx is None:
            dx = torch.empty(shape, dtype=io, device=dev)
        dims.dx_pitch = _pitch(dx, "dx", shape, io, dev)
        if dweight is None and weight is not None:
            dweight = torch.empty((D,), dtype=torch.float32, device=dev)
        _dense(dweight, "dweight", (D,), torch.float32, dev)
        need = lib.m3_rmsnorm_backward_workspace_bytes(ctypes.byref(dims)) if dweight is not None else 0
        workspace, ws_bytes = _workspace(workspace, need, dev)
        _check(lib.m3_rmsnorm_backward(ctypes.byref(dims), _ptr(r), _ptr(weight), _ptr(dy), _ptr(dr_out), _ptr(dx),
                                       _ptr(dweight), _ptr(workspace), ws_bytes, _raw_stream(dev)))
    return dx, dweight


def _grad_call(name, grads, max_norm, out, stats, workspace, stream):
    lib = load()
    pairs = []   # (gradient, where it goes)
    if isinstance(grads, dict):
        if out is not None and not isinstance(out, dict):
            raise TypeError("out must be a dict like grads")
        pairs = [(k, g, g if out is None else out[k]) for k, g in grads.items() if g is not None]
    else:
        grads = list(grads)
        dst = grads if out is None else list(out)
        if len(dst) != len(grads):
            raise ValueError("%d gradients, %d outputs" % (len(grads), len(dst)))
        pairs = [(i, g, o) for i, (g, o) in enumerate(zip(grads, dst)) if g is not None]
    dev = pairs[0][1].device if pairs else (stats.device if stats is not None else torch.device(
        "cuda", torch.cuda.current_device()))
    table = []
    for k, g, o in pairs:
        code = _io_code(g, "gradient %s" % k)
        if g.device != dev:
            raise ValueError("gradient %s is on %s, expected %s" % (k, g.device, dev))
        if not g.is_contiguous():
            raise ValueError("gradient %s must be contiguous" % k)
        if o is not g:
            _dense(o, "output %s" % k, g.shape, g.dtype, dev)
        table += (g.data_ptr(), o.data_ptr(), g.numel(), code)
    buf = array.array("Q", table)   # the fields of M3GradTensor, io and pad as one little-endian word
    ptr = buf.buffer_info()[0] if table else None
    with _scope(dev, stream):
        if stats is None:
            stats = torch.empty(2, dtype=torch.float32, device=dev)
        _dense(stats, "stats", (2,), torch.float32, dev)
        workspace, ws_bytes = _workspace(workspace, lib.m3_grad_workspace_bytes(ptr, len(pairs)), dev)
        _check(getattr(lib, name)(ptr, len(pairs), max_norm, _ptr(stats), _ptr(workspace), ws_bytes, _raw_stream(dev)))
    return stats


def m3_grad_norm(grads, max_norm=float("inf"), stats=None, workspace=None, stream=None):
    """2-norm over all elements of ``grads`` (a sequence, or a dict as the backward calls return; None
    entries are left out), and the factor that brings it to max_norm: returns stats = [norm, coef] f32
    on the device."""
    return _grad_call("m3_grad_norm", grads, max_norm, None, stats, workspace, stream)


def m3_grad_clip(grads, max_norm, out=None, stats=None, workspace=None, stream=None):
    """Scales all gradients by coef = min(1, max_norm / (norm + 1e-6)), in place or into ``out`` (tensors
    like them in a container like theirs).  Returns (grads or out, stats = [norm, coef])."""
    if not isinstance(grads, dict):
        grads = list(grads)
    stats = _grad_call("m3_grad_clip", grads, max_norm, out, stats, workspace, stream)
    return (grads if out is None else out), stats

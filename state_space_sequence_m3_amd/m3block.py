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
import ctypes
import functools

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


_new = torch.empty_like


def _io_code(t, name):
    if t.dtype is torch.bfloat16:
        return M3_BF16
    if t.dtype is torch.float32:
        return M3_F32
    raise ValueError("%s must be float32 or bfloat16, got %s" % (name, t.dtype))


# A call with small tensors takes a few microseconds on the GPU, so the host's share of it counts: the
# checks below try the ordinary case first, and device and stream are asked for as plain numbers.
_current_device = torch._C._cuda_getDevice if hasattr(torch._C, "_cuda_getDevice") else torch.cuda.current_device
_raw_stream = torch._C._cuda_getCurrentRawStream if hasattr(torch._C, "_cuda_getCurrentRawStream") else (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _here(t, stream):
    """The index of t's device if calls for it can be made as things are: it is the current device, and the
    current stream is meant.  -1: not so (see _scope)."""
    index = t.get_device()
    return index if stream is None and index >= 0 and index == _current_device() else -1


def _scope(t, stream):
    """Makes t's device current, and `stream` too when one is given."""
    if not t.is_cuda:
        raise ValueError("tensors must be on a GPU, got %s" % t.device)
    if stream is not None:
        if stream.device != t.device:
            raise ValueError("stream is on %s, the tensors on %s" % (stream.device, t.device))
        return torch.cuda.stream(stream)
    return torch.cuda.device(t.device)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _alike(t, name, shape, dtype, index):
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if t.get_device() != index:
        raise ValueError("%s is on %s, expected %s" % (name, t.device, "cuda:%d" % index if index >= 0 else "the CPU"))
    if t.dtype != dtype:
        raise ValueError("%s has dtype %s, expected %s" % (name, t.dtype, dtype))
    if t.shape != shape:
        raise ValueError("%s has shape %s, expected %s" % (name, tuple(t.shape), tuple(shape)))


def _dense(t, name, shape, dtype, index):
    """Checks a dense tensor (None passes) and returns its address."""
    if t is None:
        return None
    if isinstance(t, torch.Tensor) and t.get_device() == index and t.dtype is dtype and t.shape == shape \
            and t.is_contiguous():
        return t.data_ptr()
    _alike(t, name, shape, dtype, index)
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    return t.data_ptr()


def _pitch(t, name, shape, dtype, index):
    """Checks a tensor of rows (None passes) and returns the distance in elements between them (0: dense)."""
    if t is None:
        return 0
    if isinstance(t, torch.Tensor) and t.get_device() == index and t.dtype is dtype and t.shape == shape:
        if t.is_contiguous():
            return 0
        stride = t.stride()
        if len(stride) == 2 and stride[1] == 1 and stride[0] >= shape[1] and shape[0] > 1:
            return stride[0]
        if len(stride) == 3 and stride[2] == 1 and stride[1] >= shape[2] and shape[1] > 1 \
                and stride[0] == shape[1] * stride[1]:
            return stride[1]
    _alike(t, name, shape, dtype, index)
    if t.is_contiguous() or t.numel() == 0:
        return 0
    *rows, d = shape
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


def _workspace(workspace, need, x):
    if need == 0:
        return None, 0
    if workspace is None:
        return x.new_empty(need, dtype=torch.uint8), need
    if workspace.get_device() != x.get_device() or not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous and on %s" % x.device)
    return workspace, workspace.numel() * workspace.element_size()


def _scan_dims(x, cu_seqlens):
    """(batch, seqlen, D) of x [b, L, D], or [T, D] with offsets [b + 1]."""
    if cu_seqlens is None:
        if x.dim() != 3:
            raise ValueError("x must be [b, L, D] (or [T, D] with cu_seqlens), got %s" % (tuple(x.shape),))
        return x.shape
    if x.dim() != 2:
        raise ValueError("x must be [T, D] with cu_seqlens, got %s" % (tuple(x.shape),))
    if cu_seqlens.dim() != 1 or cu_seqlens.shape[0] < 1:
        raise ValueError("cu_seqlens must be [b + 1], got %s" % (tuple(cu_seqlens.shape),))
    _dense(cu_seqlens, "cu_seqlens", cu_seqlens.shape, torch.int32, x.get_device())
    return cu_seqlens.shape[0] - 1, x.shape[0], x.shape[1]


# Calls repeat their sizes, so the structures that carry them are kept (the library only reads them).
@functools.lru_cache(maxsize=1024)
def _scan_ref(*fields):
    return ctypes.byref(M3ScanDims(*fields))


@functools.lru_cache(maxsize=1024)
def _norm_ref(*fields):
    return ctypes.byref(M3NormDims(*fields))


@functools.lru_cache(maxsize=1024)
def _norm_workspace(rows, D, io, dev):
    """Workspace bytes of the norm's backward pass on device `dev`."""
    return load().m3_rmsnorm_backward_workspace_bytes(_norm_ref(rows, D, 0, 0, 0, 0, 0, 0, io, 0, 0.0))


@functools.lru_cache(maxsize=1024)
def _scan_sizes(b, L, D, io, packed, dev):
    """Rows of `states`, and the workspace bytes of the forward and the backward pass on device `dev`."""
    lib = load()
    ref = _scan_ref(b, L, D, 0, 0, 0, 0, 0, io, 0)
    return (lib.m3_gated_scan_chunks(ref, packed), lib.m3_gated_scan_workspace_bytes(ref, packed),
            lib.m3_gated_scan_backward_workspace_bytes(ref, packed))


def m3_gated_scan(gate, x, bias=None, h_in=None, cu_seqlens=None, y=None, h_out=None, states=None,
                  save_states=False, workspace=None, stream=None):
    """h_t = (1 - z_t) h_{t-1} + z_t x_t with z_t = sigmoid(gate_t + bias), over [b, L, D] or, with
    cu_seqlens [b + 1] int32, a packed [T, D].  bias [D], h_in [b, D] f32.  Returns (y, h_out), and
    with save_states (or states given) also the states m3_gated_scan_backward reads."""
    lib = _lib or load()
    b, L, D = _scan_dims(x, cu_seqlens)
    io, shape, dev, f32 = x.dtype, x.shape, x.get_device(), torch.float32
    packed = cu_seqlens is not None
    code = _io_code(x, "x")
    ref = _scan_ref(b, L, D, _pitch(gate, "gate", shape, io, dev), _pitch(x, "x", shape, io, dev),
                    _pitch(y, "y", shape, io, dev), 0, 0, code, 0)
    bias_p, h_in_p = _dense(bias, "bias", (D,), f32, dev), _dense(h_in, "h_in", (b, D), f32, dev)
    h_out_p = _dense(h_out, "h_out", (b, D), f32, dev)
    at = _here(x, stream)
    if at < 0:
        with _scope(x, stream):
            return m3_gated_scan(gate, x, bias, h_in, cu_seqlens, y, h_out, states, save_states, workspace)
    rows, need, _ = _scan_sizes(b, L, D, code, packed, at)
    if y is None:
        y = x.new_empty(shape)
    if h_out is None:
        h_out = x.new_empty((b, D), dtype=f32)
        h_out_p = h_out.data_ptr()
    if states is not None or save_states:
        if states is None:
            states = x.new_empty((rows, D), dtype=f32)
        else:
            _dense(states, "states", (rows, D), f32, dev)
    workspace, ws_bytes = _workspace(workspace, need, x)
    _check(lib.m3_gated_scan(ref, _ptr(cu_seqlens), gate.data_ptr(), x.data_ptr(), bias_p, h_in_p,
                             y.data_ptr(), h_out_p, _ptr(states), _ptr(workspace), ws_bytes, _raw_stream(at)))
    return (y, h_out) if states is None else (y, h_out, states)


def m3_gated_scan_step(gate, x, h, bias=None, y=None, h_out=None, stream=None):
    """One token: gate, x [b, D], state h [b, D] f32, updated in place unless h_out is given.
    Returns y."""
    lib = _lib or load()
    shape, io, dev, f32 = x.shape, x.dtype, x.get_device(), torch.float32
    if len(shape) != 2:
        raise ValueError("x must be [b, D], got %s" % (tuple(shape),))
    b, D = shape
    dense = x.is_contiguous()
    xp = 0 if dense else _pitch(x, "x", shape, io, dev)
    ref = _scan_ref(b, 1, D, _pitch(gate, "gate", shape, io, dev), xp,
                    0 if y is None else _pitch(y, "y", shape, io, dev), 0, 0, _io_code(x, "x"), 0)
    bias_p = None if bias is None else _dense(bias, "bias", (D,), f32, dev)
    h_p = h_out_p = _dense(h, "h", shape, f32, dev)
    if h_out is not None:
        h_out_p = _dense(h_out, "h_out", shape, f32, dev)
    if stream is not None or dev < 0 or dev != _current_device():
        with _scope(x, stream):
            return m3_gated_scan_step(gate, x, h, bias, y, h_out)
    if y is None:
        y = _new(x) if dense else x.new_empty(shape)
    status = lib.m3_gated_scan_step(ref, gate.data_ptr(), x.data_ptr(), bias_p, h_p, y.data_ptr(),
                                    h_out_p, _raw_stream(dev))
    if status:
        _check(status)
    return y


def m3_gated_scan_backward(gate, x, dy, states, bias=None, h_in=None, dh_out=None, cu_seqlens=None, grads=None,
                           workspace=None, stream=None):
    """Gradients of m3_gated_scan, from the states it saved.  dy like x; dh_out [b, D] f32 (None: 0).
    Returns a dict keyed by input name (gate, x, and bias, h_in where they were given); ``grads`` may
    supply preallocated tensors under those names."""
    lib = _lib or load()
    b, L, D = _scan_dims(x, cu_seqlens)
    io, shape, dev, f32 = x.dtype, x.shape, x.get_device(), torch.float32
    packed = cu_seqlens is not None
    g = dict(grads) if grads else {}
    code = _io_code(x, "x")
    ref = _scan_ref(b, L, D, _pitch(gate, "gate", shape, io, dev), _pitch(x, "x", shape, io, dev),
                    _pitch(dy, "dy", shape, io, dev), _pitch(g.get("gate"), "grad gate", shape, io, dev),
                    _pitch(g.get("x"), "grad x", shape, io, dev), code, 0)
    bias_p, h_in_p = _dense(bias, "bias", (D,), f32, dev), _dense(h_in, "h_in", (b, D), f32, dev)
    dh_out_p = _dense(dh_out, "dh_out", (b, D), f32, dev)
    _dense(g.get("bias"), "grad bias", (D,), f32, dev)
    _dense(g.get("h_in"), "grad h_in", (b, D), f32, dev)
    at = _here(x, stream)
    if at < 0:
        with _scope(x, stream):
            return m3_gated_scan_backward(gate, x, dy, states, bias, h_in, dh_out, cu_seqlens, grads, workspace)
    rows, _, need = _scan_sizes(b, L, D, code, packed, at)
    states_p = _dense(states, "states", (rows, D), f32, dev)
    if states_p is None:
        raise ValueError("states are required: m3_gated_scan(..., save_states=True) returns them")
    for k in ("gate", "x"):
        if g.get(k) is None:
            g[k] = x.new_empty(shape)
    if bias is not None and g.get("bias") is None:
        g["bias"] = x.new_empty((D,), dtype=f32)
    if h_in is not None and g.get("h_in") is None:
        g["h_in"] = x.new_empty((b, D), dtype=f32)
    workspace, ws_bytes = _workspace(workspace, need, x)
    _check(lib.m3_gated_scan_backward(
        ref, _ptr(cu_seqlens), gate.data_ptr(), x.data_ptr(), bias_p, h_in_p, states_p, dy.data_ptr(),
        dh_out_p, g["gate"].data_ptr(), g["x"].data_ptr(), _ptr(g.get("bias")), _ptr(g.get("h_in")), _ptr(workspace),
        ws_bytes, _raw_stream(at)))
    return g


def m3_rmsnorm(x, residual=None, weight=None, eps=1e-5, want_y=True, quant=False, group=0, r_out=None, y=None,
               q=None, scale=None, stream=None):
    """r = x + residual, n = r / sqrt(mean(r^2) + eps) * weight over the last dimension.  Returns (y, r_out,
    q, scale): y = n (None without want_y), r_out = r (None where there is no residual and none was
    passed), q = n / scale in float8_e4m3fn with scale f32 [..., 1] (group 0), or one for each `group`
    elements (both None without quant)."""
    lib = _lib or load()
    io, shape, dev, f32 = x.dtype, x.shape, x.get_device(), torch.float32
    if not shape:
        raise ValueError("x must have at least one dimension")
    D = shape[-1]
    dense = x.is_contiguous()
    xp = 0 if dense else _pitch(x, "x", shape, io, dev)
    pp = 0 if residual is None else _pitch(residual, "residual", shape, io, dev)
    rp = 0 if r_out is None else _pitch(r_out, "r_out", shape, io, dev)
    yp = 0 if y is None else _pitch(y, "y", shape, io, dev)
    ref = _norm_ref(x.numel() // D if D else 0, D, xp, pp, rp, yp, 0, group, _io_code(x, "x"), 0, eps)
    weight_p = None if weight is None else _dense(weight, "weight", (D,), f32, dev)
    if stream is not None or dev < 0 or dev != _current_device():
        with _scope(x, stream):
            return m3_rmsnorm(x, residual, weight, eps, want_y, quant, group, r_out, y, q, scale)
    if r_out is None and residual is not None:
        r_out = _new(x) if dense else x.new_empty(shape)
    if y is None and want_y:
        y = _new(x) if dense else x.new_empty(shape)
    if quant or q is not None or scale is not None:
        sshape = (*shape[:-1], (-(-D // group) if group > 0 else 1) if D else 0)
        if q is None:
            q = x.new_empty(shape, dtype=torch.float8_e4m3fn)
        else:
            _dense(q, "q", shape, torch.float8_e4m3fn, dev)
        if scale is None:
            scale = x.new_empty(sshape, dtype=f32)
        else:
            _dense(scale, "scale", sshape, f32, dev)
    status = lib.m3_rmsnorm(ref, x.data_ptr(), _ptr(residual), weight_p, _ptr(r_out), _ptr(y), _ptr(q),
                            _ptr(scale), _raw_stream(dev))
    if status:
        _check(status)
    return y, r_out, q, scale


def m3_rmsnorm_backward(r, dy, weight=None, dr_out=None, eps=1e-5, dx=None, dweight=None, workspace=None,
                        stream=None):
    """Gradients of the norm of r (m3_rmsnorm's r_out, or its x where there was no residual): dx, which is
    the gradient of x and of residual alike and takes the residual stream's dr_out in, and dweight
    (None where there is no weight and none was passed)."""
    lib = _lib or load()
    io, shape, dev, f32 = r.dtype, r.shape, r.get_device(), torch.float32
    if not shape:
        raise ValueError("r must have at least one dimension")
    D = shape[-1]
    ref = _norm_ref(r.numel() // D if D else 0, D, 0, _pitch(dr_out, "dr_out", shape, io, dev),
                    _pitch(r, "r", shape, io, dev), _pitch(dy, "dy", shape, io, dev),
                    _pitch(dx, "dx", shape, io, dev), 0, _io_code(r, "r"), 0, eps)
    weight_p = _dense(weight, "weight", (D,), f32, dev)
    _dense(dweight, "dweight", (D,), f32, dev)
    at = _here(r, stream)
    if at < 0:
        with _scope(r, stream):
            return m3_rmsnorm_backward(r, dy, weight, dr_out, eps, dx, dweight, workspace)
    if dx is None:
        dx = r.new_empty(shape)
    if dweight is None and weight is not None:
        dweight = r.new_empty((D,), dtype=f32)
    need = _norm_workspace(r.numel() // D if D else 0, D, _io_code(r, "r"), at) if dweight is not None else 0
    workspace, ws_bytes = _workspace(workspace, need, r)
    _check(lib.m3_rmsnorm_backward(ref, r.data_ptr(), weight_p, dy.data_ptr(), _ptr(dr_out), dx.data_ptr(), _ptr(dweight),
                                   _ptr(workspace), ws_bytes, _raw_stream(at)))
    return dx, dweight


def _grad_call(fn, grads, max_norm, out, stats, workspace, stream):
    lib = _lib or load()
    if isinstance(grads, dict):
        if out is not None and not isinstance(out, dict):
            raise TypeError("out must be a dict like grads")
        names = [k for k, g in grads.items() if g is not None]
        src, dst = [grads[k] for k in names], None if out is None else [out[k] for k in names]
    else:
        if out is not None and len(out) != len(grads):
            raise ValueError("%d gradients, %d outputs" % (len(grads), len(out)))
        names = [i for i, g in enumerate(grads) if g is not None]
        src, dst = [grads[i] for i in names], None if out is None else [out[i] for i in names]
    if not src and stats is None:
        stats = torch.empty(2, dtype=torch.float32, device="cuda")
    first = src[0] if src else stats
    dev, f32, bf16 = first.get_device(), torch.float32, torch.bfloat16
    table = []   # the fields of M3GradTensor, io and pad as one little-endian word
    for i, g in enumerate(src):
        dtype = g.dtype
        if (dtype is not f32 and dtype is not bf16) or g.get_device() != dev or not g.is_contiguous():
            _io_code(g, "gradient %s" % names[i])
            _dense(g, "gradient %s" % names[i], g.shape, dtype, dev)
        p = o = g.data_ptr()
        if dst is not None:
            t = dst[i]
            if t is None:
                raise ValueError("output %s is None" % names[i])
            if t is not g:
                o = _dense(t, "output", g.shape, dtype, dev)
        table += (p, o, g.numel(), M3_F32 if dtype is f32 else M3_BF16)
    stats_p = _dense(stats, "stats", (2,), f32, dev)
    at = _here(first, stream)
    if at < 0:
        with _scope(first, stream):
            return _grad_call(fn, grads, max_norm, out, stats, workspace, None)
    if stats is None:
        stats = first.new_empty(2, dtype=f32)
        stats_p = stats.data_ptr()
    buf = array.array("Q", table)
    ptr = buf.buffer_info()[0] if src else None
    workspace, ws_bytes = _workspace(workspace, lib.m3_grad_workspace_bytes(ptr, len(src)), first)
    _check(getattr(lib, fn)(ptr, len(src), max_norm, stats_p, _ptr(workspace), ws_bytes, _raw_stream(at)))
    return stats


def m3_grad_norm(grads, max_norm=float("inf"), stats=None, workspace=None, stream=None):
    """2-norm over all elements of ``grads`` (a sequence, or a dict as the backward calls return; None
    entries are left out), and the factor that brings it to max_norm: returns stats = [norm, coef] f32
    on the device."""
    if not isinstance(grads, (dict, list, tuple)):
        grads = list(grads)
    return _grad_call("m3_grad_norm", grads, max_norm, None, stats, workspace, stream)


def m3_grad_clip(grads, max_norm, out=None, stats=None, workspace=None, stream=None):
    """Scales all gradients by coef = min(1, max_norm / (norm + 1e-6)), in place or into ``out`` (tensors
    like them in a container like theirs).  Returns (grads or out, stats = [norm, coef])."""
    if not isinstance(grads, (dict, list, tuple)):
        grads = list(grads)
    if out is not None and not isinstance(out, (dict, list, tuple)):
        out = list(out)
    stats = _grad_call("m3_grad_clip", grads, max_norm, out, stats, workspace, stream)
    return (grads if out is None else out), stats

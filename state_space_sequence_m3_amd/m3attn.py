"""ctypes binding of the attention operators of libm3scan with the names of the C ABI (include/m3attn.h): causal
attention over whole prompts with its gradient, appending to a paged cache, one token's attention over it.

Like m3block.py it only marshals: it checks placement, dtype, shape and strides, allocates outputs and workspaces with
torch when they are not passed, and turns a non-OK status into an M3Error.  There is no fallback.  Calls run on the
tensors' device, whichever is current, on its current stream or on ``stream``; what they allocate belongs to that
stream.

Tensors of heads ([b, L, H, D], packed [T, H, D]) may have any strides that are multiples of 16 bytes, as long as the
last dimension is dense: slices of one projection, or heads before tokens through ``.transpose(1, 2)``.
"""
from __future__ import annotations

import ctypes
import functools

import torch

from . import m3scan
from .m3block import _alike, _check, _current_device, _dense, _io_code, _new, _ptr, _raw_stream, _scope, _workspace
from .m3scan import M3_BF16, M3_F32, M3Error, STATUS_NAMES  # noqa: F401

EXPORTED = ["m3_attention", "m3_attention_backward_workspace_bytes", "m3_attention_backward", "m3_cache_append",
            "m3_attention_step_workspace_bytes", "m3_attention_step"]

M3_ROTATE_HALVES = 1

_S = ctypes.c_int64 * 3


class M3AttnDims(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int64), ("seqlen", ctypes.c_int64), ("heads", ctypes.c_int64),
                ("kv_heads", ctypes.c_int64), ("head_dim", ctypes.c_int64), ("q", _S), ("k", _S), ("v", _S), ("o", _S),
                ("dout", _S), ("dq", _S), ("dk", _S), ("dv", _S), ("io", ctypes.c_int32), ("flags", ctypes.c_uint32),
                ("scale", ctypes.c_float)]


class M3CacheDims(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int64), ("seqlen", ctypes.c_int64), ("heads", ctypes.c_int64),
                ("kv_heads", ctypes.c_int64), ("head_dim", ctypes.c_int64), ("num_pages", ctypes.c_int64),
                ("page_size", ctypes.c_int64), ("table_width", ctypes.c_int64), ("rotary_dim", ctypes.c_int64),
                ("k_cache", _S), ("v_cache", _S), ("q", _S), ("k", _S), ("v", _S), ("q_out", _S), ("k_out", _S),
                ("o", _S), ("io", ctypes.c_int32), ("flags", ctypes.c_uint32), ("scale", ctypes.c_float)]


_P = ctypes.c_void_p
_Z = ctypes.c_size_t
_lib = None


def load():
    """The library with the signatures of m3attn.h declared (see m3scan.load)."""
    global _lib
    if _lib is None:
        lib = m3scan.load()
        attn, cache = ctypes.POINTER(M3AttnDims), ctypes.POINTER(M3CacheDims)
        st = ctypes.c_int
        for name, res, args in [
                ("m3_attention", st, [attn] + [_P] * 7),
                ("m3_attention_backward_workspace_bytes", _Z, [attn, st]),
                ("m3_attention_backward", st, [attn] + [_P] * 11 + [_Z, _P]),
                ("m3_cache_append", st, [cache] + [_P] * 12),
                ("m3_attention_step_workspace_bytes", _Z, [cache]),
                ("m3_attention_step", st, [cache] + [_P] * 8 + [_Z, _P])]:
            fn = getattr(lib, name)
            fn.restype, fn.argtypes = res, args
        _lib = lib
    return _lib


_DENSE = (0, 0, 0)


# Calls repeat their sizes, so the structures that carry them are kept (the library only reads them).
@functools.lru_cache(maxsize=1024)
def _attn_ref(*fields):
    return ctypes.byref(M3AttnDims(*fields))


@functools.lru_cache(maxsize=1024)
def _cache_ref(*fields):
    return ctypes.byref(M3CacheDims(*fields))


@functools.lru_cache(maxsize=1024)
def _step_workspace(b, hq, hk, d, pages, page, width, io, dev):
    """Workspace bytes of a step on device `dev`."""
    return load().m3_attention_step_workspace_bytes(
        _cache_ref(b, 1, hq, hk, d, pages, page, width, 0, *[_DENSE] * 8, io, 0, 0.0))


def _heads(t, name, shape, dtype, index):
    """Checks a tensor of heads (None passes) and returns its (batch, token, head) strides; dense: zeros."""
    if t is None:
        return _DENSE
    if not (isinstance(t, torch.Tensor) and t.shape == shape and t.dtype is dtype and t.get_device() == index):
        _alike(t, name, shape, dtype, index)
    if t.is_contiguous():
        return _DENSE
    stride = t.stride()
    if stride[-1] != 1:
        raise ValueError("%s: heads must be dense, got strides %s for shape %s" % (name, stride, tuple(shape)))
    s = stride[:-1] if len(stride) == 4 else (0, *stride[:-1])
    if s == _DENSE:
        raise ValueError("%s: strides of 0 throughout are not supported, for shape %s" % (name, tuple(shape)))
    return s


def _like(t, dense):
    """An output like t, dense."""
    return _new(t) if dense is _DENSE else t.new_empty(t.shape)


def _scale(scale):
    if scale is None:
        return 0.0
    if not scale > 2.0 ** -150:   # what fp32 rounds to 0, the default's mark
        raise ValueError("scale must be positive in float32, got %s" % (scale,))
    return scale


def _prompt_shape(q, k, cu_seqlens):
    """(b, L, Hq, Hkv, D) of q [b, L, Hq, D], or [T, Hq, D] with offsets [b + 1], and the shape of k and v."""
    if cu_seqlens is None:
        try:
            b, L, hq, d = q.shape
        except ValueError:
            raise ValueError("q must be [b, L, H, D] (or [T, H, D] with cu_seqlens), got %s" % (tuple(q.shape),)) from None
        if k.dim() != 4:
            raise ValueError("k must be like q but for its heads, got %s" % (tuple(k.shape),))
        hk = k.shape[2]
        return (b, L, hq, hk, d), (b, L, hk, d)
    shape = q.shape
    if len(shape) != 3:
        raise ValueError("q must be [b, L, H, D] (or [T, H, D] with cu_seqlens), got %s" % (tuple(shape),))
    if k.dim() != 3:
        raise ValueError("k must be like q but for its heads, got %s" % (tuple(k.shape),))
    hk = k.shape[1]
    kv = (shape[0], hk, shape[2])
    if cu_seqlens.dim() != 1 or cu_seqlens.shape[0] < 1:
        raise ValueError("cu_seqlens must be [b + 1], got %s" % (tuple(cu_seqlens.shape),))
    _dense(cu_seqlens, "cu_seqlens", cu_seqlens.shape, torch.int32, q.get_device())
    return (cu_seqlens.shape[0] - 1, shape[0], shape[1], hk, shape[2]), kv


def _lse_shape(sizes, packed):
    b, L, hq = sizes[:3]
    return (hq, L) if packed else (b, hq, L)


def m3_attention(q, k, v, cu_seqlens=None, scale=None, o=None, lse=None, save_lse=False, stream=None):
    """Causal softmax(scale q k^T) v of q [b, L, Hq, D] with k, v [b, L, Hkv, D], or with cu_seqlens [b + 1] int32
    packed [T, H, D].  scale: 1 / sqrt(D) where None.  Returns o like q, and with save_lse (or lse given)
    also the lse [b, Hq, L], packed [Hq, T] f32 that m3_attention_backward reads."""
    lib = _lib or load()
    sizes, kv = _prompt_shape(q, k, cu_seqlens)
    io, shape, dev = q.dtype, q.shape, q.get_device()
    packed = cu_seqlens is not None
    qs = _heads(q, "q", shape, io, dev)
    ref = _attn_ref(*sizes, qs, _heads(k, "k", kv, io, dev), _heads(v, "v", kv, io, dev), _heads(o, "o", shape, io, dev),
                    _DENSE, _DENSE, _DENSE, _DENSE, _io_code(q, "q"), 0, _scale(scale))
    if lse is not None:
        _dense(lse, "lse", _lse_shape(sizes, packed), torch.float32, dev)
    if stream is not None or dev < 0 or dev != _current_device():
        with _scope(q, stream):
            return m3_attention(q, k, v, cu_seqlens, scale, o, lse, save_lse)
    if o is None:
        o = _like(q, qs)
    if lse is None and save_lse:
        lse = q.new_empty(_lse_shape(sizes, packed), dtype=torch.float32)
    status = lib.m3_attention(ref, _ptr(cu_seqlens), q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), _ptr(lse),
                              _raw_stream(dev))
    if status:
        _check(status)
    return o if lse is None else (o, lse)


def m3_attention_backward(q, k, v, o, lse, dout, cu_seqlens=None, scale=None, grads=None, workspace=None, stream=None):
    """Gradients of m3_attention, from its o and lse and the loss's gradient dout of o.  Returns a dict keyed by input
    name (q, k, v); ``grads`` may supply preallocated tensors under those names."""
    lib = _lib or load()
    sizes, kv = _prompt_shape(q, k, cu_seqlens)
    io, shape, dev = q.dtype, q.shape, q.get_device()
    packed = cu_seqlens is not None
    g = dict(grads) if grads else {}
    code = _io_code(q, "q")
    ref = _attn_ref(*sizes, _heads(q, "q", shape, io, dev), _heads(k, "k", kv, io, dev), _heads(v, "v", kv, io, dev),
                    _heads(o, "o", shape, io, dev), _heads(dout, "dout", shape, io, dev),
                    _heads(g.get("q"), "grad q", shape, io, dev), _heads(g.get("k"), "grad k", kv, io, dev),
                    _heads(g.get("v"), "grad v", kv, io, dev), code, 0, _scale(scale))
    lse_p = _dense(lse, "lse", _lse_shape(sizes, packed), torch.float32, dev)
    if lse_p is None:
        raise ValueError("lse is required: m3_attention(..., save_lse=True) returns it")
    if stream is not None or dev < 0 or dev != _current_device():
        with _scope(q, stream):
            return m3_attention_backward(q, k, v, o, lse, dout, cu_seqlens, scale, grads, workspace)
    for name, like in (("q", shape), ("k", kv), ("v", kv)):
        if g.get(name) is None:
            g[name] = q.new_empty(like)
    workspace, ws_bytes = _workspace(workspace, lib.m3_attention_backward_workspace_bytes(ref, packed), q)
    status = lib.m3_attention_backward(ref, _ptr(cu_seqlens), q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse_p,
                                       dout.data_ptr(), g["q"].data_ptr(), g["k"].data_ptr(), g["v"].data_ptr(),
                                       _ptr(workspace), ws_bytes, _raw_stream(dev))
    if status:
        _check(status)
    return g


def _cache_shape(k_cache, v_cache, page_table, b, hk, d, io, dev):
    """(pages, page size, table width) and the caches' (page, token, head) strides, checked."""
    shape = k_cache.shape
    if len(shape) != 4:
        raise ValueError("k_cache must be [pages, H, page_size, D], got %s" % (tuple(shape),))
    pages, h, page, width = shape
    if h != hk or width != d:
        _alike(k_cache, "k_cache", (pages, hk, page, d), io, dev)
    ks, vs = _heads(k_cache, "k_cache", shape, io, dev), _heads(v_cache, "v_cache", shape, io, dev)
    if ks is not _DENSE:
        ks = (ks[0], ks[2], ks[1])
    if vs is not _DENSE:
        vs = (vs[0], vs[2], vs[1])
    if page_table is None or page_table.dim() != 2:
        raise ValueError("page_table must be [b, pages of a sequence]")
    width = page_table.shape[1]
    _dense(page_table, "page_table", (b, width), torch.int32, dev)
    return pages, page, width, ks, vs


def m3_cache_append(k, v, k_cache=None, v_cache=None, page_table=None, lens=None, q=None, inv_freq=None, halves=False,
                    cu_seqlens=None, q_out=None, k_out=None, stream=None):
    """Writes the new tokens' k, v [b, n, Hkv, D], or with cu_seqlens packed [T, Hkv, D], into the caches
    [pages, Hkv, page_size, D] at the positions before lens [b] int32 (their number with the new ones; None: n),
    through page_table [b, pages of a sequence] int32.  inv_freq [r / 2] f32: the first r elements of every head of k
    and q are rotated by position * inv_freq, in pairs (2k, 2k + 1), with ``halves`` (k, k + r / 2).  Returns q_out,
    the rotated q (None without q); k_out, where given, takes the rotated k.  Without caches (all None) only those
    are written."""
    lib = _lib or load()
    like = k if q is None else q
    sizes, kv = _prompt_shape(like, k, cu_seqlens)
    b, L, hq, hk, d = sizes
    io, dev, f32 = k.dtype, k.get_device(), torch.float32
    shape = like.shape
    if q is None:
        if q_out is not None:
            raise ValueError("q_out without q")
        hq = hk
    qs = _DENSE if q is None else _heads(q, "q", shape, io, dev)
    ks, vs = _heads(k, "k", kv, io, dev), _heads(v, "v", kv, io, dev)
    kos = _DENSE if k_out is None else _heads(k_out, "k_out", kv, io, dev)
    if lens is not None:
        _dense(lens, "lens", (b,), torch.int32, dev)
    rot = 0
    if inv_freq is not None:
        if inv_freq.dim() != 1:
            raise ValueError("inv_freq must be [r / 2], got %s" % (tuple(inv_freq.shape),))
        _dense(inv_freq, "inv_freq", inv_freq.shape, f32, dev)
        rot = 2 * inv_freq.shape[0]
    pages, page, width, kcs, vcs = 0, 1, 0, _DENSE, _DENSE
    if k_cache is not None or v_cache is not None or page_table is not None:
        if k_cache is None or v_cache is None or page_table is None or v is None:
            raise ValueError("k_cache, v_cache, page_table and v go together")
        pages, page, width, kcs, vcs = _cache_shape(k_cache, v_cache, page_table, b, hk, d, io, dev)
    qos = _DENSE if q_out is None else _heads(q_out, "q_out", shape, io, dev)
    ref = _cache_ref(b, L, hq, hk, d, pages, page, width, rot, kcs, vcs, qs, ks, vs, qos, kos, _DENSE, _io_code(k, "k"),
                     M3_ROTATE_HALVES if halves else 0, 0.0)
    if stream is not None or dev < 0 or dev != _current_device():
        with _scope(k, stream):
            return m3_cache_append(k, v, k_cache, v_cache, page_table, lens, q, inv_freq, halves, cu_seqlens, q_out, k_out)
    if q is not None and q_out is None:
        q_out = _like(q, qs)
    status = lib.m3_cache_append(ref, _ptr(cu_seqlens), _ptr(lens), _ptr(inv_freq), _ptr(q), k.data_ptr(), _ptr(v),
                                 _ptr(q_out), _ptr(k_out), _ptr(k_cache), _ptr(v_cache), _ptr(page_table), _raw_stream(dev))
    if status:
        _check(status)
    return q_out


def m3_attention_step(q, k_cache, v_cache, page_table, lens, scale=None, o=None, lse=None, workspace=None, stream=None):
    """One token per sequence: softmax(scale q k^T) v of q [b, Hq, D] over the first lens[s] positions of the caches
    [pages, Hkv, page_size, D] (arguments as m3_cache_append's).  Returns o like q (zeros where there is no
    position); lse [b, Hq] f32, where given, takes the scores' log sum of exponentials."""
    lib = _lib or load()
    shape, io, dev = q.shape, q.dtype, q.get_device()
    if len(shape) != 3:
        raise ValueError("q must be [b, H, D], got %s" % (tuple(shape),))
    b, hq, d = shape
    hk = k_cache.shape[1] if k_cache.dim() == 4 else 0
    pages, page, width, kcs, vcs = _cache_shape(k_cache, v_cache, page_table, b, hk, d, io, dev)
    if _dense(lens, "lens", (b,), torch.int32, dev) is None:
        raise ValueError("lens is required")
    code = _io_code(q, "q")
    dense = _heads(q, "q", shape, io, dev)
    _, qb, qh = dense
    _, ob, oh = _DENSE if o is None else _heads(o, "o", shape, io, dev)
    ref = _cache_ref(b, 1, hq, hk, d, pages, page, width, 0, kcs, vcs, (qb, 0, qh), _DENSE, _DENSE, _DENSE, _DENSE,
                     (ob, 0, oh), code, 0, _scale(scale))
    if lse is not None:
        _dense(lse, "lse", (b, hq), torch.float32, dev)
    if stream is not None or dev < 0 or dev != _current_device():
        with _scope(q, stream):
            return m3_attention_step(q, k_cache, v_cache, page_table, lens, scale, o, lse, workspace)
    if o is None:
        o = _like(q, dense)
    workspace, ws_bytes = _workspace(workspace, _step_workspace(b, hq, hk, d, pages, page, width, code, dev), q)
    status = lib.m3_attention_step(ref, q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), page_table.data_ptr(),
                                   lens.data_ptr(), o.data_ptr(), _ptr(lse), _ptr(workspace), ws_bytes, _raw_stream(dev))
    if status:
        _check(status)
    return o

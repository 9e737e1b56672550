"""Python side of include/conv_train.h: the operators a training step runs around the conv
layers -- group norm with an activation, embedding lookup and its gradient, the global gradient
norm and clipping.

The functions named like the C entry points (conv_gn_fwd, conv_embed_bwd, conv_grad_clip, ...)
take a descriptor and already-allocated CUDA tensors, like those of ``binding``.  group_norm,
group_norm_bwd, embed, embed_bwd, grad_norm and clip_grads check shapes and types and allocate
outputs and workspaces with torch first.  Everything is enqueued on the current torch stream (or
the stream given) and nothing waits for the GPU; tensors made on another stream have to be
ordered by the caller (``stream.wait_stream``), as for any torch operation.  What the allocating
functions allocate belongs to the stream they run on."""
from __future__ import annotations

import array
import ctypes
import functools
import itertools
import threading

import torch

from . import binding
from .binding import _check, _ptr, _stream

LAYOUTS = {"nchw": 0, "nhwc": 1}
ACTS = {"none": 0, "relu": 1, "silu": 2, "gelu": 3}
_DT = {torch.float32: 0, torch.bfloat16: 1}
_IDX = {torch.int32: 0, torch.int64: 1}

EXPORTS = ["conv_gn_fwd_workspace_size", "conv_gn_fwd", "conv_gn_bwd_workspace_size", "conv_gn_bwd",
           "conv_embed_fwd", "conv_embed_bwd_workspace_size", "conv_embed_bwd",
           "conv_grad_norm_workspace_size", "conv_grad_norm", "conv_grad_clip"]


class GnDesc(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("B", "C", "P", "G", "act", "layout", "dtype")] + \
        [("eps", ctypes.c_float)]


class EmbedDesc(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int64)] + \
        [(n, ctypes.c_int32) for n in ("V", "D", "padding_idx", "index_dtype", "dtype")] + [("scale", ctypes.c_float)]


class Grad(ctypes.Structure):
    _fields_ = [("grad", ctypes.c_void_p), ("out", ctypes.c_void_p), ("n", ctypes.c_int64), ("dtype", ctypes.c_int64)]


_lock = threading.Lock()
_lib = None


def lib():
    """The CUDA library with this header's signatures set.  Raises if it has not been built."""
    global _lib
    if _lib is None:
        L = binding.lib()
        with _lock:
            vp, sz, i32 = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int32
            L.conv_gn_fwd_workspace_size.argtypes = [vp]
            L.conv_gn_fwd_workspace_size.restype = sz
            L.conv_gn_fwd.argtypes = [vp] * 8 + [sz, vp]
            L.conv_gn_bwd_workspace_size.argtypes = [vp]
            L.conv_gn_bwd_workspace_size.restype = sz
            L.conv_gn_bwd.argtypes = [vp] * 11 + [sz, vp]
            L.conv_embed_fwd.argtypes = [vp] * 5
            L.conv_embed_bwd_workspace_size.argtypes = [vp]
            L.conv_embed_bwd_workspace_size.restype = sz
            L.conv_embed_bwd.argtypes = [vp] * 5 + [sz, vp]
            L.conv_grad_norm_workspace_size.argtypes = [vp, i32]
            L.conv_grad_norm_workspace_size.restype = sz
            L.conv_grad_norm.argtypes = [vp, i32, vp, vp, sz, vp]
            L.conv_grad_clip.argtypes = [vp, i32, ctypes.c_float, vp, vp, sz, vp]
            _lib = L
    return _lib


def _ref(desc):
    return ctypes.addressof(desc)


def _bytes(ws) -> int:
    return 0 if ws is None else ws.numel() * ws.element_size()


# The allocating functions are called once or more a layer and step, and a small call's time is
# the host's: they pass plain integers and take the stream's handle without building a Stream.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda device: torch.cuda.current_stream(device).cuda_stream)


def _addr(t):
    """The address of a contiguous CUDA tensor (None: NULL)."""
    if t is None:
        return None
    if not t.is_cuda or not t.is_contiguous():
        raise ValueError("tensors must be contiguous CUDA tensors")
    return t.data_ptr()


def _workspace(nbytes: int, device):
    """A workspace, its address and size."""
    if not nbytes:
        return None, None, 0
    t = torch.empty(nbytes, dtype=torch.uint8, device=device)
    return t, t.data_ptr(), nbytes


def _on_stream(f):
    """With stream=s: runs f with s current, so that outputs and workspaces come from s's memory
    pool (freed there, they cannot be handed out while a kernel of s still uses them)."""
    @functools.wraps(f)
    def g(*args, stream=None, **kw):
        if stream is None:
            return f(*args, **kw)
        with torch.cuda.stream(stream):
            return f(*args, **kw)
    return g


# ---- group norm with an activation -----------------------------------------------------------
def make_gn_desc(B, C, P, G, act, layout, dtype, eps=1e-5) -> GnDesc:
    if isinstance(dtype, torch.dtype):
        dtype = _DT[dtype]
    return GnDesc(B, C, P, G, ACTS.get(act, act), LAYOUTS.get(layout, layout), dtype, eps)


def conv_gn_fwd_workspace_size(desc: GnDesc) -> int:
    return lib().conv_gn_fwd_workspace_size(_ref(desc))


def conv_gn_fwd(desc: GnDesc, x, gamma, beta, y, mean, rstd, workspace, stream=None) -> None:
    """gamma, beta, and (both together) mean, rstd may be None."""
    _check(lib().conv_gn_fwd(_ref(desc), _ptr(x), _ptr(gamma), _ptr(beta), _ptr(y), _ptr(mean), _ptr(rstd),
                             _ptr(workspace), _bytes(workspace), _stream(stream)), "conv_gn_fwd")


def conv_gn_bwd_workspace_size(desc: GnDesc) -> int:
    return lib().conv_gn_bwd_workspace_size(_ref(desc))


def conv_gn_bwd(desc: GnDesc, x, dy, gamma, beta, mean, rstd, dx, dgamma, dbeta, workspace, stream=None) -> None:
    """gamma, beta, and (both together) dgamma, dbeta may be None."""
    _check(lib().conv_gn_bwd(_ref(desc), _ptr(x), _ptr(dy), _ptr(gamma), _ptr(beta), _ptr(mean), _ptr(rstd), _ptr(dx),
                             _ptr(dgamma), _ptr(dbeta), _ptr(workspace), _bytes(workspace), _stream(stream)),
           "conv_gn_bwd")


def _same(name, t, shape, dtype, device):
    if t.shape != shape or t.dtype != dtype or t.device != device:
        raise ValueError(f"{name}: expected {tuple(shape)} {dtype} on {device}, got {tuple(t.shape)} {t.dtype} "
                         f"on {t.device}")


def _gn_desc_of(x, groups, gamma, beta, eps, act, layout) -> GnDesc:
    dt, a, lay = _DT.get(x.dtype), ACTS.get(act), LAYOUTS.get(layout)
    if dt is None:
        raise ValueError(f"x: float32 or bfloat16, got {x.dtype}")
    if a is None or lay is None:
        raise ValueError(f"act is one of {list(ACTS)} and layout of {list(LAYOUTS)}, got {act!r}, {layout!r}")
    shape = x.shape
    if len(shape) < 2:
        raise ValueError("x: at least (batch, channels)")
    C, P = shape[1 - 2 * lay], 1  # (B, C, ...) or (B, ..., C)
    for n in (shape[1:-1] if lay else shape[2:]):
        P *= n
    if gamma is not None:
        _same("gamma", gamma, (C,), x.dtype, x.device)
    if beta is not None:
        _same("beta", beta, (C,), x.dtype, x.device)
    return GnDesc(shape[0], C, P, groups, a, lay, dt, eps)


@_on_stream
def group_norm(x, groups: int, gamma=None, beta=None, eps: float = 1e-5, act: str = "none", layout: str = "nchw",
               stats: bool = True):
    """y, mean, rstd of x (B, C, ...) for "nchw" or (B, ..., C) for "nhwc", contiguous; mean and
    rstd (fp32, (B, groups)) are what the backward takes, None with stats=False."""
    desc = _gn_desc_of(x, groups, gamma, beta, eps, act, layout)
    px, device = _addr(x), x.device
    y = torch.empty_like(x)
    mean = rstd = None
    if stats:
        mean = torch.empty((desc.B, groups), dtype=torch.float32, device=device)
        rstd = torch.empty_like(mean)
    L = lib()
    ws, pw, nw = _workspace(L.conv_gn_fwd_workspace_size(_ref(desc)), device)
    _check(L.conv_gn_fwd(_ref(desc), px, _addr(gamma), _addr(beta), y.data_ptr(), _addr(mean), _addr(rstd), pw, nw,
                         _raw_stream(device.index)), "conv_gn_fwd")
    return y, mean, rstd


@_on_stream
def group_norm_bwd(x, dy, groups: int, gamma, beta, mean, rstd, act: str = "none", layout: str = "nchw",
                   param_grads: bool = True):
    """dx, dgamma, dbeta (None, None with param_grads=False) from group_norm's inputs and stats."""
    desc = _gn_desc_of(x, groups, gamma, beta, 0.0, act, layout)
    device, dtype = x.device, x.dtype
    _same("dy", dy, x.shape, dtype, device)
    stat = (desc.B, groups)
    _same("mean", mean, stat, torch.float32, device)
    _same("rstd", rstd, stat, torch.float32, device)
    px = _addr(x)
    dx = torch.empty_like(x)
    dgamma = dbeta = None
    if param_grads:
        dgamma = torch.empty((desc.C,), dtype=dtype, device=device)
        dbeta = torch.empty_like(dgamma)
    L = lib()
    ws, pw, nw = _workspace(L.conv_gn_bwd_workspace_size(_ref(desc)), device)
    _check(L.conv_gn_bwd(_ref(desc), px, _addr(dy), _addr(gamma), _addr(beta), _addr(mean), _addr(rstd),
                         dx.data_ptr(), _addr(dgamma), _addr(dbeta), pw, nw, _raw_stream(device.index)),
           "conv_gn_bwd")
    return dx, dgamma, dbeta


# ---- embedding -------------------------------------------------------------------------------
def make_embed_desc(T, V, D, index_dtype, dtype, scale=1.0, padding_idx=-1) -> EmbedDesc:
    return EmbedDesc(T, V, D, padding_idx, _IDX.get(index_dtype, index_dtype), _DT.get(dtype, dtype), scale)


def conv_embed_fwd(desc: EmbedDesc, idx, table, y, stream=None) -> None:
    _check(lib().conv_embed_fwd(_ref(desc), _ptr(idx), _ptr(table), _ptr(y), _stream(stream)), "conv_embed_fwd")


def conv_embed_bwd_workspace_size(desc: EmbedDesc) -> int:
    return lib().conv_embed_bwd_workspace_size(_ref(desc))


def conv_embed_bwd(desc: EmbedDesc, idx, dy, dtable, workspace, stream=None) -> None:
    _check(lib().conv_embed_bwd(_ref(desc), _ptr(idx), _ptr(dy), _ptr(dtable), _ptr(workspace), _bytes(workspace),
                                _stream(stream)), "conv_embed_bwd")


def _embed_desc_of(idx, t, V, D, scale, padding_idx, name) -> EmbedDesc:
    it, dt = _IDX.get(idx.dtype), _DT.get(t.dtype)
    if it is None or dt is None:
        raise ValueError(f"idx: int32 or int64, {name}: float32 or bfloat16; got {idx.dtype}, {t.dtype}")
    if idx.device != t.device:
        raise ValueError(f"idx on {idx.device}, {name} on {t.device}")
    return EmbedDesc(idx.numel(), V, D, padding_idx, it, dt, scale)


@_on_stream
def embed(idx, table, scale: float = 1.0, padding_idx: int = -1):
    """scale * table[idx], shape idx.shape + (D,); a token equal to padding_idx or outside the
    table gives zeros."""
    if table.dim() != 2:
        raise ValueError("table: (rows, values)")
    V, D = table.shape
    desc = _embed_desc_of(idx, table, V, D, scale, padding_idx, "table")
    pi, pt, device = _addr(idx), _addr(table), table.device
    y = torch.empty(idx.shape + (D,), dtype=table.dtype, device=device)
    _check(lib().conv_embed_fwd(_ref(desc), pi, pt, y.data_ptr(), _raw_stream(device.index)), "conv_embed_fwd")
    return y


@_on_stream
def embed_bwd(idx, dy, V: int, scale: float = 1.0, padding_idx: int = -1):
    """The table's gradient (V, D) from dy of shape idx.shape + (D,)."""
    D = dy.shape[-1]
    desc = _embed_desc_of(idx, dy, V, D, scale, padding_idx, "dy")
    _same("dy", dy, idx.shape + (D,), dy.dtype, idx.device)
    pi, pd, device = _addr(idx), _addr(dy), dy.device
    dtable = torch.empty((V, D), dtype=dy.dtype, device=device)
    L = lib()
    ws, pw, nw = _workspace(L.conv_embed_bwd_workspace_size(_ref(desc)), device)
    _check(L.conv_embed_bwd(_ref(desc), pi, pd, dtable.data_ptr(), pw, nw, _raw_stream(device.index)),
           "conv_embed_bwd")
    return dtable


# ---- gradient norm and clipping --------------------------------------------------------------
def make_grads(grads, out=None):
    """The C array of a list of gradients (and outputs, default: in place).  It holds addresses,
    not references: keep the tensors alive while it is in use."""
    n = len(grads)
    # column by column: a list of hundreds of tensors is most of the call's host time
    for t in grads if out is None else itertools.chain(grads, out):
        if not t.is_cuda or not t.is_contiguous():
            raise ValueError("tensors must be contiguous CUDA tensors")
    flat = array.array("q", bytes(32 * max(1, n)))
    numels = array.array("q", [t.numel() for t in grads])
    dtypes = [t.dtype for t in grads]
    addrs = array.array("q", [t.data_ptr() for t in grads])
    flat[0:4 * n:4] = flat[1:4 * n:4] = addrs
    flat[2:4 * n:4] = numels
    try:
        flat[3:4 * n:4] = array.array("q", [_DT[d] for d in dtypes])
    except KeyError as e:
        raise ValueError(f"gradients are float32 or bfloat16, got {e.args[0]}") from None
    if out is not None:
        if [t.numel() for t in out] != numels.tolist() or [t.dtype for t in out] != dtypes:
            raise ValueError("out: each tensor with its gradient's size and dtype")
        flat[1:4 * n:4] = array.array("q", [t.data_ptr() for t in out])
    return (Grad * max(1, n)).from_buffer(flat)


def conv_grad_norm_workspace_size(grads, count: int) -> int:
    return lib().conv_grad_norm_workspace_size(ctypes.addressof(grads), count)


def conv_grad_norm(grads, count: int, norm, workspace, stream=None) -> None:
    _check(lib().conv_grad_norm(ctypes.addressof(grads), count, _ptr(norm), _ptr(workspace), _bytes(workspace),
                                _stream(stream)), "conv_grad_norm")


def conv_grad_clip(grads, count: int, max_norm: float, norm, workspace, stream=None) -> None:
    _check(lib().conv_grad_clip(ctypes.addressof(grads), count, max_norm, _ptr(norm), _ptr(workspace),
                                _bytes(workspace), _stream(stream)), "conv_grad_clip")


def _grads_call(grads, out, max_norm):
    grads = list(grads)
    if not grads:
        raise ValueError("an empty list of gradients")
    if out is not None and len(out) != len(grads):
        raise ValueError(f"out: {len(out)} tensors for {len(grads)} gradients")
    n, device = len(grads), grads[0].device
    arr = make_grads(grads, out)
    norm = torch.empty((), dtype=torch.float32, device=device)
    L, at = lib(), ctypes.addressof(arr)
    ws, pw, nw = _workspace(L.conv_grad_norm_workspace_size(at, n), device)
    if max_norm is None:
        _check(L.conv_grad_norm(at, n, norm.data_ptr(), pw, nw, _raw_stream(device.index)), "conv_grad_norm")
    else:
        _check(L.conv_grad_clip(at, n, max_norm, norm.data_ptr(), pw, nw, _raw_stream(device.index)),
               "conv_grad_clip")
    return norm


@_on_stream
def grad_norm(grads):
    """The 2-norm over all gradients, a 0-dim fp32 tensor (nothing waits for it)."""
    return _grads_call(grads, None, None)


@_on_stream
def clip_grads(grads, max_norm: float, out=None):
    """Scales the gradients by min(1, max_norm / (norm + 1e-6)), in place or into the tensors of
    ``out``; returns the norm before."""
    return _grads_call(grads, out, max_norm)

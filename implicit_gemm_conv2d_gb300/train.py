"""Python side of include/conv_train.h: the operators a training step runs around the conv
layers -- group norm with an activation, embedding lookup and its gradient, the global gradient
norm and clipping.

The functions named like the C entry points (conv_gn_fwd, conv_embed_bwd, conv_grad_clip, ...)
take a descriptor and already-allocated CUDA tensors, like those of ``binding``.  group_norm,
group_norm_bwd, embed, embed_bwd, grad_norm and clip_grads check shapes and types and allocate
outputs and workspaces with torch first.  Everything is enqueued on the current torch stream (or
the stream given) and nothing waits for the GPU; tensors made on another stream have to be
ordered by the caller (``stream.wait_stream``), as for any torch operation.  What the allocating
functions allocate belongs to the stream they run on.  A call runs on the current device, and
tensors on another one are refused (``with torch.cuda.device(x.device):``)."""
from __future__ import annotations

import ctypes
import importlib.util
import os
import threading

import torch

from . import binding
from . import build as _build
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


_native_mod = None


def _native():
    """The native binding (csrc/native.cpp): checks, allocates and calls in C++."""
    global _native_mod
    if _native_mod is None:
        lib()
        path = _build.NATIVE
        if not os.path.exists(path):
            raise RuntimeError(f"native binding not built ({path} missing): run "
                               "`python -c 'import __graft_entry__ as g; g.build()'`")
        spec = importlib.util.spec_from_file_location("_igconv_native", path)
        mod = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(mod)
        mod.set_errors(binding.ConvError, torch.OutOfMemoryError)
        _native_mod = mod
    return _native_mod


def _code(table, value, name):
    code = table.get(value)
    if code is None:
        raise ValueError(f"{name}: one of {list(table)}, got {value!r}")
    return code


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


def group_norm(x, groups: int, gamma=None, beta=None, eps: float = 1e-5, act: str = "none", layout: str = "nchw",
               stats: bool = True, stream=None):
    """y, mean, rstd of x (B, C, ...) for "nchw" or (B, ..., C) for "nhwc", contiguous; mean and
    rstd (fp32, (B, groups)) are what the backward takes, None with stats=False."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return group_norm(x, groups, gamma, beta, eps, act, layout, stats)
    return _native().group_norm(x, groups, gamma, beta, eps, _code(ACTS, act, "act"),
                                _code(LAYOUTS, layout, "layout"), stats)


def group_norm_bwd(x, dy, groups: int, gamma, beta, mean, rstd, act: str = "none", layout: str = "nchw",
                   param_grads: bool = True, stream=None):
    """dx, dgamma, dbeta (None, None with param_grads=False) from group_norm's inputs and stats."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return group_norm_bwd(x, dy, groups, gamma, beta, mean, rstd, act, layout, param_grads)
    return _native().group_norm_bwd(x, dy, groups, gamma, beta, mean, rstd, _code(ACTS, act, "act"),
                                    _code(LAYOUTS, layout, "layout"), param_grads)


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


def embed(idx, table, scale: float = 1.0, padding_idx: int = -1, stream=None):
    """scale * table[idx], shape idx.shape + (D,); a token equal to padding_idx or outside the
    table gives zeros."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return embed(idx, table, scale, padding_idx)
    return _native().embed(idx, table, scale, padding_idx)


def embed_bwd(idx, dy, V: int, scale: float = 1.0, padding_idx: int = -1, stream=None):
    """The table's gradient (V, D) from dy of shape idx.shape + (D,)."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return embed_bwd(idx, dy, V, scale, padding_idx)
    return _native().embed_bwd(idx, dy, V, scale, padding_idx)


# ---- gradient norm and clipping --------------------------------------------------------------
def make_grads(grads, out=None):
    """The C array of a list of gradients (and outputs, default: in place).  It holds addresses,
    not references: keep the tensors alive while it is in use."""
    arr = (Grad * max(1, len(grads)))()
    for e, g, o in zip(arr, grads, grads if out is None else out):
        if g.dtype not in _DT or o.dtype != g.dtype or o.numel() != g.numel():
            raise ValueError(f"float32 or bfloat16, out with its gradient's size and dtype: got {g.dtype}")
        e.grad, e.out, e.n, e.dtype = _ptr(g), _ptr(o), g.numel(), _DT[g.dtype]
    return arr


def conv_grad_norm_workspace_size(grads, count: int) -> int:
    return lib().conv_grad_norm_workspace_size(ctypes.addressof(grads), count)


def conv_grad_norm(grads, count: int, norm, workspace, stream=None) -> None:
    _check(lib().conv_grad_norm(ctypes.addressof(grads), count, _ptr(norm), _ptr(workspace), _bytes(workspace),
                                _stream(stream)), "conv_grad_norm")


def conv_grad_clip(grads, count: int, max_norm: float, norm, workspace, stream=None) -> None:
    _check(lib().conv_grad_clip(ctypes.addressof(grads), count, max_norm, _ptr(norm), _ptr(workspace),
                                _bytes(workspace), _stream(stream)), "conv_grad_clip")


def grad_norm(grads, stream=None):
    """The 2-norm over all gradients (a list or tuple, not empty), a 0-dim fp32 tensor (nothing waits
    for it)."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return grad_norm(grads)
    return _native().grads(_list(grads), None, None)


def clip_grads(grads, max_norm: float, out=None, stream=None):
    """Scales the gradients by min(1, max_norm / (norm + 1e-6)), in place or into the tensors of
    ``out``; returns the norm before.  max_norm is finite (grad_norm gives the norm alone), and no
    output may overlap another entry: a tensor is in the list once."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return clip_grads(grads, max_norm, out)
    return _native().grads(_list(grads), None if out is None else _list(out), max_norm)


def _list(tensors):
    return tensors if type(tensors) in (list, tuple) else list(tensors)

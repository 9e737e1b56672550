"""Python side of include/conv_train.h: the operators a training step runs around the conv
layers -- group norm with an activation, embedding lookup and its gradient, layer norm of a
residual sum, the gated scan over time, the loss against a teacher's top logits, the global
gradient norm and clipping.

The functions named like the C entry points (conv_gn_fwd, conv_embed_bwd, conv_grad_clip, ...)
take a descriptor and already-allocated CUDA tensors, like those of ``binding``.  group_norm,
group_norm_bwd, embed, embed_bwd, layer_norm, layer_norm_bwd, gated_scan, gated_scan_bwd, distill,
distill_bwd, distill_grad, grad_norm and clip_grads check shapes and types and allocate outputs and
workspaces with torch first.  Everything is enqueued on the current torch stream (or
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
           "conv_ln_fwd", "conv_ln_bwd_workspace_size", "conv_ln_bwd",
           "conv_scan_fwd_workspace_size", "conv_scan_fwd", "conv_scan_bwd_workspace_size", "conv_scan_bwd",
           "conv_distill_fwd", "conv_distill_bwd", "conv_distill_grad",
           "conv_grad_norm_workspace_size", "conv_grad_norm", "conv_grad_clip"]


class GnDesc(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("B", "C", "P", "G", "act", "layout", "dtype")] + \
        [("eps", ctypes.c_float)]


class EmbedDesc(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int64)] + \
        [(n, ctypes.c_int32) for n in ("V", "D", "padding_idx", "index_dtype", "dtype")] + [("scale", ctypes.c_float)]


class LnDesc(ctypes.Structure):
    _fields_ = [("N", ctypes.c_int64)] + [(n, ctypes.c_int32) for n in ("D", "rms", "dtype")] + [("eps", ctypes.c_float)]


class Rows(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int64), ("step", ctypes.c_int64)]


class ScanDesc(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("B", "T", "D", "dtype")] + \
        [(n, Rows) for n in ("x", "gate", "h", "dh", "dx", "dgate")]


class DistillDesc(ctypes.Structure):
    _fields_ = [("N", ctypes.c_int64), ("ld", ctypes.c_int64)] + \
        [(n, ctypes.c_int32) for n in ("V", "K", "dtype", "index_dtype", "teacher_dtype")] + \
        [("temperature", ctypes.c_float)]


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
            L.conv_ln_fwd.argtypes = [vp] * 10
            L.conv_ln_bwd_workspace_size.argtypes = [vp]
            L.conv_ln_bwd_workspace_size.restype = sz
            L.conv_ln_bwd.argtypes = [vp] * 11 + [sz, vp]
            L.conv_scan_fwd_workspace_size.argtypes = [vp]
            L.conv_scan_fwd_workspace_size.restype = sz
            L.conv_scan_fwd.argtypes = [vp] * 9 + [sz, vp]
            L.conv_scan_bwd_workspace_size.argtypes = [vp]
            L.conv_scan_bwd_workspace_size.restype = sz
            L.conv_scan_bwd.argtypes = [vp] * 13 + [sz, vp]
            L.conv_distill_fwd.argtypes = [vp] * 8
            L.conv_distill_bwd.argtypes = [vp] * 7 + [ctypes.c_float, vp, vp]
            L.conv_distill_grad.argtypes = [vp] * 5 + [ctypes.c_float, vp, vp, vp]
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


# ---- layer norm of a residual sum ------------------------------------------------------------
def make_ln_desc(N, D, dtype, eps=1e-5, rms=False) -> LnDesc:
    return LnDesc(N, D, int(rms), _DT.get(dtype, dtype), eps)


def conv_ln_fwd(desc: LnDesc, x, residual, gamma, beta, y, total, mean, rstd, stream=None) -> None:
    """gamma, beta, (both together) residual, total, and (both together) mean, rstd may be None; with rms
    beta and mean are."""
    _check(lib().conv_ln_fwd(_ref(desc), _ptr(x), _ptr(residual), _ptr(gamma), _ptr(beta), _ptr(y), _ptr(total),
                             _ptr(mean), _ptr(rstd), _stream(stream)), "conv_ln_fwd")


def conv_ln_bwd_workspace_size(desc: LnDesc) -> int:
    return lib().conv_ln_bwd_workspace_size(_ref(desc))


def conv_ln_bwd(desc: LnDesc, x, dy, gamma, mean, rstd, dtotal, dx, dgamma, dbeta, workspace, stream=None) -> None:
    """gamma, dtotal, and (both together) dgamma, dbeta may be None; with rms mean and dbeta are."""
    _check(lib().conv_ln_bwd(_ref(desc), _ptr(x), _ptr(dy), _ptr(gamma), _ptr(mean), _ptr(rstd), _ptr(dtotal), _ptr(dx),
                             _ptr(dgamma), _ptr(dbeta), _ptr(workspace), _bytes(workspace), _stream(stream)),
           "conv_ln_bwd")


def layer_norm(x, gamma=None, beta=None, residual=None, eps: float = 1e-5, rms: bool = False, stats: bool = True,
               stream=None):
    """y, total, mean, rstd of the rows (..., D) of x + residual: total is the sum (None without a residual),
    y its norm times gamma plus beta.  rms: the form without a mean (then beta and mean are None).  mean
    and rstd (fp32) are what the backward takes, None with stats=False."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return layer_norm(x, gamma, beta, residual, eps, rms, stats)
    return _native().layer_norm(x, gamma, beta, residual, eps, rms, stats)


def layer_norm_bwd(x, dy, gamma, mean, rstd, dtotal=None, param_grads: bool = True, stream=None):
    """dx, dgamma, dbeta from the forward's total (x without a residual) and stats; dx is the gradient of x
    and of residual.  mean None: the form without a mean (dbeta is None).  dtotal: the gradient that
    reached total beside the norm.  param_grads False: dgamma and dbeta are None."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return layer_norm_bwd(x, dy, gamma, mean, rstd, dtotal, param_grads)
    return _native().layer_norm_bwd(x, dy, gamma, mean, rstd, dtotal, param_grads)


# ---- gated scan over time --------------------------------------------------------------------
def _row_distances(t) -> Rows:
    return Rows(t.stride(0) if t.shape[0] > 1 else 0, t.stride(1) if t.shape[1] > 1 else 0)


def _rows_ptr(t):
    """The address of a (batch, time, channels) tensor whose channels lie one behind the other."""
    if t is None:
        return None
    if t.dim() != 3 or (t.shape[2] > 1 and t.stride(2) != 1 and t.numel() > 0):
        raise ValueError("(batch, time, channels), a step's channels one behind the other")
    return _ptr(t[:1, :1]) if t.numel() else _ptr(torch.empty_strided((0,), (1,), dtype=t.dtype, device=t.device))


def make_scan_desc(x, gate, h, dh=None, dx=None, dgate=None) -> ScanDesc:
    """Sizes, type and distances of the call's arrays, each (batch, time, channels)."""
    d = ScanDesc(*x.shape, _DT[x.dtype])
    for name, t in (("x", x), ("gate", gate), ("h", h), ("dh", dh), ("dx", dx), ("dgate", dgate)):
        if t is not None:
            if t.shape != x.shape or t.dtype != x.dtype:
                raise ValueError(f"{name}: x's sizes and dtype")
            setattr(d, name, _row_distances(t))
    return d


def conv_scan_fwd_workspace_size(desc: ScanDesc) -> int:
    return lib().conv_scan_fwd_workspace_size(_ref(desc))


def conv_scan_fwd(desc: ScanDesc, x, gate, h0, reset, lengths, h, last, workspace, stream=None) -> None:
    """h0, reset, lengths and last may be None."""
    _check(lib().conv_scan_fwd(_ref(desc), _rows_ptr(x), _rows_ptr(gate), _ptr(h0), _ptr(reset), _ptr(lengths),
                               _rows_ptr(h), _ptr(last), _ptr(workspace), _bytes(workspace), _stream(stream)),
           "conv_scan_fwd")


def conv_scan_bwd_workspace_size(desc: ScanDesc) -> int:
    return lib().conv_scan_bwd_workspace_size(_ref(desc))


def conv_scan_bwd(desc: ScanDesc, x, gate, h, dh, h0, dlast, reset, lengths, dx, dgate, dh0, workspace,
                  stream=None) -> None:
    """h0, dlast, reset, lengths and dh0 may be None."""
    _check(lib().conv_scan_bwd(_ref(desc), _rows_ptr(x), _rows_ptr(gate), _rows_ptr(h), _rows_ptr(dh), _ptr(h0),
                               _ptr(dlast), _ptr(reset), _ptr(lengths), _rows_ptr(dx), _rows_ptr(dgate), _ptr(dh0),
                               _ptr(workspace), _bytes(workspace), _stream(stream)), "conv_scan_bwd")


def gated_scan(x, gate, h0=None, reset=None, lengths=None, out=None, last=None, stream=None):
    """h, last of h[t] = h[t-1] + sigmoid(gate[t]) * (x[t] - h[t-1]) over (batch, time, channels): every
    step's state, and the one behind each row's last step (fp32, (batch, channels)).

    x and gate may be views (halves of one projection, time first) as long as a step's channels lie
    one behind the other.  h0: the states that the rows begin with (fp32).  reset (batch, time), bool
    or uint8: steps where a new sequence begins with a state of 0.  lengths (batch), int32: the steps
    that each row has; h is 0 behind them.  out and last: tensors to write to, out apart from the inputs;
    last may be h0, so that a rollout keeps its states in one place."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return gated_scan(x, gate, h0, reset, lengths, out, last)
    return _native().gated_scan(x, gate, h0, reset, lengths, out, last)


def gated_scan_bwd(x, gate, h, dh, h0=None, dlast=None, reset=None, lengths=None, dx=None, dgate=None, stream=None):
    """dx, dgate, dh0 (None where h0 is) from gated_scan's inputs, its h, and the gradients of h and
    (dlast, fp32) of last.  dx and dgate: tensors to write to, such as the halves of one gradient, apart
    from the inputs and one another."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return gated_scan_bwd(x, gate, h, dh, h0, dlast, reset, lengths, dx, dgate)
    return _native().gated_scan_bwd(x, gate, h, dh, h0, dlast, reset, lengths, dx, dgate)


# ---- loss against a teacher's top logits -----------------------------------------------------
def _logits_ptr(t):
    """The address of (rows, logits) whose rows may be any distance apart."""
    if t.dim() != 2 or (t.shape[1] > 1 and t.stride(1) != 1):
        raise ValueError("(rows, logits), a row's logits one behind the other")
    return _ptr(t[:1])


def _same_layout(desc: DistillDesc, dz) -> None:
    """dz is laid out as the descriptor's logits: its rows are written at their distances, which for a contiguous dz
    beside a view of wider rows would end behind it."""
    if dz.dim() != 2 or tuple(dz.shape) != (desc.N, desc.V) or (desc.N > 1 and dz.stride(0) != desc.ld):
        raise ValueError("dz: z's sizes and distances")


def make_distill_desc(z, ids, teacher, temperature=1.0) -> DistillDesc:
    return DistillDesc(z.shape[0], z.stride(0) if z.shape[0] > 1 else z.shape[1], z.shape[1], ids.shape[1], _DT[z.dtype],
                       _IDX[ids.dtype], _DT[teacher.dtype], temperature)


def conv_distill_fwd(desc: DistillDesc, z, ids, teacher, loss, zmax, zlog, stream=None) -> None:
    _check(lib().conv_distill_fwd(_ref(desc), _logits_ptr(z), _ptr(ids), _ptr(teacher), _ptr(loss), _ptr(zmax), _ptr(zlog),
                                  _stream(stream)), "conv_distill_fwd")


def conv_distill_bwd(desc: DistillDesc, z, ids, teacher, zmax, zlog, weight, scale, dz, stream=None) -> None:
    """weight may be None; dz has z's sizes and distances (ValueError otherwise) and may be z."""
    _same_layout(desc, dz)
    _check(lib().conv_distill_bwd(_ref(desc), _logits_ptr(z), _ptr(ids), _ptr(teacher), _ptr(zmax), _ptr(zlog),
                                  _ptr(weight), scale, _logits_ptr(dz), _stream(stream)), "conv_distill_bwd")


def conv_distill_grad(desc: DistillDesc, z, ids, teacher, weight, scale, loss, dz, stream=None) -> None:
    """weight may be None; dz has z's sizes and distances (ValueError otherwise) and may be z."""
    _same_layout(desc, dz)
    _check(lib().conv_distill_grad(_ref(desc), _logits_ptr(z), _ptr(ids), _ptr(teacher), _ptr(weight), scale, _ptr(loss),
                                   _logits_ptr(dz), _stream(stream)), "conv_distill_grad")


def distill(z, ids, teacher, temperature: float = 1.0, stream=None):
    """loss, zmax, zlog of logits z (rows, V) against a teacher's logits (rows, K) at ids (rows, K): the
    Kullback-Leibler divergence of the teacher's distribution over the K entries from the softmax of z,
    both at the temperature, times its square.  Entries outside [0, V) or of -inf count for nothing; a
    row without others has loss 0.  One entry a row at temperature 1 is the cross entropy.  zmax and
    zlog are what distill_bwd takes.  z's rows may be any distance apart; every tensor begins at a multiple
    of 16 bytes, which a slice from some row or entry on may not (ConvError)."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return distill(z, ids, teacher, temperature)
    return _native().distill(z, ids, teacher, temperature)


def distill_bwd(z, ids, teacher, zmax, zlog, weight=None, scale: float = 1.0, temperature: float = 1.0, out=None,
                stream=None):
    """dz of sum over the rows of scale * weight * loss, with z's distances between the rows; out: a tensor
    with the same to write to, which may be z."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return distill_bwd(z, ids, teacher, zmax, zlog, weight, scale, temperature, out)
    return _native().distill_bwd(z, ids, teacher, zmax, zlog, weight, scale, temperature, out)


def distill_grad(z, ids, teacher, weight=None, scale: float = 1.0, temperature: float = 1.0, out=None, stream=None):
    """loss and dz (distill, then distill_bwd) in one call that reads z once, for weights known before the
    losses; the losses are without weight and scale."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return distill_grad(z, ids, teacher, weight, scale, temperature, out)
    return _native().distill_grad(z, ids, teacher, weight, scale, temperature, out)


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

"""The dense operators around the KDA op in a block's training step: layer norm,
the linear layer with bias, activation and residual in its epilogue, and the
clipping of the gradients' global norm.

Each has the package's two forms: direct calls (``layer_norm_fwd`` /
``layer_norm_bwd``, ``linear_fwd`` / ``linear_bwd``, ``clip_grad_norm``), and
``layer_norm`` / ``linear`` with autograd.  PyTorch provides device memory and
the current stream; every step of the computation runs in libkda's CUDA kernels
(include/kda.h), which neither allocate nor synchronise, so the calls can be
captured into CUDA graphs.  Tensors are contiguous, bf16 or fp32.
"""
from __future__ import annotations

import ctypes
from array import array
from math import inf
from operator import attrgetter
from typing import Optional, Sequence

import torch
from torch.autograd.function import once_differentiable

from . import _lib
from .ops import _check_tensor, _current_device, _refuse_device

__all__ = ["layer_norm", "layer_norm_fwd", "layer_norm_bwd", "linear", "linear_fwd", "linear_bwd", "linear_status",
           "clip_grad_norm"]

_DTYPE = {torch.float32: _lib.KDA_F32, torch.bfloat16: _lib.KDA_BF16}
_dtype_of = attrgetter("dtype")
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_SIZE_MAX = ctypes.c_size_t(-1).value
_ACT = {None: 0, "silu": 1, "gelu": 2, "sigmoid": 3}


def _p(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _stream(device):
    # a tenth of a small call's time: the raw handle (a torch.cuda.Stream object costs 2 us), few lookups
    index = device.index
    if _current_device() != index:
        _refuse_device(device)
    return _raw_stream(index)


def _scratch(nbytes: int, device):
    """A 256-byte aligned workspace: (tensor that owns it, address, bytes)."""
    ws = torch.empty(nbytes + 256, dtype=torch.uint8, device=device)
    at = (ws.data_ptr() + 255) & ~255
    return ws, at, nbytes


def _workspace(need: int, device):
    """_scratch, or none where none is needed.  SIZE_MAX marks a problem that the library refuses: the call itself
    then raises its message."""
    return _scratch(need, device) if 0 < need < _SIZE_MAX else (None, None, 0)


def _check_input(name, t):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a tensor")
    if not t.is_cuda:
        raise ValueError("KDA kernels run on CUDA tensors only")
    if t.dtype not in _DTYPE:
        raise TypeError(f"{name} must be bfloat16 or float32")
    if t.dim() < 1:
        raise ValueError(f"{name} must have at least one dimension")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


# ---- layer norm ---------------------------------------------------------------

def _norm_struct(x, weight, bias, eps):
    _check_input("x", x)
    width = x.shape[-1]
    if width < 1:
        raise ValueError("x has an empty last axis")
    params = [t for t in (weight, bias) if t is not None]
    pt = params[0].dtype if params else x.dtype
    if pt not in (x.dtype, torch.float32):
        raise TypeError(f"weight and bias must be float32 or {x.dtype}, not {pt}")
    for name, t in (("weight", weight), ("bias", bias)):
        if t is not None:
            _check_tensor(name, t, pt, x.device, (width,))
    return _lib.KdaNorm(x.numel() // width, width, _DTYPE[x.dtype], _DTYPE[pt], eps, x.data_ptr(), _p(weight), _p(bias))


def layer_norm_fwd(x, weight=None, bias=None, eps: float = 1e-5):
    """Layer norm over the last axis (no autograd).  weight and bias [D] are fp32
    or x's type; None: ones / zeros.  Returns (y, mean, rstd) with mean and rstd
    fp32, one a row: what the backward reads."""
    lib = _lib.load()
    s = _norm_struct(x, weight, bias, eps)
    y = torch.empty_like(x)
    mean = torch.empty(x.shape[:-1], dtype=torch.float32, device=x.device)
    rstd = torch.empty_like(mean)
    _lib.check(lib, lib.kda_layer_norm_fwd(s, y.data_ptr(), mean.data_ptr(), rstd.data_ptr(), _stream(x.device)))
    return y, mean, rstd


def layer_norm_bwd(dy, x, mean, rstd, weight=None, bias=None, need_dx: bool = True, need_dweight: bool = True):
    """Backward of :func:`layer_norm_fwd`.  Returns (dx, dweight, dbias): dx and
    dweight are None where they are not needed, dweight and dbias where their
    parameter is None."""
    lib = _lib.load()
    s = _norm_struct(x, weight, bias, 0.0)
    _check_tensor("dy", dy, x.dtype, x.device, tuple(x.shape))
    for name, t in (("mean", mean), ("rstd", rstd)):
        _check_tensor(name, t, torch.float32, x.device, tuple(x.shape[:-1]))
    dx = torch.empty_like(x) if need_dx else None
    dw = torch.empty_like(weight) if need_dweight and weight is not None else None
    db = None if bias is None else torch.empty_like(bias)
    if dx is None and dw is None and db is None:
        return None, None, None
    ws, wp, wb = None, None, 0
    if dw is not None or db is not None:
        ws, wp, wb = _scratch(lib.kda_layer_norm_bwd_workspace_size(s), x.device)
    _lib.check(lib, lib.kda_layer_norm_bwd(s, dy.data_ptr(), mean.data_ptr(), rstd.data_ptr(), _p(dx), _p(dw), _p(db),
                                           wp, wb, _stream(x.device)))
    return dx, dw, db


class LayerNormFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, eps):
        y, mean, rstd = layer_norm_fwd(x, weight, bias, eps)
        ctx.save_for_backward(x, mean, rstd, weight, bias)
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        x, mean, rstd, weight, bias = ctx.saved_tensors
        need = ctx.needs_input_grad
        dx, dw, db = layer_norm_bwd(dy.contiguous(), x, mean, rstd, weight, bias if need[2] else None,
                                    need_dx=need[0], need_dweight=need[1])
        return dx, dw, db, None


def layer_norm(x, weight=None, bias=None, eps: float = 1e-5):
    """Layer norm over the last axis, with autograd; see :func:`layer_norm_fwd`."""
    return LayerNormFunction.apply(x, weight, bias, eps)


# ---- linear ---------------------------------------------------------------------

def _linear_struct(x, weight, bias, residual, activation):
    _check_input("x", x)
    if not isinstance(weight, torch.Tensor) or weight.dim() != 2:
        raise ValueError("weight must be [outs, ins]")
    outs, ins = weight.shape
    if outs < 1 or ins < 1:
        raise ValueError("weight has an empty axis")
    _check_tensor("weight", weight, x.dtype, x.device, (outs, x.shape[-1]))
    if bias is not None:
        _check_tensor("bias", bias, x.dtype, x.device, (outs,))
    if residual is not None:
        _check_tensor("residual", residual, x.dtype, x.device, tuple(x.shape[:-1]) + (outs,))
    if activation not in _ACT:
        raise ValueError(f"activation must be one of {sorted(k for k in _ACT if k)} or None, not {activation!r}")
    return _lib.KdaLinear(x.numel() // ins, outs, ins, _DTYPE[x.dtype], _ACT[activation], x.data_ptr(),
                          weight.data_ptr(), _p(bias), _p(residual))


def linear_fwd(x, weight, bias=None, activation: Optional[str] = None, residual=None, keep_preact: bool = False):
    """y = act(x weight^T + bias) + residual (no autograd): x [..., ins], weight
    [outs, ins], bias [outs], residual and y [..., outs], all of one type;
    activation None, "silu", "gelu" or "sigmoid".  Returns (y, preact): with
    keep_preact and an activation, preact is the value before the activation
    that :func:`linear_bwd` reads, else None."""
    lib = _lib.load()
    s = _linear_struct(x, weight, bias, residual, activation)
    y = torch.empty(x.shape[:-1] + (s.outs,), dtype=x.dtype, device=x.device)
    z = torch.empty_like(y) if keep_preact and activation is not None else None
    ws, wp, wb = _workspace(lib.kda_linear_fwd_workspace_size(s), x.device)
    _lib.check(lib, lib.kda_linear_fwd(s, y.data_ptr(), _p(z), wp, wb, _stream(x.device)))
    return y, z


def linear_bwd(dy, x, weight, bias=None, activation: Optional[str] = None, preact=None, need_dx: bool = True,
               need_dweight: bool = True):
    """Backward of :func:`linear_fwd`.  Returns (dx, dweight, dbias): dx and
    dweight are None where they are not needed, dbias where bias is None.  The
    residual's gradient is dy itself."""
    lib = _lib.load()
    s = _linear_struct(x, weight, bias, None, activation)
    shape = tuple(x.shape[:-1]) + (s.outs,)
    _check_tensor("dy", dy, x.dtype, x.device, shape)
    if activation is not None:
        _check_tensor("preact", preact, x.dtype, x.device, shape)
    else:
        preact = None
    dx = torch.empty_like(x) if need_dx else None
    dw = torch.empty_like(weight) if need_dweight else None
    db = None if bias is None else torch.empty_like(bias)
    if dx is None and dw is None and db is None:
        return None, None, None
    ws, wp, wb = _workspace(lib.kda_linear_bwd_workspace_size(s), x.device)
    _lib.check(lib, lib.kda_linear_bwd(s, dy.data_ptr(), _p(preact), _p(dx), _p(dw), _p(db), wp, wb,
                                       _stream(x.device)))
    return dx, dw, db


class LinearFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, activation, residual, grad_mode):
        # needs_input_grad is set under no_grad too, and grad mode is always off in here: apply's caller reads it
        y, z = linear_fwd(x, weight, bias, activation, residual,
                          keep_preact=grad_mode and any(ctx.needs_input_grad[:3]))
        ctx.save_for_backward(x, weight, bias, z)
        ctx.activation = activation
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        x, weight, bias, z = ctx.saved_tensors
        need = ctx.needs_input_grad
        d = dy.contiguous()
        dx = dw = db = None
        if any(need[:3]):
            dx, dw, db = linear_bwd(d, x, weight, bias if need[2] else None, ctx.activation, z, need_dx=need[0],
                                    need_dweight=need[1])
        return dx, dw, db, None, dy if need[4] else None, None


def linear(x, weight, bias=None, activation: Optional[str] = None, residual=None):
    """y = act(x weight^T + bias) + residual, with autograd; see :func:`linear_fwd`."""
    return LinearFunction.apply(x, weight, bias, activation, residual, torch.is_grad_enabled())


class _DeviceWord:
    def __init__(self, address: int):
        self.__cuda_array_interface__ = {"shape": (), "typestr": "<i4", "data": (address, False), "version": 2}


def linear_status(device="cuda"):
    """A 0-d int32 tensor on the device: nonzero if a bounded device wait of a linear call
    gave up by this point of the current stream (the results of such a call are invalid).
    The word is never cleared.  Nothing is synchronised: reading the tensor is the caller's
    moment to wait, once a step or once a run."""
    device = torch.device(device)
    if device.index is not None and device.index != _current_device():
        _refuse_device(device)
    lib = _lib.load()
    word = ctypes.c_void_p()
    _lib.check(lib, lib.kda_linear_status(ctypes.byref(word)))
    return torch.as_tensor(_DeviceWord(word.value), device=device).clone()


# ---- gradient clipping ------------------------------------------------------------

def _refuse_list(name, ts, device):
    for i, t in enumerate(ts):
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name}[{i}] must be a tensor")
        if t.dtype not in _DTYPE:
            raise TypeError(f"{name}[{i}] must be bfloat16 or float32")
        if t.device != device:
            raise ValueError(f"{name}[{i}] is on {t.device}, expected {device}")
        if not t.is_contiguous():
            raise ValueError(f"{name}[{i}] must be contiguous")


def _check_list(name, ts, device):
    """(types, sizes, addresses) of the tensors of a list, after their checks.
    Hundreds of tensors are ordinary: the checks run over the whole list, and only
    a list that fails one is gone through for the tensor at fault."""
    T = torch.Tensor
    tensors = all(issubclass(kind, T) for kind in set(map(type, ts)))
    kinds = list(map(_DTYPE.get, map(_dtype_of, ts))) if tensors else [None]
    if None in kinds or set(map(T.get_device, ts)) != {device.index} or not all(map(T.is_contiguous, ts)):
        _refuse_list(name, ts, device)
    return array("i", kinds), array("q", map(T.numel, ts)), array("Q", map(T.data_ptr, ts))


def clip_grad_norm(tensors: Sequence[torch.Tensor], max_norm: float, out: Optional[Sequence[torch.Tensor]] = None):
    """Scales the tensors (bf16 and fp32, mixed) so that their global L2 norm is
    at most max_norm: out[i] = tensors[i] * min(1, max_norm / (norm + 1e-6)), in
    place without ``out``; autograd counts it as a modification of what is written.
    Returns the norm before clipping, a 0-d fp32 tensor on the device (nothing is
    synchronised).  max_norm = inf computes the norm and scales nothing.  What is
    written must not overlap (a tensor may be read twice, but is written once)."""
    tensors = list(tensors)
    if not tensors:
        raise ValueError("clip_grad_norm needs at least one tensor")
    lib = _lib.load()
    if not isinstance(tensors[0], torch.Tensor):
        raise TypeError("tensors[0] must be a tensor")
    device = tensors[0].device
    if device.type != "cuda":
        raise ValueError("KDA kernels run on CUDA tensors only")
    kinds, sizes, src = _check_list("tensors", tensors, device)
    dst = src
    if out is not None:
        out = list(out)
        if len(out) != len(tensors):
            raise ValueError(f"out has {len(out)} tensors, expected {len(tensors)}")
        out_kinds, out_sizes, dst = _check_list("out", out, device)
        if out_kinds != kinds or out_sizes != sizes:
            raise ValueError("out must have the tensors' types and sizes")
    norm = torch.empty((), dtype=torch.float32, device=device)
    ws, wp, wb = _scratch(lib.kda_clip_grad_norm_workspace_size(len(tensors)), device)
    _lib.check(lib, lib.kda_clip_grad_norm(len(tensors), src.buffer_info()[0], dst.buffer_info()[0],
                                           sizes.buffer_info()[0], kinds.buffer_info()[0], max_norm, norm.data_ptr(),
                                           wp, wb, _stream(device)))
    if out is not None or max_norm != inf:
        torch.autograd.graph.increment_version(tensors if out is None else out)
    return norm

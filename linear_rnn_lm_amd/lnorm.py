"""Layer norm (C ABI in ``include/lnorm.h``): the norm in front of a time mix and,
with ``groups`` = heads, the per-head norm of its output.

    y, mean, rstd = ln_fwd(x, weight, bias, groups=H)
    dx, dweight, dbias = ln_bwd(dy, x, weight, mean, rstd, groups=H)
    y = LN.apply(x, weight, bias, groups, eps, out_dtype)     # autograd op

Each of ``groups`` equal parts of a row's C channels is normalised by itself:
y = (x - mean) / sqrt(var + eps) * weight + bias.  x: (..., C) fp32 or bf16; y has
x's type, or bf16 for an fp32 x with ``out_dtype=torch.bfloat16`` (the
recurrence's fp32 output into a bf16 layer).  weight, bias: (C,) fp32 or bf16, or
None.  mean, rstd: (rows, groups) fp32.  dx has x's type, dweight and dbias are fp32.
Tensors are dense and, where the parts are a multiple of 8 channels, lie at multiples of
16 bytes; LN makes copies of those that do not.  Calls of several streams or threads
may overlap as long as they share no output and no workspace, and calls can be captured
into a graph (as with every autograd op, a backward only on leaves that no live eager
graph uses).
"""
from __future__ import annotations

import ctypes
import functools

from . import BF16, F32, _check_bytes, _dense, _dense_on, _fits, _launch, _LazyOpOf, _ptr, _where, lib


@functools.lru_cache(maxsize=None)
def _lib():
    L = lib()
    vp, i, i64, sz, f = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t, ctypes.c_float
    L.ln_fwd.argtypes, L.ln_fwd.restype = [i64] + [i] * 5 + [vp] * 3 + [f] + [vp] * 4, i
    L.ln_bwd.argtypes, L.ln_bwd.restype = [i64] + [i] * 5 + [vp] * 8 + [vp, sz, vp], i
    L.ln_bwd_workspace_bytes.argtypes, L.ln_bwd_workspace_bytes.restype = [i64, i, i], sz
    return L


@functools.lru_cache(maxsize=None)
def _types():
    """The two types and their codes (None: no tensor, any code)."""
    import torch
    return {torch.float32: F32, torch.bfloat16: BF16, None: F32}


@functools.lru_cache(maxsize=1024)
def _workspace_bytes(rows, C, groups):
    return _lib().ln_bwd_workspace_bytes(rows, C, groups)


def _check_x(fn, x, weight, bias, groups):
    """(rows, C) of x, with the type codes of x and of the weights."""
    types, dev, shape = _types(), x.device, x.shape
    C, n = shape[-1] if shape else 0, x.numel()
    if n < 1:
        raise ValueError(f"{fn}: x must be (..., C) and not empty, got {tuple(shape)}")
    if x.dtype not in types:
        raise TypeError(f"{fn}: x must be float32 or bfloat16, got {x.dtype}")
    if groups < 1 or C % groups or C // groups > 16384:
        raise ValueError(f"{fn}: groups must divide C into parts of at most 16384, got C = {C}, groups = {groups}")
    if not x.is_contiguous():
        _dense_on(fn, "x", x, dev)
    wd = None
    for name, w in (("weight", weight), ("bias", bias)):
        if w is not None:
            if w.dtype not in types or (wd is not None and w.dtype != wd) or w.shape != (C,):
                raise ValueError(f"{fn}: {name} is {_where(w)}, expected ({C},) float32 or bfloat16, both of one type")
            if w.device != dev or not w.is_contiguous():
                _dense_on(fn, name, w, dev)
            wd = w.dtype
    return n // C, C, types[x.dtype], types[wd]


def _check_like(fn, name, t, shape, dtype, dev):
    if _fits(t, shape, dtype, dev):
        return
    if tuple(t.shape) != tuple(shape) or t.dtype != dtype:
        raise ValueError(f"{fn}: {name} is {_where(t)}, expected {tuple(shape)} {dtype}")
    _dense_on(fn, name, t, dev)


def _out_dtype(fn, x, out_dtype):
    import torch
    out_dtype = out_dtype or x.dtype
    if out_dtype != x.dtype and not (x.dtype == torch.float32 and out_dtype == torch.bfloat16):
        raise TypeError(f"{fn}: {x.dtype} rows cannot give {out_dtype}")
    return out_dtype


def ln_fwd(x, weight=None, bias=None, *, groups=1, eps=1e-5, out_dtype=None, want_stats=True, y=None, mean=None,
           rstd=None):
    """Forward.  Returns (y, mean, rstd); the statistics are None if not wanted."""
    import torch
    fn = "ln_fwd"
    rows, C, xcode, wcode = _check_x(fn, x, weight, bias, groups)
    dev, ycode = x.device, xcode
    if y is None and (out_dtype is None or out_dtype == x.dtype):
        y = torch.empty_like(x)
    else:
        out_dtype = _out_dtype(fn, x, out_dtype if y is None else y.dtype)
        ycode = _types()[out_dtype]
        if y is None:
            y = torch.empty_like(x, dtype=out_dtype)
        _check_like(fn, "y", y, x.shape, out_dtype, dev)
    if (mean is None) != (rstd is None):
        raise ValueError(f"{fn}: mean and rstd go together")
    if mean is None and want_stats:
        mean, rstd = x.new_empty((2, rows, groups), dtype=torch.float32).unbind(0)
    elif mean is not None:
        _check_like(fn, "mean", mean, (rows, groups), torch.float32, dev)
        _check_like(fn, "rstd", rstd, (rows, groups), torch.float32, dev)
    _launch(fn, _lib().ln_fwd, dev, rows, C, groups, xcode, ycode, wcode, x.data_ptr(), _ptr(weight), _ptr(bias), eps,
            y.data_ptr(), _ptr(mean), _ptr(rstd))
    return y, mean, rstd


def ln_bwd(dy, x, weight, mean, rstd, *, groups=1, want_dx=True, want_dw=True, workspace=None, out=None):
    """Backward of ``ln_fwd``: (dx, dweight, dbias); entries not wanted are None.
    ``out`` may hold the three (None for one not wanted)."""
    import torch
    fn = "ln_bwd"
    rows, C, xcode, wcode = _check_x(fn, x, weight, None, groups)
    dev, ydt = x.device, dy.dtype
    if ydt != x.dtype:
        _out_dtype(fn, x, ydt)
    _check_like(fn, "dy", dy, x.shape, ydt, dev)
    _check_like(fn, "mean", mean, (rows, groups), torch.float32, dev)
    _check_like(fn, "rstd", rstd, (rows, groups), torch.float32, dev)
    if out is None:
        dx = torch.empty_like(x) if want_dx else None
        dw, db = x.new_empty((2, C), dtype=torch.float32).unbind(0) if want_dw else (None, None)
    else:
        if len(out) != 3:
            raise ValueError(f"{fn}: out must hold 3 entries, got {len(out)}")
        dx, dw, db = out
        for n, t, shape, dt in (("dx", dx, x.shape, x.dtype), ("dweight", dw, (C,), torch.float32),
                                ("dbias", db, (C,), torch.float32)):
            if t is not None:
                _check_like(fn, n, t, shape, dt, dev)
    if (dw is None) != (db is None) or (dx is None and dw is None):
        raise ValueError(f"{fn}: dx, or dweight and dbias together, must be wanted")
    need = 0 if dw is None else _workspace_bytes(rows, C, groups)
    if workspace is not None:
        _check_bytes(fn, "workspace", workspace, need, dev)
    elif need:
        workspace = x.new_empty(need, dtype=torch.uint8)
    _launch(fn, _lib().ln_bwd, dev, rows, C, groups, xcode, _types()[ydt], wcode, dy.data_ptr(), x.data_ptr(), _ptr(weight),
            mean.data_ptr(), rstd.data_ptr(), _ptr(dx), _ptr(dw), _ptr(db), _ptr(workspace), need)
    return dx, dw, db


def _make_autograd():
    import torch
    from torch.autograd.function import once_differentiable

    class LN(torch.autograd.Function):
        """Differentiable op: (x, weight, bias, groups, eps, out_dtype) -> y, gradients by
        ln_bwd in the inputs' types."""

        @staticmethod
        def forward(ctx, x, weight=None, bias=None, groups=1, eps=1e-5, out_dtype=None):
            # other widths go value by value, at any address of theirs
            align = 1 if x.dim() and x.shape[-1] % 8 else 16
            x = _dense(x, align)
            weight, bias = (None if t is None else _dense(t, align) for t in (weight, bias))
            y, mean, rstd = ln_fwd(x, weight, bias, groups=groups, eps=eps, out_dtype=out_dtype)
            ctx.save_for_backward(x, weight, mean, rstd)
            ctx.groups, ctx.out, ctx.align, ctx.tb = groups, y.dtype, align, None if bias is None else bias.dtype
            return y

        @staticmethod
        @once_differentiable                               # a gradient of the gradient is an error, not a zero
        def backward(ctx, dy):
            x, weight, mean, rstd = ctx.saved_tensors
            nx, nw, nb = (*ctx.needs_input_grad, False, False)[:3]     # only what was passed is listed
            if not (nx or nw or nb):
                return (None,) * 6
            dx, dw, db = ln_bwd(_dense(dy.to(ctx.out), ctx.align), x, weight, mean, rstd, groups=ctx.groups, want_dx=nx,
                                want_dw=nw or nb)
            return dx, dw.to(weight.dtype) if nw else None, db.to(ctx.tb) if nb else None, None, None, None

    return LN


LN = _LazyOpOf(_make_autograd)

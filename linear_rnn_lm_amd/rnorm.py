"""The fused end of a block (C ABI in ``include/rnorm.h``): the norm of a time mix's output,
its gate, the scaled residual and the next block's norm.

    r, h, stats = rn_fwd(o, gate, res, weight=w, scale=s, weight2=w2, groups=H, norm="layer", norm2="rms")
    do, dgate, dres, dweight, dbias, dscale, dweight2, dbias2 = rn_bwd(dr, dh, o, gate, res, stats, weight=w, ...)
    r, h = RN.apply(o, gate, res, weight, bias, scale, weight2, bias2, options)     # autograd op

r = res + scale act(gate) (norm1(o) weight + bias), h = norm2(r) weight2 + bias2.  ``norm`` (over
each of ``groups`` equal parts of a row) is "layer" or "rms", ``norm2`` (over the row) also None:
then h is None.  ``act`` is "silu" or "sigmoid"; without a gate it does not matter.  Every
tensor but o may be None: no gate, no residual (r has the layer's type then), weights of 1,
biases of 0, a scale of 1.

o, gate, res, r, h: (..., C), C at most 8192; with groups > 1 a part has 64, 128, 256 or 512
channels.  The layer's type (gate, h) is o's, or bf16 for an fp32 o with
``out_dtype=torch.bfloat16``; res and r have that type or fp32.  The weights are (C,), all fp32 or
all bf16; their gradients are fp32.  ``stats`` (rows, 2 groups + 2) is what ``rn_bwd`` needs.

Tensors are dense (gate may be a slice of wider rows) and, where C is a multiple of 8, lie at
multiples of 16 bytes; RN makes copies of those that do not.  Calls of several streams or
threads may overlap as long as they share no output and no workspace, and calls can be captured
into a graph (as with every autograd op, a backward only on leaves that no live eager graph uses).
"""
from __future__ import annotations

import ctypes
import functools

from . import F32, _check_bytes, _dense, _launch, _LazyOpOfEither, _new_like, _ptr, _types, _where, lib
from .ssm import _check_tensor

_NORMS = {None: 0, "layer": 1, "rms": 2}
_ACTS = {"silu": 1, "sigmoid": 2}


@functools.lru_cache(maxsize=None)
def _lib():
    L = lib()
    vp, i, i64, sz, f = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t, ctypes.c_float
    L.rn_fwd.argtypes, L.rn_fwd.restype = [i64] + [i] * 9 + [f] * 2 + [vp] * 2 + [i64] + [vp] * 10, i
    L.rn_bwd.argtypes, L.rn_bwd.restype = [i64] + [i] * 9 + [vp] * 4 + [i64] + [vp] * 10 + [vp, sz, vp], i
    L.rn_bwd_workspace_bytes.argtypes, L.rn_bwd_workspace_bytes.restype = [i64, i, i], sz
    return L


@functools.lru_cache(maxsize=1024)
def _workspace_bytes(rows, C, groups):
    return _lib().rn_bwd_workspace_bytes(rows, C, groups)


def _gate_ld(fn, gate, shape, dtype, dev):
    """Distance between gate's rows: dense, or the first C values of wider dense rows."""
    if tuple(gate.shape) != tuple(shape) or gate.dtype != dtype or gate.device != dev:
        raise ValueError(f"{fn}: gate is {_where(gate)}, expected {tuple(shape)} {dtype} on {dev}")
    if gate.is_contiguous():
        return shape[-1]
    ld = _uniform_ld(gate)
    if ld is None:
        raise ValueError(f"{fn}: gate's rows must have one distance and their values lie side by side "
                         f"(got strides {gate.stride()})")
    return ld


def _uniform_ld(t):
    """The one distance between the rows of (..., C), or None."""
    C = t.shape[-1]
    if C > 1 and t.stride(-1) != 1:
        return None
    ld, rows = None, 1
    for size, stride in zip(reversed(t.shape[:-1]), reversed(t.stride()[:-1])):
        if size == 1:
            continue
        if ld is None:
            ld = stride
        elif stride != rows * ld:
            return None
        rows *= size
    return C if ld is None else ld if ld >= C else None


def _setup(fn, o, gate, res, ws, groups, norm, norm2, act, layer, r_dtype):
    """(rows, C), the leading arguments of a call, and gate's row distance."""
    codes, _ = _types()
    shape, dev = o.shape, o.device
    C, n = shape[-1] if shape else 0, o.numel()
    if n < 1:
        raise ValueError(f"{fn}: o must be (..., C) and not empty, got {tuple(shape)}")
    if o.dtype not in codes or layer not in codes:
        raise TypeError(f"{fn}: o and the layer's type must be float32 or bfloat16, got {o.dtype} and {layer}")
    import torch
    if o.dtype != layer and o.dtype != torch.float32:
        raise TypeError(f"{fn}: {o.dtype} rows cannot give {layer}")
    if C > 8192 or groups < 1 or C % groups or (groups > 1 and C // groups not in (64, 128, 256, 512)):
        raise ValueError(f"{fn}: C must be at most 8192 and parts of 64, 128, 256, 512 channels or a whole row, got "
                         f"C = {C}, groups = {groups}")
    if norm not in ("layer", "rms") or norm2 not in _NORMS:
        raise ValueError(f"{fn}: norm must be 'layer' or 'rms' and norm2 one of them or None, got {norm!r} and {norm2!r}")
    if gate is not None and act not in _ACTS:
        raise ValueError(f"{fn}: act must be 'silu' or 'sigmoid', got {act!r}")
    _check_tensor(fn, "o", o, shape, o.dtype, dev)
    if r_dtype not in (layer, torch.float32) or (res is None and r_dtype != layer):
        raise TypeError(f"{fn}: res must be {layer} or float32, got {r_dtype}")
    _check_tensor(fn, "res", res, shape, r_dtype, dev)
    wd = None
    for name, w in ws:
        if w is not None:
            if w.dtype not in codes or (wd is not None and w.dtype != wd):
                raise ValueError(f"{fn}: {name} is {_where(w)}, expected ({C},) float32 or bfloat16, all of one type")
            wd = w.dtype
            _check_tensor(fn, name, w, (C,), wd, dev)
    ld = C if gate is None else _gate_ld(fn, gate, shape, layer, dev)
    kinds = (groups, _NORMS[norm], _NORMS[norm2], 0 if gate is None else _ACTS[act], codes[o.dtype], codes[layer],
             codes[r_dtype], F32 if wd is None else codes[wd])
    return n // C, C, kinds, ld


def rn_fwd(o, gate=None, res=None, *, weight=None, bias=None, scale=None, weight2=None, bias2=None, groups=1, norm="layer",
           norm2=None, act="silu", eps=1e-5, eps2=1e-5, out_dtype=None, want_stats=True, r=None, h=None, stats=None):
    """Forward.  Returns (r, h, stats): h is None without norm2, stats if not wanted."""
    import torch
    fn = "rn_fwd"
    layer = out_dtype or (o.dtype if gate is None else gate.dtype)
    r_dtype = layer if res is None else res.dtype
    rows, C, kinds, ld = _setup(fn, o, gate, res, (("weight", weight), ("bias", bias), ("scale", scale),
                                                   ("weight2", weight2), ("bias2", bias2)), groups, norm, norm2, act,
                                layer, r_dtype)
    dev, shape = o.device, o.shape
    if norm2 is None and (weight2 is not None or bias2 is not None or h is not None):
        raise ValueError(f"{fn}: weight2, bias2 and h need norm2")
    if r is None:
        r = _new_like(o if res is None else res, r_dtype)
    else:
        _check_tensor(fn, "r", r, shape, r_dtype, dev)
    if h is not None:
        _check_tensor(fn, "h", h, shape, layer, dev)
    elif norm2 is not None:
        h = _new_like(o if gate is None else gate, layer)
    if stats is not None:
        _check_tensor(fn, "stats", stats, (rows, 2 * groups + 2), torch.float32, dev)
    elif want_stats:
        stats = torch.empty((rows, 2 * groups + 2), dtype=torch.float32, device=dev)
    _launch(fn, _lib().rn_fwd, dev, rows, C, *kinds, eps, eps2, o.data_ptr(), _ptr(gate), ld,
            *map(_ptr, (res, weight, bias, scale, weight2, bias2, r, h, stats)))
    return r, h, stats


def rn_bwd(dr, dh, o, gate, res, stats, *, weight=None, bias=None, scale=None, weight2=None, bias2=None, groups=1,
           norm="layer", norm2=None, act="silu", want_do=True, want_dres=True, want_dw=True, workspace=None):
    """Backward of ``rn_fwd``: (do, dgate, dres, dweight, dbias, dscale, dweight2, dbias2), None
    where the input is None or the gradient not wanted.  dr or dh may be None, for zero."""
    import torch
    fn = "rn_bwd"
    if dr is None and dh is None:
        raise ValueError(f"{fn}: dr or dh is required")
    ws = (("weight", weight), ("bias", bias), ("scale", scale), ("weight2", weight2), ("bias2", bias2))
    layer = gate.dtype if gate is not None else dh.dtype if dh is not None else dr.dtype if res is None else None
    if layer is None:                                      # only r is known: a residual in fp32 leaves the layer's type open
        layer = o.dtype if res.dtype == torch.float32 else res.dtype
    r_dtype = layer if res is None else res.dtype
    rows, C, kinds, ld = _setup(fn, o, gate, res, ws, groups, norm, norm2, act, layer, r_dtype)
    dev, shape = o.device, o.shape
    if dh is not None and norm2 is None:
        raise ValueError(f"{fn}: dh needs norm2")
    _check_tensor(fn, "dr", dr, shape, r_dtype, dev)
    _check_tensor(fn, "dh", dh, shape, layer, dev)
    _check_tensor(fn, "stats", stats, (rows, 2 * groups + 2), torch.float32, dev)
    do = torch.empty_like(o) if want_do else None
    dgate = None if gate is None else _new_like(gate, layer)
    dres = torch.empty_like(res) if res is not None and want_dres else None
    want_dw = want_dw and any(w is not None for _, w in ws)
    dw, need = None, 0
    if want_dw:
        dw, need = torch.empty((5, C), dtype=torch.float32, device=dev), _workspace_bytes(rows, C, groups)
        if workspace is None:
            workspace = torch.empty(need, dtype=torch.uint8, device=dev)
        else:
            _check_bytes(fn, "workspace", workspace, need, dev)
    if do is None and dgate is None and dres is None and dw is None:
        raise ValueError(f"{fn}: no gradient is wanted")
    _launch(fn, _lib().rn_bwd, dev, rows, C, *kinds, _ptr(dr), _ptr(dh), o.data_ptr(), _ptr(gate), ld,
            *map(_ptr, (res, stats, weight, bias, scale, weight2, do, dgate, dres, dw)), _ptr(workspace) if want_dw else None,
            need)
    return (do, dgate, dres, *(None if w is None or dw is None else dw[i] for i, (_, w) in enumerate(ws)))


def _make_autograd():
    import torch
    from torch.autograd.function import once_differentiable

    class RN(torch.autograd.Function):
        """Differentiable op: (o, gate, res, weight, bias, scale, weight2, bias2, options) -> (r, h), h None
        without norm2; ``options`` is a dict of rn_fwd's groups, norm, norm2, act, eps, eps2 and
        out_dtype.  Gradients by rn_bwd in the inputs' types."""

        @staticmethod
        def forward(ctx, o, gate=None, res=None, weight=None, bias=None, scale=None, weight2=None, bias2=None, options=None):
            ctx.set_materialize_grads(False)               # a gradient that is not there costs nothing
            opt = dict(options or {})
            align = 1 if o.dim() and o.shape[-1] % 8 else 16
            fit = lambda t: None if t is None else _dense(t, align)  # noqa: E731
            o, res, weight, bias, scale, weight2, bias2 = map(fit, (o, res, weight, bias, scale, weight2, bias2))
            if gate is not None:
                ld = _uniform_ld(gate)
                if ld is None or (align == 16 and (ld * gate.element_size() % 16 or gate.data_ptr() % 16)):
                    gate = fit(gate)
            r, h, stats = rn_fwd(o, gate, res, weight=weight, bias=bias, scale=scale, weight2=weight2, bias2=bias2,
                                 want_stats=any(ctx.needs_input_grad), **opt)
            ctx.save_for_backward(o, gate, res, weight, bias, scale, weight2, bias2, stats)
            ctx.opt = {k: opt[k] for k in ("groups", "norm", "norm2", "act") if k in opt}
            ctx.align, ctx.r, ctx.h = align, r.dtype, None if h is None else h.dtype
            return r, h

        @staticmethod
        @once_differentiable                               # a gradient of the gradient is an error, not a zero
        def backward(ctx, dr, dh=None):
            o, gate, res, *ws, stats = ctx.saved_tensors
            if dr is None and dh is None:
                return (None,) * 9
            dr = None if dr is None else _dense(dr.to(ctx.r), ctx.align)
            dh = None if dh is None else _dense(dh.to(ctx.h), ctx.align)
            names = ("weight", "bias", "scale", "weight2", "bias2")
            needs = (*ctx.needs_input_grad, *(False,) * 9)[:9]
            do, dgate, dres, *dws = rn_bwd(dr, dh, o, gate, res, stats, **dict(zip(names, ws)), **ctx.opt,
                                           want_do=needs[0], want_dres=needs[2], want_dw=any(needs[3:8]))
            dws = [None if g is None else g.to(w.dtype) for g, w in zip(dws, ws)]
            return do, dgate, dres, *dws, None

    return RN


RN = _LazyOpOfEither(_make_autograd)

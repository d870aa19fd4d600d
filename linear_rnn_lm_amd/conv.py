"""The short causal convolution (C ABI in ``include/conv.h``), one filter per channel:
what stands in front of a time mix.

    y, hT = conv_fwd(x, weight, bias, h0, cu_seqlens=cu)
    dx, dweight, dbias, dh0 = conv_bwd(dy, x, weight, bias, h0, dhT, cu_seqlens=cu)
    y = conv_step(x, weight, bias, state, slots=slots)            # state updated in place
    y, hT = CONV.apply(x, weight, bias, h0, cu, silu)             # autograd op

y_t = act(bias + sum_j weight[:, j] x_(t - W + 1 + j)), act SiLU, or none with
``silu=False``.  x: (B, T, C) fp32 or bf16, weight: (C, W), W 2, 3 or 4, bias: (C,) or None, both
fp32 or bf16.  A sequence's state, (N, W - 1, C) of x's type, is its last W - 1 inputs, oldest
first; None stands for zeros.  y, dx and the states' gradients have x's type, dweight and
dbias are fp32.

Packed sequences (``cu_seqlens``), pools of states (``slots``), streams and graphs are as for
the selective scan (ssm.py).  x may be a slice of wider rows; everything else is dense.
CONV makes copies of what is neither.
"""
from __future__ import annotations

import ctypes
import functools

from . import (_check_bytes, _dense, _launch, _LazyOpOf, _new_like, _ptr, _row_ld, _rows, _types, _where,
               lib)
from .gdr import _check_cu
from .ssm import _check_tensor


@functools.lru_cache(maxsize=None)
def _lib():
    L = lib()
    vp, i, i64, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t
    dims = [i] * 6
    L.conv_fwd.argtypes = dims + [vp, i64, vp, vp, i, vp, i, i] + [vp] * 4
    L.conv_bwd_workspace_bytes.argtypes, L.conv_bwd_workspace_bytes.restype = [i] * 6, sz
    L.conv_bwd.argtypes = dims + [vp] * 3 + [i64, vp, vp, i, vp, i, i] + [vp] * 6 + [sz, vp]
    L.conv_step.argtypes = dims + [vp, i64, vp, vp, i, vp, i] + [vp] * 4
    for n in ("conv_fwd", "conv_bwd", "conv_step"):
        getattr(L, n).restype = i
    return L


@functools.lru_cache(maxsize=1024)
def _workspace_bytes(B, T, C, W, N):
    return _lib().conv_bwd_workspace_bytes(B, T, C, W, N, int(N > 0))


def _inputs(fn, x, weight, bias):
    """(B, T, C, W, x's code, the weights' code) and the distance between x's rows."""
    if x.dim() != 3 or weight.dim() != 2:
        raise ValueError(f"{fn}: x must be (B, T, C) and weight (C, W), got {tuple(x.shape)} and {tuple(weight.shape)}")
    (B, T, C), W = x.shape, weight.shape[1]
    if B < 1 or T < 1 or C < 1 or W not in (2, 3, 4):
        raise ValueError(f"{fn}: B, T and C must be at least 1 and W 2, 3 or 4, got x {tuple(x.shape)}, "
                         f"weight {tuple(weight.shape)}")
    codes, _ = _types()
    if x.dtype not in codes or weight.dtype not in codes:
        raise TypeError(f"{fn}: x and weight must be float32 or bfloat16, got {x.dtype} and {weight.dtype}")
    ld = _row_ld(fn, "x", x, (B, T, C), x.dtype, x.device)
    _check_tensor(fn, "weight", weight, (C, W), weight.dtype, x.device)
    _check_tensor(fn, "bias", bias, (C,), weight.dtype, x.device)
    return (B, T, C, W, codes[x.dtype], codes[weight.dtype]), ld


def conv_fwd(x, weight, bias=None, h0=None, *, silu=True, cu_seqlens=None, want_hT=True, y=None, hT=None):
    """Forward.  Returns (y, hT), hT None if not wanted."""
    import torch
    fn = "conv_fwd"
    dims, ld = _inputs(fn, x, weight, bias)
    B, T, C, W = dims[:4]
    dev = x.device
    N = _check_cu(fn, cu_seqlens, B, dev)
    states = (N or B, W - 1, C)
    _check_tensor(fn, "h0", h0, states, x.dtype, dev)
    fresh = int(y is None)                                 # of a new y the rows outside packed sequences are zeroed
    if fresh:
        y = _new_like(x, x.dtype)
    else:
        _check_tensor(fn, "y", y, (B, T, C), x.dtype, dev)
    if hT is not None:
        _check_tensor(fn, "hT", hT, states, x.dtype, dev)
    elif want_hT:
        hT = torch.empty(states, dtype=x.dtype, device=dev) if h0 is None else torch.empty_like(h0)
    _launch(fn, _lib().conv_fwd, dev, *dims, x.data_ptr(), ld, weight.data_ptr(), _ptr(bias), int(bool(silu)),
            _ptr(cu_seqlens), N, fresh, _ptr(h0), y.data_ptr(), _ptr(hT))
    return y, hT


def conv_bwd(dy, x, weight, bias=None, h0=None, dhT=None, *, silu=True, cu_seqlens=None, want_dh0=True, workspace=None,
             out=None):
    """Backward.  Returns (dx, dweight, dbias, dh0): dbias is None without a bias, dh0 if not
    wanted; ``out`` may hold the first three."""
    import torch
    fn = "conv_bwd"
    dims, ld = _inputs(fn, x, weight, bias)
    B, T, C, W = dims[:4]
    dev = x.device
    N = _check_cu(fn, cu_seqlens, B, dev)
    states = (N or B, W - 1, C)
    _check_tensor(fn, "dy", dy, (B, T, C), x.dtype, dev)
    _check_tensor(fn, "h0", h0, states, x.dtype, dev)
    _check_tensor(fn, "dhT", dhT, states, x.dtype, dev)
    fresh = int(out is None)
    if fresh:
        dx = _new_like(x, x.dtype)
        dw = _new_like(weight, torch.float32)
        db = None if bias is None else _new_like(bias, torch.float32)
    else:
        if len(out) != 3:
            raise ValueError(f"{fn}: out must hold 3 entries, got {len(out)}")
        dx, dw, db = out
        if dx is None or dw is None or (db is None) != (bias is None):
            raise ValueError(f"{fn}: out must hold dx, dweight and, with a bias, dbias")
        for n, t, shape, dt in (("dx", dx, (B, T, C), x.dtype), ("dweight", dw, (C, W), torch.float32),
                                ("dbias", db, (C,), torch.float32)):
            _check_tensor(fn, n, t, shape, dt, dev)
    dh0 = torch.empty(states, dtype=x.dtype, device=dev) if want_dh0 else None
    need = _workspace_bytes(B, T, C, W, N)
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    else:
        _check_bytes(fn, "workspace", workspace, need, dev)
    _launch(fn, _lib().conv_bwd, dev, *dims, dy.data_ptr(), _ptr(dhT), x.data_ptr(), ld, weight.data_ptr(), _ptr(bias),
            int(bool(silu)), _ptr(cu_seqlens), N, fresh, _ptr(h0), dx.data_ptr(), dw.data_ptr(), _ptr(db), _ptr(dh0),
            workspace.data_ptr(), workspace.numel() * workspace.element_size())
    return dx, dw, db, dh0


def conv_step(x, weight, bias, state, *, silu=True, slots=None, state_out=None, y=None):
    """B rows of T new tokens; returns y.  ``state`` (P, W - 1, C) is updated in place, or into
    ``state_out``; ``slots`` as in ``ssm_step``."""
    import torch
    fn = "conv_step"
    dims, ld = _inputs(fn, x, weight, bias)
    B, T, C, W = dims[:4]
    dev, P = x.device, state.shape[0] if state.dim() == 3 else 0
    if P < 1:
        raise ValueError(f"{fn}: state must be (P, W - 1, C), got {_where(state)}")
    if slots is None:
        if P < B:
            raise ValueError(f"{fn}: state holds {P} states for {B} rows")
    else:
        _check_tensor(fn, "slots", slots, (B,), torch.int32, dev)
    _check_tensor(fn, "state", state, (P, W - 1, C), x.dtype, dev)
    if state_out is None:
        state_out = state
    else:
        _check_tensor(fn, "state_out", state_out, (P, W - 1, C), x.dtype, dev)
    if y is None:
        y = _new_like(x, x.dtype)
    else:
        _check_tensor(fn, "y", y, (B, T, C), x.dtype, dev)
    _launch(fn, _lib().conv_step, dev, *dims, x.data_ptr(), ld, weight.data_ptr(), _ptr(bias), int(bool(silu)),
            _ptr(slots), P, state.data_ptr(), state_out.data_ptr(), y.data_ptr())
    return y


def _make_autograd():
    import torch
    from torch.autograd.function import once_differentiable

    class CONV(torch.autograd.Function):
        """Differentiable op: (x, weight, bias, h0, cu_seqlens, silu) -> (y, hT), gradients by
        conv_bwd in the inputs' types.  weight and bias may be of two types; h0 has x's."""

        @staticmethod
        def forward(ctx, x, weight, bias=None, h0=None, cu_seqlens=None, silu=True):
            ctx.set_materialize_grads(False)               # a gradient that is not there costs nothing
            x, tw, tb = _rows(x), weight.dtype, None if bias is None else bias.dtype
            wide = tw if tb is None else torch.promote_types(tw, tb)       # of two types the one that holds both
            weight = weight.to(wide).contiguous()
            bias = None if bias is None else bias.to(wide).contiguous()
            h0 = None if h0 is None else h0.contiguous()
            y, hT = conv_fwd(x, weight, bias, h0, silu=silu, cu_seqlens=cu_seqlens)
            ctx.save_for_backward(x, weight, bias, h0, cu_seqlens)
            ctx.silu, ctx.tw, ctx.tb, ctx.has_h0 = silu, tw, tb, h0 is not None
            return y, hT

        @staticmethod
        @once_differentiable                               # a gradient of the gradient is an error, not a zero
        def backward(ctx, dy, dhT):
            x, weight, bias, h0, cu = ctx.saved_tensors
            dy = torch.zeros(x.shape, dtype=x.dtype, device=x.device) if dy is None else _dense(dy.to(x.dtype))
            dhT = None if dhT is None else _dense(dhT.to(x.dtype))
            dx, dw, db, dh0 = conv_bwd(dy, x, weight, bias, h0, dhT, silu=ctx.silu, cu_seqlens=cu,
                                       want_dh0=ctx.has_h0)
            return dx, dw.to(ctx.tw), None if ctx.tb is None else db.to(ctx.tb), dh0, None, None

    return CONV


CONV = _LazyOpOf(_make_autograd)

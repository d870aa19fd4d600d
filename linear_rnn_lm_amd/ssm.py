"""The selective state space scan (C ABI in ``include/ssm.h``): a linear-RNN time mix
whose decay differs per channel, state and token.

    y, ckpt, hT = ssm_fwd(x, dt, A, b, c, D, z, h0, dt_bias=bias, cu_seqlens=cu)
    dx, ddt, dA, db, dc, dD, dz, ddt_bias, dh0 = ssm_bwd(dy, x, dt, A, b, c, ckpt, D, z, dhT, dt_bias=bias, cu_seqlens=cu)
    y = ssm_step(x, dt, A, b, c, state, D, z, dt_bias=bias, slots=slots)     # state updated in place
    y, hT = SSM.apply(x, dt, A, b, c, D, z, bias, h0, cu, softplus)          # autograd op

Every channel carries S fp32 states h; per token delta = softplus(dt + dt_bias),
h = exp(delta A) h + delta x b, y = (sum_s c h + D x) z sigmoid(z).  x, dt, z:
(B, T, C); b, c: (B, T, G, S), each group shared by C / G channels (a multiple of 64 where
G > 1); S 16, 32 or 64; all of one type, fp32 or bf16.  A: (C, S), D, dt_bias: (C,), states
(N, C, S), all fp32.  D, z, dt_bias and h0 may be None; ``softplus=False`` takes dt + dt_bias as
it is.  y and the token gradients have the inputs' type, the other gradients are fp32.

``cu_seqlens`` (int32, N + 1 offsets on the GPU, B = 1) packs N sequences of any
lengths, empty ones included, along T.  The offsets stay on the GPU: nothing waits for
them, and a call can be captured into a graph and replayed with other offsets.  (As with
every autograd op, capture a backward only on leaves that no live eager graph uses.)

x, dt, b, c and z may be slices of wider rows (one distance between all rows, for ssm_fwd and
ssm_bwd at most 2 ** 24 values, the values of a row side by side); everything else is dense.
SSM makes copies of what is neither.
Calls of several streams or threads may overlap as long as they share no output and no
workspace.
"""
from __future__ import annotations

import ctypes
import functools

from . import (_check_bytes, _dense, _dense_on, _launch, _LazyOpOfEither, _new_like, _ptr, _row_ld, _rows, _types, _where,
               lib)
from .gdr import _check_cu

SSM_BLOCK = 16
_MAX_LD = 1 << 24


@functools.lru_cache(maxsize=None)
def _lib():
    L = lib()
    vp, i, i64, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t
    dims, row = [i] * 5, [vp, i64]
    ins = row * 2 + [vp] + row * 2 + [vp] + row + [vp, i]
    L.ssm_slots.argtypes, L.ssm_slots.restype = [i] * 4, i64
    for n in ("ssm_ckpt_bytes", "ssm_fwd_workspace_bytes", "ssm_bwd_workspace_bytes"):
        getattr(L, n).argtypes, getattr(L, n).restype = dims + [i] * 2, sz
    L.ssm_fwd.argtypes = dims + [i] + ins + [vp, i, i] + [vp] * 4 + [vp, sz, vp]
    L.ssm_bwd.argtypes = dims + [i] + [vp] * 2 + ins + [vp, i, i] + [vp] * 10 + [vp, sz, vp]
    L.ssm_step.argtypes = dims + [i] + ins + [vp, i] + [vp] * 4
    for n in ("ssm_fwd", "ssm_bwd", "ssm_step"):
        getattr(L, n).restype = i
    return L


@functools.lru_cache(maxsize=1024)
def _sizes(dims, N):
    """Bytes of the checkpoints and of the two workspaces."""
    L, packed = _lib(), int(N > 0)
    return (L.ssm_ckpt_bytes(*dims, N, packed), L.ssm_fwd_workspace_bytes(*dims, N, packed),
            L.ssm_bwd_workspace_bytes(*dims, N, packed))


def _check_tensor(fn, name, t, shape, dtype, dev):
    if t is None or (t.shape == shape and t.dtype is dtype and t.device == dev and t.is_contiguous()):
        return
    if tuple(t.shape) != tuple(shape) or t.dtype != dtype:
        raise ValueError(f"{fn}: {name} is {_where(t)}, expected {tuple(shape)} {dtype}")
    _dense_on(fn, name, t, dev)


def _inputs(fn, x, dt, A, b, c, D, z, dt_bias, softplus):
    """(B, T, C, S, G) of the inputs, their type's code, and their part of a call's arguments."""
    if x.dim() != 3 or b.dim() != 4:
        raise ValueError(f"{fn}: x must be (B, T, C) and b (B, T, G, S), got {tuple(x.shape)} and {tuple(b.shape)}")
    (B, T, C), (_, _, G, S) = x.shape, b.shape
    if B < 1 or T < 1 or C < 1 or G < 1 or S not in (16, 32, 64):
        raise ValueError(f"{fn}: B, T, C and G must be at least 1 and S 16, 32 or 64, got x {tuple(x.shape)}, "
                         f"b {tuple(b.shape)}")
    if C % G or (G > 1 and C // G % 64):
        raise ValueError(f"{fn}: G must divide C into groups of a multiple of 64 channels, got C = {C}, G = {G}")
    codes, f32 = _types()
    if x.dtype not in codes:
        raise TypeError(f"{fn}: x must be float32 or bfloat16, got {x.dtype}")
    row, mat, dtype, dev = x.shape, b.shape, x.dtype, x.device
    if mat[0] != B or mat[1] != T:
        raise ValueError(f"{fn}: b is {_where(b)}, expected {(B, T, G, S)} {dtype}")
    args = (x.data_ptr(), _row_ld(fn, "x", x, row, dtype, dev), dt.data_ptr(), _row_ld(fn, "dt", dt, row, dtype, dev),
            A.data_ptr(), b.data_ptr(), _row_ld(fn, "b", b, mat, dtype, dev), c.data_ptr(),
            _row_ld(fn, "c", c, mat, dtype, dev), None if D is None else D.data_ptr(), None if z is None else z.data_ptr(),
            _row_ld(fn, "z", z, row, dtype, dev), None if dt_bias is None else dt_bias.data_ptr(), 1 if softplus else 0)
    _check_tensor(fn, "A", A, (C, S), f32, dev)
    _check_tensor(fn, "D", D, (C,), f32, dev)
    _check_tensor(fn, "dt_bias", dt_bias, (C,), f32, dev)
    return (B, T, C, S, G), codes[dtype], args


def _workspace(fn, workspace, need, dev):
    import torch
    if workspace is None:
        return torch.empty(need, dtype=torch.uint8, device=dev), need
    _check_bytes(fn, "workspace", workspace, need, dev)
    return workspace, workspace.numel() * workspace.element_size()


def ssm_fwd(x, dt, A, b, c, D=None, z=None, h0=None, *, dt_bias=None, softplus=True, cu_seqlens=None, want_y=True,
            want_ckpt=True, want_hT=True, y=None, ckpt=None, hT=None, workspace=None):
    """Forward.  Returns (y, ckpt, hT); entries not wanted are None.  Pre-allocated
    outputs may be passed; hT may be h0 (in-place update).  ``ckpt`` (slots, C, S), the
    states entering every 16th token, is what ``ssm_bwd`` needs: not wanted for inference."""
    import torch
    fn = "ssm_fwd"
    dims, code, args = _inputs(fn, x, dt, A, b, c, D, z, dt_bias, softplus)
    B, T, C, S, _ = dims
    dev, f32 = x.device, torch.float32
    N = _check_cu(fn, cu_seqlens, B, dev)
    nck, nws, _ = _sizes(dims, N)
    states = (N or B, C, S)
    _check_tensor(fn, "h0", h0, states, f32, dev)
    fresh = 0                                              # of a new y the rows outside packed sequences are zeroed
    if y is not None:
        _check_tensor(fn, "y", y, (B, T, C), x.dtype, dev)
    elif want_y:
        y, fresh = _new_like(x, x.dtype), 1
    if ckpt is not None:
        _check_tensor(fn, "ckpt", ckpt, (nck // (4 * C * S), C, S), f32, dev)
    elif want_ckpt:
        ckpt = torch.empty((nck // (4 * C * S), C, S), dtype=f32, device=dev)
    if hT is not None:
        _check_tensor(fn, "hT", hT, states, f32, dev)
    elif want_hT:
        hT = torch.empty(states, dtype=f32, device=dev) if h0 is None else torch.empty_like(h0)
    workspace, wsb = _workspace(fn, workspace, nws, dev)
    _launch(fn, _lib().ssm_fwd, dev, *dims, code, *args, _ptr(cu_seqlens), N, fresh, _ptr(h0), _ptr(y), _ptr(ckpt),
            _ptr(hT), workspace.data_ptr(), wsb)
    return y, ckpt, hT


def ssm_bwd(dy, x, dt, A, b, c, ckpt, D=None, z=None, dhT=None, *, dt_bias=None, softplus=True, cu_seqlens=None,
            want_dh0=True, workspace=None, out=None):
    """Backward.  Returns (dx, ddt, dA, db, dc, dD, dz, ddt_bias, dh0), None where the input
    is None (dh0: where not wanted); ``out`` may hold the first eight."""
    import torch
    fn = "ssm_bwd"
    dims, code, args = _inputs(fn, x, dt, A, b, c, D, z, dt_bias, softplus)
    B, T, C, S, G = dims
    dev, f32, states = x.device, torch.float32, None
    N = _check_cu(fn, cu_seqlens, B, dev)
    nck, _, nws = _sizes(dims, N)
    states = (N or B, C, S)
    _check_tensor(fn, "dy", dy, (B, T, C), x.dtype, dev)
    _check_tensor(fn, "ckpt", ckpt, (nck // (4 * C * S), C, S), f32, dev)
    _check_tensor(fn, "dhT", dhT, states, f32, dev)
    want = (("dx", (B, T, C), x.dtype, x), ("ddt", (B, T, C), x.dtype, dt), ("dA", (C, S), f32, A),
            ("db", (B, T, G, S), x.dtype, b), ("dc", (B, T, G, S), x.dtype, c), ("dD", (C,), f32, D),
            ("dz", (B, T, C), x.dtype, z), ("ddt_bias", (C,), f32, dt_bias))
    fresh = int(out is None)                               # of new gradients the rows outside packed sequences are zeroed
    if out is None:
        out = [None if t is None else _new_like(t, t.dtype) for *_, t in want]
    elif len(out) != 8:
        raise ValueError(f"{fn}: out must hold 8 entries, got {len(out)}")
    else:
        for (n, shape, dtype, t), o in zip(want, out):
            if (o is None) != (t is None):
                raise ValueError(f"{fn}: {n} must be given where its input is, and only there")
            _check_tensor(fn, n, o, shape, dtype, dev)
    dh0 = torch.empty(states, dtype=f32, device=dev) if want_dh0 else None
    workspace, wsb = _workspace(fn, workspace, nws, dev)
    _launch(fn, _lib().ssm_bwd, dev, *dims, code, dy.data_ptr(), _ptr(dhT), *args, _ptr(cu_seqlens), N, fresh,
            ckpt.data_ptr(), *map(_ptr, out), _ptr(dh0), workspace.data_ptr(), wsb)
    return (*out, dh0)


def ssm_step(x, dt, A, b, c, state, D=None, z=None, *, dt_bias=None, softplus=True, slots=None, state_out=None, y=None):
    """B rows of T new tokens, token by token; returns y.

    ``state`` (P, C, S) fp32 is updated in place, or into ``state_out`` (a tensor of the
    same shape, of which only the states worked on are written).  ``slots`` (B,) int32
    picks each row's state (row r uses state r without it); a row whose slot is outside
    0 .. P - 1 is padding: its y is 0 and its inputs are not read.  Rows with the same slot
    are consecutive tokens of one sequence, in row order."""
    import torch
    fn = "ssm_step"
    dims, code, args = _inputs(fn, x, dt, A, b, c, D, z, dt_bias, softplus)
    B, T, C, S, _ = dims
    dev, P = x.device, state.shape[0] if state.dim() == 3 else 0
    if P < 1:
        raise ValueError(f"{fn}: state must be (P, C, S), got {tuple(state.shape)}")
    if slots is None:
        if P < B:
            raise ValueError(f"{fn}: state holds {P} states for {B} rows")
    else:
        _check_tensor(fn, "slots", slots, (B,), torch.int32, dev)
    _check_tensor(fn, "state", state, (P, C, S), torch.float32, dev)
    if state_out is None:
        state_out = state
    else:
        _check_tensor(fn, "state_out", state_out, (P, C, S), torch.float32, dev)
    if y is None:
        y = _new_like(x, x.dtype)
    else:
        _check_tensor(fn, "y", y, (B, T, C), x.dtype, dev)
    _launch(fn, _lib().ssm_step, dev, *dims, code, *args, _ptr(slots), P, state.data_ptr(), state_out.data_ptr(),
            y.data_ptr())
    return y


def _make_autograd():
    import torch
    from torch.autograd.function import once_differentiable

    class SSM(torch.autograd.Function):
        """Differentiable op: (x, dt, A, b, c, D, z, dt_bias, h0, cu_seqlens, softplus) -> (y, hT),
        gradients by ssm_bwd in the inputs' types.  Rows that no packed sequence covers have
        y = 0 and zero gradients.  Where gradients are off it leaves no checkpoints."""

        @staticmethod
        def forward(ctx, x, dt, A, b, c, D=None, z=None, dt_bias=None, h0=None, cu_seqlens=None, softplus=True):
            ctx.set_materialize_grads(False)               # a gradient that is not there costs nothing
            toks = [None if t is None else _rows(t, _MAX_LD) for t in (x, dt, b, c, z)]
            A_, D_, bias, h0_ = (None if t is None else _dense(t.float()) for t in (A, D, dt_bias, h0))
            need = any(ctx.needs_input_grad)
            X, DT, Bm, Cm, Z = toks
            y, ckpt, hT = ssm_fwd(X, DT, A_, Bm, Cm, D_, Z, h0_, dt_bias=bias, softplus=softplus, cu_seqlens=cu_seqlens,
                                  want_ckpt=need)
            ctx.save_for_backward(X, DT, A_, Bm, Cm, D_, Z, bias, ckpt, cu_seqlens)
            ctx.softplus = softplus
            ctx.types = [None if t is None else t.dtype for t in (A, D, dt_bias, h0)]
            return y, hT

        @staticmethod
        @once_differentiable                               # a gradient of the gradient is an error, not a zero
        def backward(ctx, dy, dhT):
            x, dt, A, b, c, D, z, bias, ckpt, cu = ctx.saved_tensors
            dy = torch.zeros(x.shape, dtype=x.dtype, device=x.device) if dy is None else dy.to(x.dtype).contiguous()
            dhT = None if dhT is None else _dense(dhT.float())
            tA, tD, tb, th = ctx.types
            dx, ddt, dA, db, dc, dD, dz, dbias, dh0 = ssm_bwd(
                dy, x, dt, A, b, c, ckpt, D, z, dhT, dt_bias=bias, softplus=ctx.softplus, cu_seqlens=cu,
                want_dh0=th is not None)
            cast = lambda g, t: None if t is None else g.to(t)  # noqa: E731
            return dx, ddt, cast(dA, tA), db, dc, cast(dD, tD), dz, cast(dbias, tb), cast(dh0, th), None, None

    return SSM


SSM = _LazyOpOfEither(_make_autograd)

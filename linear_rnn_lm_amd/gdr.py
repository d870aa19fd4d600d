"""The gated delta rule (C ABI in ``include/gdr.h``): a linear-RNN time mix with
one decay per head and token.

    o, ckpt, hT = gdr_fwd(q, k, v, g, beta, h0, cu_seqlens=cu)
    dq, dk, dv, dg, dbeta, dh0 = gdr_bwd(do, q, k, v, g, beta, ckpt, dhT, cu_seqlens=cu)
    o = gdr_step(q, k, v, g, beta, state, slots=slots)     # state updated in place
    o, hT = GDR.apply(q, k, v, g, beta, h0, cu, scale)     # autograd op

Per value head a V x K fp32 state S; per token S = e^g S, u = beta (v - S k),
S = S + u k^T, o = scale S q.  q, k: (B, T, Hk, K); v: (B, T, H, V), H a multiple
of Hk; K and V 64 or 128; fp32 or bf16.  g, beta: (B, T, H) fp32.  Outputs and
token gradients have the inputs' type; states and the gradients of g and beta
are fp32.  ``scale`` defaults to K ** -0.5.

``cu_seqlens`` (int32, N + 1 offsets on the GPU, B = 1) packs N sequences of any
lengths, empty ones included, along T; states are then (N, H, V, K).  The
offsets stay on the GPU: nothing waits for them, and a call can be captured into
a graph and replayed with other offsets.  (As with every autograd op, capture a
backward only on leaves that no live eager graph uses.)

Tensors are dense and lie at multiples of 16 bytes (g and beta: 4); GDR makes copies of
those that do not.  Calls of several
streams or threads may overlap as long as they share no output and no workspace.
"""
from __future__ import annotations

import ctypes
import functools

from . import BF16, F32, _check_bytes, _dense, _dense_on, _fits, _launch, _LazyOpOf, _ptr, _where, lib

GDR_CHUNK = 64


@functools.lru_cache(maxsize=None)
def _lib():
    L = lib()
    vp, i, i64, sz, f = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t, ctypes.c_float
    dims = [i] * 6
    L.gdr_slots.argtypes, L.gdr_slots.restype = [i] * 4, i64
    L.gdr_ckpt_bytes.argtypes, L.gdr_ckpt_bytes.restype = dims + [i] * 2, sz
    for n in ("gdr_fwd_workspace_bytes", "gdr_fwd_train_workspace_bytes", "gdr_bwd_workspace_bytes"):
        getattr(L, n).argtypes, getattr(L, n).restype = dims + [i] * 3, sz
    L.gdr_fwd.argtypes = dims + [i] + [vp] * 6 + [i, f] + [vp] * 4 + [vp, sz, vp]
    L.gdr_bwd.argtypes = dims + [i] + [vp] * 8 + [i, f] + [vp] * 7 + [vp, sz, vp]
    L.gdr_step.argtypes = dims + [i] + [vp] * 6 + [i, f] + [vp] * 4
    L.gdr_zero_outside.argtypes = [i, i, vp, i, vp, vp, vp]
    for n in ("gdr_fwd", "gdr_bwd", "gdr_step", "gdr_zero_outside"):
        getattr(L, n).restype = i
    return L


@functools.lru_cache(maxsize=None)
def _types():
    """The input types and their codes, and the type of gates and states."""
    import torch
    return {torch.float32: F32, torch.bfloat16: BF16}, torch.float32


@functools.lru_cache(maxsize=1024)
def _sizes(dims, code, N):
    """Bytes of the checkpoints, of the forward's workspace without and with them, and of the backward's."""
    L, packed = _lib(), int(N > 0)
    return (L.gdr_ckpt_bytes(*dims, N, packed), L.gdr_fwd_workspace_bytes(*dims, code, N, packed),
            L.gdr_fwd_train_workspace_bytes(*dims, code, N, packed), L.gdr_bwd_workspace_bytes(*dims, code, N, packed))


def _check_inputs(fn, q, k, v, g, beta):
    """(B, T, Hk, H, K, V) of the five token inputs, checked."""
    qs, vs = q.shape, v.shape
    if len(qs) != 4 or len(vs) != 4:
        raise ValueError(f"{fn}: q must be (B, T, Hk, K) and v (B, T, H, V), got {tuple(qs)} and {tuple(vs)}")
    B, T, Hk, K = qs
    H, V = vs[2], vs[3]
    if (K != 64 and K != 128) or (V != 64 and V != 128):
        raise ValueError(f"{fn}: K and V must be 64 or 128, got {K} and {V}")
    if B < 1 or T < 1 or Hk < 1 or H < 1 or H % Hk:
        raise ValueError(f"{fn}: B, T and heads must be at least 1 and H a multiple of Hk, got q {tuple(qs)}, "
                         f"v {tuple(vs)}")
    codes, f32 = _types()
    dev, dt, gs = q.device, q.dtype, (B, T, H)
    if dt not in codes:
        raise TypeError(f"{fn}: q must be float32 or bfloat16, got {dt}")
    if not (q.is_contiguous() and _fits(k, qs, dt, dev) and _fits(v, (B, T, H, V), dt, dev)
            and _fits(g, gs, f32, dev) and _fits(beta, gs, f32, dev)):
        for n, t, shape, d in (("q", q, qs, dt), ("k", k, qs, dt), ("v", v, (B, T, H, V), dt), ("g", g, gs, f32),
                               ("beta", beta, gs, f32)):
            _check_tensor(fn, n, t, shape, d, dev)
    return B, T, Hk, H, K, V


def _check_tensor(fn, name, t, shape, dtype, dev):
    if _fits(t, shape, dtype, dev):
        return
    if tuple(t.shape) != tuple(shape) or t.dtype != dtype:
        raise ValueError(f"{fn}: {name} is {_where(t)}, expected {tuple(shape)} {dtype}")
    _dense_on(fn, name, t, dev)


def _check_state(fn, name, t, shape, dev):
    if t is not None:
        _check_tensor(fn, name, t, shape, _types()[1], dev)


def _check_cu(fn, cu, B, dev):
    """Number of packed sequences (0: none)."""
    import torch
    if cu is None:
        return 0
    if cu.dtype != torch.int32 or cu.dim() != 1 or cu.numel() < 2:
        raise ValueError(f"{fn}: cu_seqlens is {_where(cu)}, expected (N + 1,) torch.int32")
    if B != 1:
        raise ValueError(f"{fn}: packed sequences need B = 1, got B = {B}")
    _dense_on(fn, "cu_seqlens", cu, dev)
    return cu.numel() - 1


def _code(dtype):
    return _types()[0][dtype]


def _workspace(fn, workspace, need, dev):
    import torch
    if workspace is None:
        return torch.empty(need, dtype=torch.uint8, device=dev), need
    _check_bytes(fn, "workspace", workspace, need, dev)
    return workspace, workspace.numel() * workspace.element_size()


def _zero_outside(cu, N, T, fresh):
    """Zero the rows of freshly made token tensors that no sequence covers."""
    n = len(fresh)
    ptrs = (ctypes.c_void_p * n)(*[t.data_ptr() for t in fresh])
    rows = (ctypes.c_int64 * n)(*[t.numel() // T * t.element_size() for t in fresh])
    _launch("gdr_zero_outside", _lib().gdr_zero_outside, cu.device, T, N, cu.data_ptr(), n, ptrs, rows)


def gdr_fwd(q, k, v, g, beta, h0=None, *, cu_seqlens=None, scale=None, want_o=True, want_ckpt=True, want_hT=True,
            o=None, ckpt=None, hT=None, workspace=None):
    """Forward.  Returns (o, ckpt, hT); entries not wanted are None.  Pre-allocated
    outputs may be passed; hT may be h0 (in-place update).  ``ckpt`` is what
    ``gdr_bwd`` needs, a flat fp32 tensor: not wanted for inference."""
    import torch
    fn = "gdr_fwd"
    B, T, Hk, H, K, V = _check_inputs(fn, q, k, v, g, beta)
    dev = q.device
    N = _check_cu(fn, cu_seqlens, B, dev)
    L, packed, states = _lib(), int(N > 0), (N or B, H, V, K)
    dims = (B, T, Hk, H, K, V)
    _check_state(fn, "h0", h0, states, dev)
    fresh = []
    if o is not None:
        _check_tensor(fn, "o", o, v.shape, v.dtype, dev)
    elif want_o:
        o = torch.empty_like(v)
        fresh.append(o)
    code = _code(q.dtype)
    nck, nws, nws_train, _ = _sizes(dims, code, N)
    if ckpt is not None:
        _check_state(fn, "ckpt", ckpt, (nck // 4,), dev)
    elif want_ckpt:
        ckpt = torch.empty(nck // 4, dtype=torch.float32, device=dev)
    if hT is not None:
        _check_state(fn, "hT", hT, states, dev)
    elif want_hT:
        hT = torch.empty(states, dtype=torch.float32, device=dev)
    workspace, wsb = _workspace(fn, workspace, nws if ckpt is None else nws_train, dev)
    _launch(fn, L.gdr_fwd, dev, *dims, code, q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(), beta.data_ptr(),
            _ptr(cu_seqlens), N, K ** -0.5 if scale is None else scale, _ptr(h0), _ptr(o), _ptr(ckpt), _ptr(hT),
            workspace.data_ptr(), wsb)
    if packed and fresh:
        _zero_outside(cu_seqlens, N, T, fresh)
    return o, ckpt, hT


def gdr_bwd(do, q, k, v, g, beta, ckpt, dhT=None, *, cu_seqlens=None, scale=None, want_dh0=True, workspace=None,
            out=None):
    """Backward.  Returns (dq, dk, dv, dg, dbeta, dh0); ``out`` may hold the first five."""
    import torch
    fn = "gdr_bwd"
    B, T, Hk, H, K, V = _check_inputs(fn, q, k, v, g, beta)
    dev = q.device
    N = _check_cu(fn, cu_seqlens, B, dev)
    L, packed, states = _lib(), int(N > 0), (N or B, H, V, K)
    dims = (B, T, Hk, H, K, V)
    _check_tensor(fn, "do", do, v.shape, v.dtype, dev)
    code = _code(q.dtype)
    nck, *_, nws = _sizes(dims, code, N)
    _check_state(fn, "ckpt", ckpt, (nck // 4,), dev)
    _check_state(fn, "dhT", dhT, states, dev)
    fresh = []
    if out is None:
        out = fresh = [torch.empty_like(x) for x in (q, k, v, g, beta)]
    if len(out) != 5:
        raise ValueError(f"{fn}: out must hold 5 tensors, got {len(out)}")
    for n, x, like in zip(("dq", "dk", "dv", "dg", "dbeta"), out, (q, k, v, g, beta)):
        _check_tensor(fn, n, x, like.shape, like.dtype, dev)
    dh0 = torch.empty(states, dtype=torch.float32, device=dev) if want_dh0 else None
    workspace, wsb = _workspace(fn, workspace, nws, dev)
    _launch(fn, L.gdr_bwd, dev, *dims, code, *map(_ptr, (do, dhT, q, k, v, g, beta, cu_seqlens)), N,
            K ** -0.5 if scale is None else scale, *map(_ptr, (ckpt, *out, dh0, workspace)), wsb)
    if packed and fresh:
        _zero_outside(cu_seqlens, N, T, fresh)
    return (*out, dh0)


def gdr_step(q, k, v, g, beta, state, *, slots=None, scale=None, state_out=None, o=None):
    """B rows of T new tokens, token by token; returns o.

    ``state`` (P, H, V, K) fp32 is updated in place, or into ``state_out`` (a
    tensor of the same shape, of which only the states worked on are written).
    ``slots`` (B,) int32 picks each row's state (row b uses state b without it);
    a row whose slot is outside 0 .. P - 1 is padding: its o is 0.  Rows with the
    same slot are consecutive tokens of one sequence, in row order."""
    fn = "gdr_step"
    B, T, Hk, H, K, V = _check_inputs(fn, q, k, v, g, beta)
    dev, P = q.device, state.shape[0] if state.dim() == 4 else 0
    if P < 1:
        raise ValueError(f"{fn}: state must be (P, H, V, K), got {tuple(state.shape)}")
    if slots is None:
        if P < B:
            raise ValueError(f"{fn}: state holds {P} states for {B} rows")
    else:
        import torch
        _check_tensor(fn, "slots", slots, (B,), torch.int32, dev)
    _check_state(fn, "state", state, (P, H, V, K), dev)
    if state_out is None:
        state_out = state
    else:
        _check_state(fn, "state_out", state_out, (P, H, V, K), dev)
    if o is None:
        o = v.new_empty(v.shape)
    else:
        _check_tensor(fn, "o", o, v.shape, v.dtype, dev)
    _launch(fn, _lib().gdr_step, dev, B, T, Hk, H, K, V, _code(q.dtype), q.data_ptr(), k.data_ptr(), v.data_ptr(),
            g.data_ptr(), beta.data_ptr(), _ptr(slots), P, K ** -0.5 if scale is None else scale, state.data_ptr(),
            state_out.data_ptr(), o.data_ptr())
    return o


def _make_autograd():
    import torch
    from torch.autograd.function import once_differentiable

    class GDR(torch.autograd.Function):
        """Differentiable op: (q, k, v, g, beta, h0, cu_seqlens, scale) -> (o, hT),
        gradients by gdr_bwd in the inputs' types.  Rows that no packed sequence
        covers have o = 0 and zero gradients."""

        @staticmethod
        def forward(ctx, q, k, v, g, beta, h0=None, cu_seqlens=None, scale=None):
            ctx.set_materialize_grads(False)               # a gradient that is not there costs nothing
            ins = [_dense(q), _dense(k), _dense(v), g.contiguous().float(), beta.contiguous().float()]
            h0c = None if h0 is None else _dense(h0.float())
            need = any(ctx.needs_input_grad)
            o, ckpt, hT = gdr_fwd(*ins, h0c, cu_seqlens=cu_seqlens, scale=scale, want_ckpt=need)
            ctx.save_for_backward(*ins, ckpt, cu_seqlens)
            ctx.scale, ctx.types = scale, (g.dtype, beta.dtype, None if h0 is None else h0.dtype)
            return o, hT

        @staticmethod
        @once_differentiable                               # a gradient of the gradient is an error, not a zero
        def backward(ctx, do, dhT):
            *ins, ckpt, cu = ctx.saved_tensors
            do = torch.zeros_like(ins[2]) if do is None else _dense(do.to(ins[2].dtype))
            dhT = None if dhT is None else _dense(dhT.float())
            tg, tb, th = ctx.types
            dq, dk, dv, dg, dbeta, dh0 = gdr_bwd(do, *ins, ckpt, dhT, cu_seqlens=cu, scale=ctx.scale,
                                                 want_dh0=th is not None)
            return dq, dk, dv, dg.to(tg), dbeta.to(tb), None if th is None else dh0.to(th), None, None

    return GDR


GDR = _LazyOpOf(_make_autograd)

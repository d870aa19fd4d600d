"""Calls of the gated delta rule and the layer norm that a program makes and their other tests do not."""
import pytest
import torch

import linear_rnn_lm_amd as L
from linear_rnn_lm_amd import gdr
from tests.gdr_util import make
from tests.gpu_util import note

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("dtype,code", [(BF, 1), (F32, 0)])
def test_workspace_of_the_training_forward_exactly(dtype, code):
    """A workspace of exactly the size that a forward with checkpoints asks for, with guards on both sides."""
    note(f"gdr training workspace {dtype}")
    q, k, v, g, beta, h0, do, dhT = [t.to(DEV) for t in make(2, 130, 2, 4, 64, 128, dtype, seed=3)]
    n = gdr._lib().gdr_fwd_train_workspace_bytes(2, 130, 2, 4, 64, 128, code, 0, 0)
    buf = torch.full((n + 512,), 7, dtype=torch.uint8, device=DEV)
    o, ckpt, hT = L.gdr_fwd(q, k, v, g, beta, h0, workspace=buf[256:256 + n])
    o2, _, hT2 = L.gdr_fwd(q, k, v, g, beta, h0, want_ckpt=False)
    grads = L.gdr_bwd(do, q, k, v, g, beta, ckpt, dhT)
    o3, ckpt3, _ = L.gdr_fwd(q, k, v, g, beta, h0)
    grads3 = L.gdr_bwd(do, q, k, v, g, beta, ckpt3, dhT)
    torch.cuda.synchronize()
    assert (buf[:256] == 7).all() and (buf[256 + n:] == 7).all()
    assert torch.equal(o, o2) and torch.equal(hT, hT2) and torch.equal(o, o3)
    assert all(torch.equal(a, b) for a, b in zip(grads, grads3))


def test_memory_of_the_training_forward():
    """Beside its outputs a forward of bf16 inputs with checkpoints allocates next to nothing."""
    note("gdr training memory")
    q, k, v, g, beta, *_ = [t.to(DEV) for t in make(1, 2048, 4, 4, 64, 64, BF, seed=4, h0=False) if t is not None]
    L.gdr_fwd(q, k, v, g, beta)
    torch.cuda.synchronize()
    torch.cuda.reset_peak_memory_stats()
    before = torch.cuda.memory_allocated()
    kept = L.gdr_fwd(q, k, v, g, beta)
    torch.cuda.synchronize()
    left = torch.cuda.memory_allocated() - before
    assert left >= sum(t.numel() * t.element_size() for t in kept)
    assert torch.cuda.max_memory_allocated() - before - left <= 4096


def at_odd(t):
    """The same values at an address that is no multiple of 16 bytes."""
    buf = torch.empty(t.numel() + 1, dtype=t.dtype, device=DEV)
    buf[1:] = t.to(DEV).reshape(-1)
    out = buf[1:].view(t.shape)
    assert out.is_contiguous() and out.data_ptr() % 16
    return out


@pytest.mark.parametrize("dtype", [BF, F32])
def test_autograd_ops_at_any_address(dtype):
    """Inputs, and the gradients that a concatenation of the outputs hands back, at odd addresses."""
    note(f"GDR and LN at odd addresses {dtype}")
    B, T, H, K = 1, 70, 2, 64
    q, k, v, g, beta, h0, do, dhT = make(B, T, H, H, K, K, dtype, seed=6)
    w = torch.randn(H * K, generator=torch.Generator().manual_seed(1))
    pieces = [torch.randn(n, generator=torch.Generator().manual_seed(n)).to(DEV) for n in (B * T * H * K, H * K * K)]

    def grads(place, cut):
        leaves = [place(t).requires_grad_() for t in (q, k, v, g, beta, h0, w, w + 1)]
        Q, Kk, Vv, G, Bt, S0, W, Bi = leaves
        x = L.LN.apply(Vv.reshape(B, T, H * K), W, Bi, H)
        o, hT = L.GDR.apply(Q, Kk, x.view(B, T, H, K), G, Bt, S0)
        y = L.LN.apply(o.reshape(B, T, H * K), W, Bi)
        outs = [y.reshape(-1), o.reshape(-1), hT.reshape(-1)]
        cots = [pieces[0].to(dtype), pieces[0].flip(0).to(dtype), pieces[1]]
        if cut:                                            # each output's gradient is a piece of a longer one
            outs = [torch.cat([t.new_zeros(1), t]) for t in outs]
            cots = [torch.cat([t.new_zeros(1), t]) for t in cots]
        return [y, o, hT, *torch.autograd.grad(outs, leaves, cots)]

    want = grads(lambda t: t.clone().to(DEV), False)
    for got in (grads(at_odd, False), grads(at_odd, True), grads(lambda t: t.clone().to(DEV), True)):
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_raw_calls_refuse_odd_addresses():
    note("gdr and ln, odd addresses refused")
    q, k, v, g, beta, h0, *_ = [t.to(DEV) for t in make(1, 5, 1, 1, 64, 64, BF, seed=6)]
    for args in ((at_odd(q), k, v, g, beta, h0), (q, k, at_odd(v), g, beta, h0), (q, k, v, g, beta, at_odd(h0))):
        with pytest.raises(L.Wkv7Error):
            L.gdr_fwd(*args)
    with pytest.raises(L.Wkv7Error):
        L.ln_fwd(at_odd(v.view(5, 64)))


@pytest.mark.parametrize("K,V,dtype", [(64, 64, BF), (128, 128, BF), (64, 128, F32)])
def test_rows_outside_are_not_read(K, V, dtype):
    """NaN in every input's rows before the first and behind the last sequence, and next to them."""
    note(f"gdr NaN outside K{K} V{V} {dtype}")
    cu, T = torch.tensor([7, 77, 77, 150], dtype=torch.int32, device=DEV), 170
    x = [t.to(DEV) for t in make(1, T, 2, 4, K, V, dtype, seed=8, N=3)]

    def both(q, k, v, g, beta, h0, do, dhT):
        o, ckpt, hT = L.gdr_fwd(q, k, v, g, beta, h0, cu_seqlens=cu)
        return [o, hT, *L.gdr_bwd(do, q, k, v, g, beta, ckpt, dhT, cu_seqlens=cu)]

    want = both(*x)
    for bad in (float("nan"), float("inf")):
        y = [t.clone() for t in x]
        for t in (*y[:5], y[6]):
            t[:, :7], t[:, 150:] = bad, bad
        got = both(*y)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_step_padding_and_other_states_are_not_read():
    """A padded batch whose padding rows, and states that no row works on, hold NaN; into another pool."""
    note("gdr step NaN in padding")
    B, P = 6, 5
    q, k, v, g, beta, h0, *_ = [t.to(DEV) for t in make(B, 2, 1, 2, 64, 64, BF, seed=9, N=P) if t is not None]
    slots = torch.tensor([3, -1, 0, P, 3, 2 ** 31 - 1], dtype=torch.int32, device=DEV)
    state, out = h0.clone(), torch.full_like(h0, 5.0)
    want = L.gdr_step(q, k, v, g, beta, state, slots=slots)
    x, s = [t.clone() for t in (q, k, v, g, beta)], h0.clone()
    for t in x:
        t[[1, 3, 5]] = float("nan")
    s[[1, 2, 4]] = float("nan")
    o = L.gdr_step(*x, s, slots=slots, state_out=out)
    torch.cuda.synchronize()
    assert torch.equal(o, want) and (o[[1, 3, 5]] == 0).all()
    assert torch.equal(out[[0, 3]], state[[0, 3]]) and (out[[1, 2, 4]] == 5).all()
    assert torch.equal(s[[0, 3]], h0[[0, 3]])


def test_two_backwards_of_one_graph():
    note("GDR and LN, backward twice")
    q, k, v, g, beta, h0, do, _ = [t.to(DEV) for t in make(1, 80, 1, 2, 128, 64, BF, seed=10)]
    leaves = [t.requires_grad_() for t in (q, k, v, g, beta, h0)]
    x = L.LN.apply(v.reshape(1, 80, 128), None, None, 2)
    o, hT = L.GDR.apply(q, k, x.view(v.shape), g, beta, h0)
    first = torch.autograd.grad(o, leaves, do, retain_graph=True)
    L.GDR.apply(q.detach() * 0.5, k, x.view(v.shape).detach(), g, beta, h0)       # other work in between
    second = torch.autograd.grad(o, leaves, do)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) and torch.isfinite(a).all() for a, b in zip(first, second))


def test_captured_packed_training_step():
    """Forward and backward through the autograd op, captured, replayed with other offsets and a gradient that is a
    piece of a longer one."""
    note("GDR packed autograd in a graph")
    T, N = 150, 3
    vals = [t.to(DEV) for t in make(1, T, 1, 2, 64, 64, BF, seed=12, N=N)[:6]]
    cu = torch.tensor([0, 70, 70, 150], dtype=torch.int32, device=DEV)
    cot = torch.randn(1 + T * 128, generator=torch.Generator().manual_seed(2)).to(DEV, BF)

    def grads(leaves):
        o, hT = L.GDR.apply(*leaves, cu)
        return [*torch.autograd.grad([torch.cat([o.new_zeros(1), o.reshape(-1)]), hT], leaves, [cot, torch.ones_like(hT)])]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        grads([x.clone().requires_grad_() for x in vals])
    torch.cuda.current_stream().wait_stream(side)
    leaves = [x.clone().requires_grad_() for x in vals]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = grads(leaves)
    for offsets in ([0, 70, 70, 150], [3, 64, 128, 140], [0, 0, 0, 0], [0, 1, 149, 150], [0, 70, 70, 150]):
        cu.copy_(torch.tensor(offsets, dtype=torch.int32))
        graph.replay()
        got = [t.clone() for t in outs]
        want = grads([x.detach().clone().requires_grad_() for x in leaves])
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)), offsets

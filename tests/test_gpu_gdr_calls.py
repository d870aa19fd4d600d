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

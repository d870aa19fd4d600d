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

"""Where the gated delta rule's products nearly cancel: its results have to keep the digits that fp32 has."""
import pytest
import torch

import linear_rnn_lm_amd as L
from tests.gdr_util import make, reference, rel, tol_bwd
from tests.gpu_util import note

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
BF, F32 = torch.bfloat16, torch.float32


# B, Hk, H: one slice per workgroup, two, and (K = 64) four
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("K,V,B,Hk,H", [(64, 64, 1, 1, 1), (64, 128, 1, 40, 40), (64, 128, 2, 16, 64), (128, 64, 1, 1, 2),
                                        (128, 128, 2, 10, 20)])
def test_a_large_state_is_overwritten(K, V, B, Hk, H, dtype):
    """q = k, one unit vector per token and each its own, beta = 1, g = 0: token t replaces column t of a state of
    size R and reads the new value, o = scale v, as the difference of two terms of size R.

    Every sum has one or two terms that are not 0, and every gate, T and M are 1 or 0, exactly.  So o is off by
    its own rounding (2^-8 for bf16) and by the additions of terms of size R: s from its planes, v - s, the same
    two once more for u, and the planes of u added to s, at most eight of them, each rounded or cut in its last
    place (2^-23 R): 16 2^-24 R scale.  Two planes for s or u would leave out 2^-18 R."""
    note(f"gdr overwritten state K{K} V{V} B{B} Hk{Hk} H{H} {dtype}")
    T, R, scale = 100, 2.0 ** 16, 0.5
    _, _, v, g, _, h0, *_ = make(B, T, Hk, H, K, V, dtype, seed=K + V)
    one = torch.zeros(B, T, Hk, K)
    one[:, torch.arange(T), :, torch.arange(T) % K] = 1.0
    x = (one.to(dtype), one.to(dtype), v, torch.zeros_like(g), torch.ones_like(g))
    h0 = R * (2 * torch.rand(h0.shape, generator=torch.Generator().manual_seed(1)) - 1)
    o, _, hT = L.gdr_fwd(*[t.to(DEV) for t in x], h0.to(DEV), scale=scale)
    torch.cuda.synchronize()
    want = reference(*x, h0, scale=scale)
    half = 2.0 ** -8 if dtype == BF else 2.0 ** -24
    first = (o.double().cpu() - want["o"]).abs() - half * want["o"].abs()
    assert first.max() <= 16 * 2.0 ** -24 * R * scale, first.max()
    assert (hT.double().cpu() - want["hT"]).abs().max() <= 16 * 2.0 ** -24 * R


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("K,V,Hk,H", [(64, 64, 2, 2), (64, 128, 1, 3), (128, 64, 2, 2), (128, 128, 2, 4)])
@pytest.mark.parametrize("kind", [-2.0, -5.0, -10.0, -20.0, "some"])
def test_gradient_of_strong_decays(kind, K, V, Hk, H, dtype):
    """dg in relation to its own size, however much the heads forget.

    Every part of dg carries the decay of its token, so the sums' bound holds relative to dg.  A
    decay e^x is rounded by 2^-24 |x| log2(e) relative (the exponent's last place), twice where it
    is a factor of a derived operand too: 3 |g| 2^-24 more.  "some": g = -20 at every seventh token, -0.01 at the
    others, and the two kinds of tokens are looked at apart."""
    note(f"gdr dg under decays {kind} K{K} V{V} Hk{Hk} H{H} {dtype}")
    T = 150
    q, k, v, g, beta, h0, do, dhT = make(2, T, Hk, H, K, V, dtype, seed=17)
    strong = torch.zeros(T, dtype=torch.bool)
    if kind == "some":
        strong[::7] = True
        g = torch.where(strong[:, None], torch.tensor(-20.0), torch.tensor(-0.01)).expand_as(g).contiguous()
    else:
        g = torch.full_like(g, kind)
    want = reference(q, k, v, g, beta, h0, do, dhT)
    ins = [t.to(DEV) for t in (q, k, v, g, beta)]
    _, ckpt, _ = L.gdr_fwd(*ins, h0.to(DEV))
    got = L.gdr_bwd(do.to(DEV), *ins, ckpt, dhT.to(DEV))
    torch.cuda.synchronize()
    for n, t in zip(("dq", "dk", "dv", "dg", "dbeta", "dh0"), got):
        tol = tol_bwd(K, V, t.dtype) + 3 * g.abs().max().item() * 2.0 ** -24
        if n == "dg" and kind == "some":
            for at in (strong, ~strong):
                assert rel(t[:, at], want[n][:, at]) <= tol, (n, rel(t[:, at], want[n][:, at]), tol)
        else:
            assert rel(t, want[n]) <= tol, (n, rel(t, want[n]), tol)

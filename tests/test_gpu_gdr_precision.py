"""Where the gated delta rule's products nearly cancel: its results have to keep the digits that fp32 has."""
import pytest
import torch

import linear_rnn_lm_amd as L
from tests.gdr_util import make, reference
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

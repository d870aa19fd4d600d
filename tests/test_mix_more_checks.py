"""More of what the selective scan, the short convolution and the block norm take and refuse, on the
host (CPU only): made-up device addresses; every call fails a check, so nothing is launched."""
import torch

import linear_rnn_lm_amd as L
from linear_rnn_lm_amd import rnorm, ssm
from tests.test_abi import ERR_ALIGN, ERR_ARG, ERR_SHAPE, fake, needs_no_gpu
from tests.test_mix_checks import call


@needs_no_gpu
def test_row_distances():
    """A step takes the last tokens of long rows; over sequences the distance is limited."""
    lib = ssm._lib()
    dims = dict(B=2, T=1, C=64, S=16, G=1, t=1)
    big = dict(x=fake(0), xl=64, dt=fake(20), dl=64, A=fake(2), b=fake(30), bl=16, c=fake(40), cl=16, D=fake(5), z=fake(50), zl=64,
               bias=fake(7), sp=1)
    s = lambda **o: call(lib.ssm_step, dict(**dims, **big, slots=None, P=2, st=fake(8), so=fake(9), y=fake(10)), o)  # noqa: E731
    f = lambda **o: call(lib.ssm_fwd, dict(**dims, **big, cu=None, N=0, zo=0, h0=None, y=fake(8), ck=fake(9), hT=fake(10),  # noqa: E731
                                           ws=fake(11), wsb=1 << 24), o)
    for n in ("xl", "dl", "bl", "cl", "zl"):
        # past the check of shapes the missing output is what is wrong
        assert s(**{n: (1 << 24) + 8}, y=None) == ERR_ARG
        assert f(**{n: (1 << 24) + 8}) == ERR_SHAPE == s(**{n: 1 << 41}, y=None)


def test_many_sequences():
    """As many segments as a launch has threads for, fewer than 2^32 at 512 to a segment and 64 channels."""
    lib = ssm._lib()
    most = 2 ** 23 - 1
    for size in (lib.ssm_fwd_workspace_bytes, lib.ssm_bwd_workspace_bytes):
        assert size(most, 1, 64, 16, 1, 0, 0) > 0 == size(most + 1, 1, 64, 16, 1, 0, 0)
        assert size(most // 64, 1, 4096, 16, 1, 0, 0) > 0 == size(most // 64 + 1, 1, 4096, 16, 1, 0, 0)
        assert size(1, 15, 64, 16, 1, most, 1) > 0 == size(1, 15, 64, 16, 1, most + 1, 1)


def test_nothing_for_a_backward_without_gradients(monkeypatch):
    """SSM's checkpoints and RN's statistics are asked for only where a backward may follow."""
    asked = []

    def scan(x, dt, A, *rest, want_ckpt, **kw):
        asked.append(want_ckpt)
        return x.clone(), torch.zeros(1), x.new_zeros(1, *A.shape)

    def norm(o, *rest, want_stats, **kw):
        asked.append(want_stats)
        return o.clone(), None, torch.zeros(1)

    monkeypatch.setattr(ssm, "ssm_fwd", scan)
    monkeypatch.setattr(rnorm, "rn_fwd", norm)
    x, A, b = torch.zeros(1, 3, 8), torch.zeros(8, 16), torch.zeros(1, 3, 1, 16)
    param, w = A.clone().requires_grad_(), torch.ones(8, requires_grad=True)
    for mode, want in ((torch.enable_grad, True), (torch.no_grad, False), (torch.inference_mode, False)):
        asked.clear()
        with mode():
            y, hT = L.SSM.apply(x, x, param, b, b)
            r, h = L.RN.apply(x[0], None, None, w)
        assert asked == [want, want] and h is None
        assert y.requires_grad == hT.requires_grad == r.requires_grad == want
    asked.clear()
    L.SSM.apply(x, x, A, b, b)                             # nothing has a gradient
    L.RN.apply(x[0])
    assert asked == [False, False]


@needs_no_gpu
def test_gate_rows_at_multiples_of_16_bytes():
    lib = rnorm._lib()
    kinds = dict(rows=4, C=128, G=2, n1=1, n2=2, act=1, o_t=0, io_t=1, r_t=1, w_t=0)
    w = dict(w1=None, b1=None, sc=None, w2=None)
    f = lambda **o: call(lib.rn_fwd, dict(**kinds, e1=1e-5, e2=1e-5, o=fake(0), g=fake(1), gl=128, res=fake(2), **w, b2=None,  # noqa: E731
                                          r=None, h=fake(10), st=None), o)
    g = lambda **o: call(lib.rn_bwd, dict(**kinds, dr=fake(12), dh=fake(13), o=fake(0), g=fake(1), gl=128, res=fake(2),  # noqa: E731
                                          st=None, **w, do=fake(14), dg=fake(15), dres=None, dw=None, ws=None, wsb=0), o)
    for c in (f, g):                                       # what is missing is found behind the rows' distance
        assert c(io_t=0, r_t=0, gl=132) == c(gl=136) == ERR_ARG
        assert c(io_t=0, r_t=0, gl=130) == c(gl=132) == ERR_ALIGN

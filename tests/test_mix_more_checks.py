"""More of what the selective scan, the short convolution and the block norm take and refuse, on the
host (CPU only): made-up device addresses; every call fails a check, so nothing is launched."""
import linear_rnn_lm_amd as L  # noqa: F401  (the binding sets the library's argument types)
from linear_rnn_lm_amd import ssm
from tests.test_abi import ERR_ARG, ERR_SHAPE, fake, needs_no_gpu
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

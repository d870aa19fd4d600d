"""Refusals of the selective scan, the short convolution and the block norm, on the host (CPU
only): the C entry points reject bad arguments before anything is launched (made-up device
addresses; every case fails a check), and the binding checks every tensor."""
import os
import random
import re

import pytest
import torch

import linear_rnn_lm_amd as L
from linear_rnn_lm_amd import conv, rnorm, ssm
from tests.test_abi import ERR_ALIAS, ERR_ALIGN, ERR_ARG, ERR_DTYPE, ERR_SHAPE, ERR_WS, fake, needs_no_gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("prefix,header", [("ssm", "ssm.h"), ("conv", "conv.h"), ("rn", "rnorm.h")])
def test_declared_functions_are_exported(prefix, header):
    src = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", header)).read(), flags=re.S)
    names = set(re.findall(rf"\b({prefix}_[a-z0-9_]+)\s*\(", src))
    assert names
    out = os.popen(f"nm -D --defined-only {L.LIB_PATH}").read()
    assert set(re.findall(rf"\bT ({prefix}_[a-z0-9_]+)\b", out)) == names


def test_size_queries():
    lib = ssm._lib()
    assert [lib.ssm_slots(2, t, 0, 0) for t in (1, 16, 17)] == [2, 2, 4]
    assert lib.ssm_slots(1, 200, 5, 1) == 200 // 16 + 5
    assert lib.ssm_slots(2, 200, 5, 1) == 0 and lib.ssm_slots(1, 0, 1, 0) == 0
    assert lib.ssm_ckpt_bytes(2, 17, 10, 16, 1, 0, 0) == 4 * 10 * 16 * 4
    for bad in ((0, 17, 10, 16, 1), (2, 0, 10, 16, 1), (2, 17, 0, 16, 1), (2, 17, 10, 8, 1), (2, 17, 10, 16, 3),
                (2, 17, 96, 16, 2), (1, 2 ** 31 - 1, 2 ** 20, 16, 1)):
        assert lib.ssm_ckpt_bytes(*bad, 0, 0) == lib.ssm_fwd_workspace_bytes(*bad, 0, 0) == 0
        assert lib.ssm_bwd_workspace_bytes(*bad, 0, 0) == 0
    assert lib.ssm_fwd_workspace_bytes(2, 17, 10, 16, 1, 0, 0) > 0 and lib.ssm_bwd_workspace_bytes(2, 17, 10, 16, 1, 0, 0) > 0
    c = conv._lib()
    assert c.conv_bwd_workspace_bytes(1, 16, 8, 4, 0, 0) == 5 * 8 * 4
    assert c.conv_bwd_workspace_bytes(1, 16, 8, 5, 0, 0) == 0 and c.conv_bwd_workspace_bytes(2, 16, 8, 4, 3, 1) == 0
    # positions of 32 bits, with room behind the last token; and one more offset than sequences
    assert lib.ssm_fwd_workspace_bytes(1, 2 ** 31 - 1024, 16, 16, 1, 0, 0) == 0 < lib.ssm_fwd_workspace_bytes(1, 2 ** 31 - 1025, 16, 16, 1, 0, 0)
    assert c.conv_bwd_workspace_bytes(1, 2 ** 31 - 1024, 1, 4, 0, 0) == 0 < c.conv_bwd_workspace_bytes(1, 2 ** 31 - 1025, 1, 4, 0, 0)
    assert c.conv_bwd_workspace_bytes(1, 16, 1, 4, 2 ** 31 - 1, 1) == 0 == lib.ssm_bwd_workspace_bytes(1, 16, 1, 16, 1, 2 ** 31 - 1, 1)
    r = rnorm._lib()
    assert r.rn_bwd_workspace_bytes(1, 8, 1) == 8 * 5 * 4
    assert r.rn_bwd_workspace_bytes(0, 8, 1) == 0 and r.rn_bwd_workspace_bytes(4, 96, 2) == 0
    assert r.rn_bwd_workspace_bytes(4, 8200, 1) == 0


def test_checkpoint_and_segment_slots_never_overlap():
    """Slots of packed pieces, as the kernels count them: within their number, no two the same."""
    rnd = random.Random(0)
    for _ in range(300):
        T, N, length = rnd.randint(1, 400), rnd.randint(1, 12), rnd.choice([16, 32, 64, 128])
        cu = sorted(rnd.randint(0, T) for _ in range(N + 1))
        seen = set()
        for n in range(N):
            pieces = max(1, -(-(cu[n + 1] - cu[n]) // length))
            for i in range(pieces):
                s = cu[n] // length + n + i
                assert 0 <= s < T // length + N and s not in seen
                seen.add(s)


def ins(x=0, ld=None):
    return dict(x=fake(x), xl=64, dt=fake(x + 1), dl=64, A=fake(x + 2), b=fake(x + 3), bl=16, c=fake(x + 4), cl=16, D=fake(x + 5),
                z=fake(x + 6), zl=64, bias=fake(x + 7), sp=1)


def call(fn, base, over):
    assert set(over) <= set(base), over
    return fn(*{**base, **over}.values(), None)


@needs_no_gpu
def test_ssm_entry_points_reject_bad_arguments():
    lib = ssm._lib()
    dims = dict(B=1, T=40, C=64, S=16, G=1, t=1)
    f = lambda **o: call(lib.ssm_fwd, dict(**dims, **ins(), cu=None, N=0, zo=0, h0=None, y=fake(8), ck=fake(9), hT=fake(10),  # noqa: E731
                                           ws=fake(11), wsb=1 << 24), o)
    g = lambda **o: call(lib.ssm_bwd, dict(**dims, dy=fake(8), dhT=None, **ins(), cu=None, N=0, zo=0, ck=fake(9), dx=fake(10),  # noqa: E731
                                           ddt=fake(11), dA=fake(12), db=fake(13), dc=fake(14), dD=fake(15), dz=fake(16),
                                           dbias=fake(17), dh0=fake(18), ws=fake(19), wsb=1 << 24), o)
    s = lambda **o: call(lib.ssm_step, dict(**dims, **ins(), slots=None, P=1, st=fake(8), so=fake(9), y=fake(10)), o)  # noqa: E731
    for c in (f, g, s):
        assert c(B=0) == c(T=0) == c(C=0) == c(S=8) == c(G=0) == c(G=2) == ERR_SHAPE
        assert c(C=100) == ERR_SHAPE                       # rows of 64 values would overlap
        assert c(xl=63) == c(dl=10) == c(bl=15) == c(cl=0) == c(zl=1) == c(xl=2 ** 62) == ERR_SHAPE
        assert c(t=2) == c(t=-1) == ERR_DTYPE
        for n in ("x", "dt", "A", "b", "c"):
            assert c(**{n: None}) == ERR_ARG
        assert c(x=fake(0) + 1) == c(A=fake(2) + 8) == c(D=fake(5) + 2) == ERR_ALIGN
    for c in (f, g):
        assert c(B=2, cu=fake(20), N=2) == c(cu=fake(20), N=0) == ERR_SHAPE
        assert c(cu=fake(20) + 2, N=1) == ERR_ALIGN
        assert c(ws=None) == ERR_WS and c(wsb=8) == ERR_WS
    assert f(y=None, ck=None, hT=None) == ERR_ARG
    assert f(y=fake(0)) == f(hT=fake(9)) == f(ck=fake(8)) == f(h0=fake(10) + 64) == f(ws=fake(8)) == ERR_ALIAS
    assert f(hT=fake(10) + 4) == ERR_ALIGN
    for n in ("dy", "ck", "dx", "ddt", "dA", "db", "dc", "dD", "dz"):
        assert g(**{n: None}) == ERR_ARG
    assert g(D=None) == g(z=None) == ERR_ARG               # their gradients without them
    assert g(dx=fake(8)) == g(dc=fake(13)) == g(dh0=fake(9)) == g(dhT=fake(18)) == ERR_ALIAS
    assert s(P=0) == s(B=2, P=1) == ERR_SHAPE and s(slots=fake(11) + 2) == ERR_ALIGN
    assert s(st=None) == s(so=None) == s(y=None) == ERR_ARG
    assert s(so=fake(8) + 64) == s(y=fake(8)) == s(slots=fake(10)) == ERR_ALIAS


@needs_no_gpu
def test_conv_entry_points_reject_bad_arguments():
    lib = conv._lib()
    dims = dict(B=1, T=40, C=64, W=4, t=1, wt=0)
    x = dict(x=fake(0), xl=64, w=fake(1), bias=fake(2), silu=1)
    f = lambda **o: call(lib.conv_fwd, dict(**dims, **x, cu=None, N=0, zo=0, h0=fake(3), y=fake(4), hT=fake(5)), o)  # noqa: E731
    g = lambda **o: call(lib.conv_bwd, dict(**dims, dy=fake(6), dhT=None, **x, cu=None, N=0, zo=0, h0=fake(3), dx=fake(7),  # noqa: E731
                                            dw=fake(8), db=fake(9), dh0=fake(10), ws=fake(11), wsb=1 << 24), o)
    s = lambda **o: call(lib.conv_step, dict(**dims, **x, slots=None, P=1, st=fake(3), so=fake(4), y=fake(5)), o)  # noqa: E731
    for c in (f, g, s):
        assert c(B=0) == c(T=0) == c(C=0) == c(W=1) == c(W=5) == c(xl=63) == ERR_SHAPE
        assert c(t=2) == c(wt=7) == ERR_DTYPE
        assert c(x=None) == c(w=None) == ERR_ARG
        assert c(x=fake(0) + 1) == c(w=fake(1) + 2) == ERR_ALIGN
    for c in (f, g):
        assert c(B=2, cu=fake(20), N=2) == c(cu=fake(20), N=0) == ERR_SHAPE
    assert f(y=None) == ERR_ARG and f(y=fake(0)) == f(hT=fake(3)) == f(hT=fake(4)) == ERR_ALIAS
    for n in ("dy", "dx", "dw"):
        assert g(**{n: None}) == ERR_ARG
    assert g(dx=fake(6)) == g(dh0=fake(3)) == g(db=fake(8)) == ERR_ALIAS and g(ws=None) == g(wsb=4) == ERR_WS
    assert s(P=0) == s(B=2, P=1) == ERR_SHAPE and s(st=None) == s(so=None) == s(y=None) == ERR_ARG
    assert s(so=fake(3) + 64) == s(y=fake(3)) == ERR_ALIAS


@needs_no_gpu
def test_rn_entry_points_reject_bad_arguments():
    lib = rnorm._lib()
    kinds = dict(rows=4, C=128, G=2, n1=1, n2=2, act=1, o_t=0, io_t=1, r_t=1, w_t=0)
    w = dict(w1=fake(4), b1=fake(5), sc=fake(6), w2=fake(7))
    f = lambda **o: call(lib.rn_fwd, dict(**kinds, e1=1e-5, e2=1e-5, o=fake(0), g=fake(1), gl=128, res=fake(2), **w, b2=fake(8),  # noqa: E731
                                          r=fake(9), h=fake(10), st=fake(11)), o)
    g = lambda **o: call(lib.rn_bwd, dict(**kinds, dr=fake(12), dh=fake(13), o=fake(0), g=fake(1), gl=128, res=fake(2),  # noqa: E731
                                          st=fake(11), **w, do=fake(14), dg=fake(15), dres=fake(16), dw=fake(17), ws=fake(18),
                                          wsb=1 << 20), o)
    for c in (f, g):
        assert c(rows=0) == c(C=8320, G=1) == c(C=96) == c(G=0) == c(C=32) == c(gl=100) == ERR_SHAPE
        assert c(o_t=1, io_t=0) == c(r_t=1, io_t=0) == c(w_t=3) == c(o_t=2) == ERR_DTYPE
        assert c(res=None, r_t=0) == ERR_DTYPE
        assert c(n1=0) == c(n2=3) == c(act=5) == c(act=0) == c(g=None) == c(o=None) == ERR_ARG
        assert c(o=fake(0) + 8) == c(gl=129) == c(w1=fake(4) + 4) == ERR_ALIGN
    assert f(r=None) == f(h=None) == f(n2=0) == ERR_ARG
    assert f(r=fake(2)) == f(h=fake(1)) == f(st=fake(9)) == ERR_ALIAS
    assert g(dr=None, dh=None) == g(n2=0) == g(dg=None) == g(st=None) == g(res=None) == ERR_ARG
    assert g(do=fake(12)) == g(dg=fake(1)) == g(dw=fake(18)) == ERR_ALIAS and g(ws=None) == g(wsb=100) == ERR_WS


# ------------------------------------------------------------------ the binding
def scan_ins(B=2, T=5, C=128, S=16, G=2, dt=BF):
    z = lambda *s: torch.zeros(*s, dtype=dt)  # noqa: E731
    return [z(B, T, C), z(B, T, C), torch.zeros(C, S), z(B, T, G, S), z(B, T, G, S)]


def swap(x, i, t):
    x = list(x)
    x[i] = t
    return x


def test_binding_checks_ssm():
    x = scan_ins()
    ck, st = torch.zeros(2, 128, 16), torch.zeros(2, 128, 16)
    calls = [lambda *a, **k: L.ssm_fwd(*a, **k), lambda *a, **k: L.ssm_step(*a, st, **k),
             lambda *a, **k: L.ssm_bwd(torch.zeros(2, 5, 128, dtype=BF), *a, ck, **k)]
    for f in calls:
        with pytest.raises(ValueError, match="GPU tensors"):
            f(*x)
        with pytest.raises(ValueError, match="dt is"):
            f(*swap(x, 1, x[1].float()))
        with pytest.raises(ValueError, match="A is"):
            f(*swap(x, 2, x[2].to(BF)))
        with pytest.raises(ValueError, match="c is"):
            f(*swap(x, 4, x[4][:, :, :1].contiguous()))
        with pytest.raises(ValueError, match="A must be contiguous"):
            f(*swap(x, 2, torch.zeros(16, 128).t()))
        with pytest.raises(ValueError, match="one distance"):
            f(*swap(x, 0, torch.zeros(5, 2, 128, dtype=BF).transpose(0, 1)))
        with pytest.raises(ValueError, match="one distance"):
            f(*swap(x, 3, torch.zeros(2, 5, 16, 2, dtype=BF).transpose(2, 3)))
        with pytest.raises(ValueError, match="one distance"):
            f(*swap(x, 1, torch.zeros(2, 1, 128, dtype=BF).expand(2, 5, 128)))
        with pytest.raises(ValueError, match="16, 32 or 64"):
            f(*scan_ins(S=8))
        with pytest.raises(ValueError, match="multiple of 64"):
            f(*scan_ins(C=96))
        with pytest.raises(TypeError, match="float32 or bfloat16"):
            f(*scan_ins(dt=torch.float16))
        with pytest.raises(ValueError, match="dt_bias is"):
            f(*x, dt_bias=torch.zeros(64))
    one = scan_ins(B=1)
    with pytest.raises(ValueError, match="B = 1"):
        L.ssm_fwd(*x, cu_seqlens=torch.tensor([0, 5], dtype=torch.int32))
    with pytest.raises(ValueError, match="int32"):
        L.ssm_fwd(*one, cu_seqlens=torch.tensor([0, 5]))
    with pytest.raises(ValueError, match="h0"):
        L.ssm_fwd(*x, None, None, torch.zeros(1, 128, 16))
    with pytest.raises(ValueError, match="z is"):
        L.ssm_fwd(*x, None, torch.zeros(2, 5, 64, dtype=BF))
    with pytest.raises(ValueError, match="ckpt"):
        L.ssm_fwd(*x, ckpt=torch.zeros(1, 128, 16))
    with pytest.raises(ValueError, match="workspace"):
        L.ssm_bwd(torch.zeros(2, 5, 128, dtype=BF), *x, ck, workspace=torch.zeros(16, dtype=torch.uint8))
    with pytest.raises(ValueError, match="8 entries"):
        L.ssm_bwd(torch.zeros(2, 5, 128, dtype=BF), *x, ck, out=[None] * 3)
    with pytest.raises(ValueError, match="dx must be given"):
        L.ssm_bwd(torch.zeros(2, 5, 128, dtype=BF), *x, ck, out=[None] * 8)
    with pytest.raises(ValueError, match="1 states for 2 rows"):
        L.ssm_step(*x, st[:1].contiguous())
    with pytest.raises(ValueError, match="slots"):
        L.ssm_step(*x, st, slots=torch.zeros(2, dtype=torch.int64))
    with pytest.raises(ValueError, match="state_out"):
        L.ssm_step(*x, st, state_out=st.to(BF))


def test_binding_checks_conv():
    x, w, b, st = torch.zeros(2, 5, 24, dtype=BF), torch.zeros(24, 4), torch.zeros(24), torch.zeros(2, 3, 24, dtype=BF)
    calls = [lambda *a: L.conv_fwd(*a), lambda *a: L.conv_step(*a, st), lambda *a: L.conv_bwd(torch.zeros_like(x), *a)]
    for f in calls:
        with pytest.raises(ValueError, match="GPU tensors"):
            f(x, w, b)
        with pytest.raises(ValueError, match="W 2, 3 or 4"):
            f(x, torch.zeros(24, 5), b)
        with pytest.raises(ValueError, match="bias is"):
            f(x, w, b.to(BF))
        with pytest.raises(ValueError, match="weight is"):
            f(x, torch.zeros(23, 4), b)
        with pytest.raises(ValueError, match="contiguous"):
            f(x, torch.zeros(4, 24).t(), b)
        with pytest.raises(TypeError, match="float32 or bfloat16"):
            f(x.half(), w, b)
        with pytest.raises(ValueError, match="one distance"):
            f(torch.zeros(2, 24, 5, dtype=BF).transpose(1, 2), w, b)
    with pytest.raises(ValueError, match="h0"):
        L.conv_fwd(x, w, b, st.float())
    with pytest.raises(ValueError, match="hT"):
        L.conv_fwd(x, w, b, hT=torch.zeros(2, 4, 24, dtype=BF))
    with pytest.raises(ValueError, match="dbias"):
        L.conv_bwd(torch.zeros_like(x), x, w, b, out=(torch.zeros_like(x), w, None))
    with pytest.raises(ValueError, match="state is"):
        L.conv_step(x, w, b, st.float())
    with pytest.raises(ValueError, match="1 states for 2 rows"):
        L.conv_step(x, w, b, st[:1].contiguous())


def test_binding_checks_rn():
    o, w = torch.zeros(4, 128), torch.zeros(128)
    with pytest.raises(ValueError, match="GPU tensors"):
        L.rn_fwd(o, o, o, weight=w)
    with pytest.raises(ValueError, match="parts"):
        L.rn_fwd(o, groups=4)
    with pytest.raises(ValueError, match="at most 8192"):
        L.rn_fwd(torch.zeros(1, 8200))
    with pytest.raises(ValueError, match="not empty"):
        L.rn_fwd(torch.zeros(0, 8))
    with pytest.raises(ValueError, match="norm must be"):
        L.rn_fwd(o, norm=None)
    with pytest.raises(ValueError, match="act must be"):
        L.rn_fwd(o, o, act="tanh")
    with pytest.raises(ValueError, match="need norm2"):
        L.rn_fwd(o, weight2=w)
    with pytest.raises(ValueError, match="one type"):
        L.rn_fwd(o, weight=w, scale=w.to(BF))
    with pytest.raises(TypeError, match="cannot give"):
        L.rn_fwd(o.to(BF), out_dtype=F32)
    with pytest.raises(TypeError, match="res must be"):
        L.rn_fwd(o, None, o.to(BF))
    with pytest.raises(ValueError, match="gate"):
        L.rn_fwd(o, torch.zeros(4, 64))
    with pytest.raises(ValueError, match="one distance"):
        L.rn_fwd(o, torch.zeros(128, 4).t())
    with pytest.raises(ValueError, match="contiguous"):
        L.rn_fwd(torch.zeros(128, 4).t())
    st = torch.zeros(4, 4)
    with pytest.raises(ValueError, match="dr or dh"):
        L.rn_bwd(None, None, o, None, None, st)
    with pytest.raises(ValueError, match="needs norm2"):
        L.rn_bwd(None, o, o, None, None, st)
    with pytest.raises(ValueError, match="stats"):
        L.rn_bwd(o, None, o, None, None, st, groups=2)
    with pytest.raises(ValueError, match="wanted"):
        L.rn_bwd(o, None, o, None, None, st, weight=w, want_do=False, want_dw=False)

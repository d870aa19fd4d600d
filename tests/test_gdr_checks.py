"""The gated delta rule's and the layer norm's refusals, on the host (CPU only):
the C entry points reject bad arguments before anything is launched (made-up
device addresses; every case fails a check), the binding checks every tensor,
and the chunk slots of packed sequences never overlap or leave their buffers."""
import ctypes
import os
import random
import re

import pytest
import torch

import linear_rnn_lm_amd as L
from linear_rnn_lm_amd import gdr, lnorm
from tests.test_abi import ERR_ALIAS, ERR_ALIGN, ERR_ARG, ERR_DTYPE, ERR_SHAPE, ERR_WS, fake, needs_no_gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("header", ["gdr.h", "lnorm.h"])
def test_declared_functions_are_exported(header):
    src = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", header)).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b((?:gdr|ln)_[a-z0-9_]+)\s*\(", src)))
    assert names
    out = os.popen(f"nm -D --defined-only {L.LIB_PATH}").read()
    prefix = "gdr" if header == "gdr.h" else "ln"
    exported = set(re.findall(rf"\bT ({prefix}_[a-z0-9_]+)\b", out))
    assert exported == set(names)


def test_size_queries():
    lib = gdr._lib()
    assert [lib.gdr_slots(2, t, 0, 0) for t in (1, 64, 65)] == [2, 2, 4]
    assert lib.gdr_slots(1, 200, 5, 1) == 200 // 64 + 5
    assert lib.gdr_slots(2, 200, 5, 1) == 0 and lib.gdr_slots(1, 0, 1, 0) == 0
    assert lib.gdr_ckpt_bytes(2, 65, 2, 4, 64, 128, 0, 0) == 4 * 4 * ((64 + 64) * 128 + 6464) * 4
    assert lib.gdr_ckpt_bytes(2, 65, 3, 4, 64, 128, 0, 0) == 0          # H not a multiple of Hk
    assert lib.gdr_ckpt_bytes(2, 65, 2, 4, 96, 128, 0, 0) == 0
    f = [lib.gdr_fwd_workspace_bytes(2, 65, 2, 4, 64, 128, dt, 0, 0) for dt in (0, 1)]
    assert f[0] == f[1] + 2 * 3 * 2 * (2 * 65 * 2 * 64)                 # planes of fp32 q and k
    assert f[1] == 16 * 3392 * 4
    assert lib.gdr_bwd_workspace_bytes(2, 65, 2, 4, 64, 128, 1, 0, 0) == 16 * 128 * (64 + 64) * 4
    assert lib.gdr_fwd_workspace_bytes(2, 65, 2, 4, 64, 128, 3, 0, 0) == 0
    ln = lnorm._lib()
    assert ln.ln_bwd_workspace_bytes(1, 8, 1) == 8 * 2 * 4
    assert ln.ln_bwd_workspace_bytes(0, 8, 1) == 0 and ln.ln_bwd_workspace_bytes(4, 9, 2) == 0
    assert ln.ln_bwd_workspace_bytes(4, 16385, 1) == 0


def _fwd(**over):
    a = dict(B=1, T=64, Hk=1, H=2, K=64, V=64, dt=1, q=fake(0), k=fake(1), v=fake(2), g=fake(3), beta=fake(4), cu=None,
             N=0, scale=0.1, h0=None, o=fake(5), ck=fake(6), hT=fake(7), ws=fake(8), wsb=1 << 25)
    a.update(over)
    return gdr._lib().gdr_fwd(*a.values(), None)


@needs_no_gpu
def test_gdr_fwd_rejects_bad_arguments():
    assert _fwd(B=0) == ERR_SHAPE and _fwd(T=0) == ERR_SHAPE and _fwd(Hk=0) == ERR_SHAPE
    assert _fwd(H=3, Hk=2) == ERR_SHAPE and _fwd(K=32) == ERR_SHAPE and _fwd(V=256) == ERR_SHAPE
    assert _fwd(B=2, cu=fake(9), N=2) == ERR_SHAPE                      # packed sequences need B = 1
    assert _fwd(cu=fake(9), N=0) == ERR_SHAPE
    assert _fwd(T=2 ** 31 - 1, H=1024, Hk=1) == ERR_SHAPE
    assert _fwd(dt=2) == ERR_DTYPE
    for n in ("q", "k", "v", "g", "beta"):
        assert _fwd(**{n: None}) == ERR_ARG
    assert _fwd(o=None, ck=None, hT=None) == ERR_ARG
    assert _fwd(q=fake(0) + 8) == ERR_ALIGN and _fwd(hT=fake(7) + 4) == ERR_ALIGN
    assert _fwd(cu=fake(9) + 2, N=1) == ERR_ALIGN
    assert _fwd(o=fake(2)) == ERR_ALIAS and _fwd(hT=fake(5)) == ERR_ALIAS
    assert _fwd(h0=fake(7) + 64) == ERR_ALIAS                           # overlapping, not equal
    assert _fwd(ws=fake(5)) == ERR_ALIAS
    assert _fwd(ws=None) == ERR_WS and _fwd(wsb=100) == ERR_WS


@needs_no_gpu
def test_gdr_bwd_rejects_bad_arguments():
    def c(**over):
        a = dict(B=1, T=64, Hk=1, H=2, K=64, V=64, dt=1, do=fake(0), dhT=None, q=fake(1), k=fake(2), v=fake(3),
                 g=fake(4), beta=fake(5), cu=None, N=0, scale=0.1, ck=fake(6), dq=fake(7), dk=fake(8), dv=fake(9),
                 dg=fake(10), db=fake(11), dh0=fake(12), ws=fake(13), wsb=1 << 25)
        a.update(over)
        return gdr._lib().gdr_bwd(*a.values(), None)

    assert c(K=0) == ERR_SHAPE and c(dt=9) == ERR_DTYPE
    for n in ("do", "ck", "dq", "dk", "dv", "dg", "db"):
        assert c(**{n: None}) == ERR_ARG
    assert c(dq=fake(8)) == ERR_ALIAS and c(dv=fake(0)) == ERR_ALIAS and c(dh0=fake(6)) == ERR_ALIAS
    assert c(dhT=fake(14), dh0=fake(14)) == ERR_ALIAS
    assert c(dg=fake(10) + 2) == ERR_ALIGN and c(dq=fake(7) + 8) == ERR_ALIGN
    assert c(wsb=1000) == ERR_WS


@needs_no_gpu
def test_gdr_step_rejects_bad_arguments():
    def c(**over):
        a = dict(B=2, T=1, Hk=1, H=2, K=64, V=64, dt=1, q=fake(0), k=fake(1), v=fake(2), g=fake(3), beta=fake(4),
                 slots=None, P=2, scale=0.1, s=fake(5), so=fake(6), o=fake(7))
        a.update(over)
        return gdr._lib().gdr_step(*a.values(), None)

    assert c(P=1) == ERR_SHAPE and c(P=0, slots=fake(8)) == ERR_SHAPE and c(T=0) == ERR_SHAPE
    assert c(dt=-1) == ERR_DTYPE
    assert c(s=None) == ERR_ARG and c(so=None) == ERR_ARG and c(o=None) == ERR_ARG
    assert c(so=fake(5) + 64) == ERR_ALIAS and c(o=fake(5)) == ERR_ALIAS and c(slots=fake(7)) == ERR_ALIAS
    assert c(slots=fake(8) + 1) == ERR_ALIGN


@needs_no_gpu
def test_gdr_zero_outside_rejects_bad_arguments():
    def c(T=8, N=1, cu=fake(0), p=fake(1), rb=128, n=1):
        ptrs, rows = (ctypes.c_void_p * 1)(p), (ctypes.c_int64 * 1)(rb)
        return gdr._lib().gdr_zero_outside(T, N, cu, n, ptrs, rows, None)

    assert c(T=0) == ERR_SHAPE and c(N=0) == ERR_SHAPE and c(rb=2) == ERR_SHAPE
    assert c(cu=None) == ERR_ARG and c(p=None) == ERR_ARG and c(n=9) == ERR_ARG and c(n=0) == ERR_ARG
    assert c(p=fake(1) + 2) == ERR_ALIGN


@needs_no_gpu
def test_ln_rejects_bad_arguments():
    lib = lnorm._lib()

    def f(**over):
        a = dict(rows=4, C=64, G=2, xd=0, yd=1, wd=0, x=fake(0), w=fake(1), b=fake(2), eps=1e-5, y=fake(3), m=fake(4),
                 r=fake(5))
        a.update(over)
        return lib.ln_fwd(*a.values(), None)

    def b(**over):
        a = dict(rows=4, C=64, G=2, xd=0, yd=1, wd=0, dy=fake(0), x=fake(1), w=fake(2), m=fake(3), r=fake(4), dx=fake(5),
                 dw=fake(6), db=fake(7), ws=fake(8), wsb=1 << 16)
        a.update(over)
        return lib.ln_bwd(*a.values(), None)

    for c in (f, b):
        assert c(rows=0) == ERR_SHAPE and c(C=63) == ERR_SHAPE and c(G=0) == ERR_SHAPE and c(C=40000, G=1) == ERR_SHAPE
        assert c(xd=1, yd=0) == ERR_DTYPE and c(wd=5) == ERR_DTYPE
        assert c(x=None) == ERR_ARG and c(w=fake(2) + 2) == ERR_ALIGN
    assert f(y=None) == ERR_ARG and f(m=None) == ERR_ARG
    assert f(y=fake(0)) == ERR_ALIAS and f(m=fake(5)) == ERR_ALIAS
    assert b(dw=None) == ERR_ARG and b(dx=None, dw=None, db=None) == ERR_ARG and b(m=None) == ERR_ARG
    assert b(dx=fake(0)) == ERR_ALIAS and b(ws=fake(5)) == ERR_ALIAS
    assert b(ws=None) == ERR_WS and b(wsb=8) == ERR_WS


def toks(B=2, T=5, Hk=2, H=4, K=64, V=128, dtype=BF):
    return [torch.zeros(B, T, Hk, K, dtype=dtype), torch.zeros(B, T, Hk, K, dtype=dtype),
            torch.zeros(B, T, H, V, dtype=dtype), torch.zeros(B, T, H), torch.zeros(B, T, H)]


def _with(x, i, t):
    x = list(x)
    x[i] = t
    return x


def test_binding_checks_gdr_inputs():
    x = toks()
    calls = [lambda *a: L.gdr_fwd(*a), lambda *a: L.gdr_step(*a, torch.zeros(2, 4, 128, 64)),
             lambda *a: L.gdr_bwd(torch.zeros(2, 5, 4, 128, dtype=BF), *a, torch.zeros(1))]
    for f in calls[:2]:
        with pytest.raises(ValueError, match="GPU tensors"):
            f(*x)
    for f in calls:
        with pytest.raises(ValueError, match="k is"):
            f(*_with(x, 1, x[1].float()))
        with pytest.raises(ValueError, match="g is"):
            f(*_with(x, 3, x[3].to(BF)))
        with pytest.raises(ValueError, match="beta is"):
            f(*_with(x, 4, torch.zeros(2, 5, 2)))
        with pytest.raises(ValueError, match="contiguous"):
            f(*_with(x, 0, torch.zeros(2, 2, 5, 64, dtype=BF).transpose(1, 2)))
        with pytest.raises(ValueError, match="multiple of Hk"):
            f(*toks(Hk=3))
        with pytest.raises(ValueError, match="64 or 128"):
            f(*toks(K=32))
        with pytest.raises(TypeError, match="float32 or bfloat16"):
            f(*[t.half() for t in x[:3]], *x[3:])
    with pytest.raises(ValueError, match="ckpt"):
        calls[2](*x)


def test_binding_checks_gdr_states_and_offsets():
    x, one = toks(), toks(B=1)
    with pytest.raises(ValueError, match="h0"):
        L.gdr_fwd(*x, torch.zeros(2, 4, 64, 128))
    with pytest.raises(ValueError, match="B = 1"):
        L.gdr_fwd(*x, cu_seqlens=torch.tensor([0, 5], dtype=torch.int32))
    with pytest.raises(ValueError, match="int32"):
        L.gdr_fwd(*one, cu_seqlens=torch.tensor([0, 5]))
    with pytest.raises(ValueError, match="int32"):
        L.gdr_fwd(*one, cu_seqlens=torch.tensor([5], dtype=torch.int32))
    with pytest.raises(ValueError, match="h0"):
        L.gdr_fwd(*one, torch.zeros(1, 4, 128, 64), cu_seqlens=torch.tensor([0, 2, 5], dtype=torch.int32))
    with pytest.raises(ValueError, match="o is"):
        L.gdr_fwd(*x, o=torch.zeros(2, 5, 4, 128))
    with pytest.raises(ValueError, match="workspace"):
        L.gdr_fwd(*x, workspace=torch.zeros(16, dtype=torch.uint8))
    s = torch.zeros(2, 4, 128, 64)
    with pytest.raises(ValueError, match="1 states for 2 rows"):
        L.gdr_step(*x, s[:1].contiguous())
    with pytest.raises(ValueError, match="slots"):
        L.gdr_step(*x, s, slots=torch.zeros(2, dtype=torch.int64))
    with pytest.raises(ValueError, match="slots"):
        L.gdr_step(*x, s, slots=torch.zeros(3, dtype=torch.int32))
    with pytest.raises(ValueError, match="state is"):
        L.gdr_step(*x, s.to(BF))
    with pytest.raises(ValueError, match="state_out"):
        L.gdr_step(*x, s, state_out=torch.zeros(3, 4, 128, 64))


def test_binding_checks_ln():
    x, w = torch.zeros(4, 64), torch.zeros(64)
    with pytest.raises(ValueError, match="GPU tensors"):
        L.ln_fwd(x, w, w)
    with pytest.raises(ValueError, match="groups"):
        L.ln_fwd(x, groups=3)
    with pytest.raises(ValueError, match="contiguous"):
        L.ln_fwd(torch.zeros(64, 4).t())
    with pytest.raises(TypeError, match="float32 or bfloat16"):
        L.ln_fwd(x.half())
    with pytest.raises(TypeError, match="cannot give"):
        L.ln_fwd(x.to(BF), out_dtype=F32)
    with pytest.raises(ValueError, match="not empty"):
        L.ln_fwd(torch.zeros(0, 64))
    with pytest.raises(ValueError, match="weight"):
        L.ln_fwd(x, w[:32].contiguous())
    with pytest.raises(ValueError, match="one type"):
        L.ln_fwd(x, w, w.to(BF))
    with pytest.raises(ValueError, match="go together"):
        L.ln_fwd(x, mean=torch.zeros(4, 1))
    m = torch.zeros(4, 1)
    with pytest.raises(ValueError, match="dy"):
        L.ln_bwd(x[:2].contiguous(), x, w, m, m)
    with pytest.raises(ValueError, match="rstd"):
        L.ln_bwd(x, x, w, m, torch.zeros(4, 2))
    with pytest.raises(ValueError, match="wanted"):
        L.ln_bwd(x, x, w, m, m, want_dx=False, want_dw=False)


# The kernels' arithmetic on offsets (gdr_device.h, seq_span and slot_chunk).
def _seq_span(cu, n, T):
    a = min(max(cu[n], 0), T)
    b = min(max(cu[n + 1], a), T)
    return a, b - a, a // 64 + n


def _slot_chunk(cu, slot, T):
    lo, hi = 0, len(cu) - 2
    while lo < hi:
        mid = (lo + hi + 1) // 2
        if min(max(cu[mid], 0), T) // 64 + mid <= slot:
            lo = mid
        else:
            hi = mid - 1
    t0, ln, s0 = _seq_span(cu, lo, T)
    c = slot - s0
    return None if c < 0 or c * 64 >= ln else (lo, t0 + 64 * c, min(64, ln - 64 * c))


def test_slots_of_packed_sequences():
    r = random.Random(0)
    for case in range(400):
        T, N = r.randint(1, 700), r.randint(1, 12)
        cu = sorted(r.randint(0, T) for _ in range(N + 1))
        slots = gdr._lib().gdr_slots(1, T, N, 1)
        want = {}
        for n in range(N):
            a, ln, s0 = _seq_span(cu, n, T)
            for c in range(-(-ln // 64)):
                assert s0 + c not in want and 0 <= s0 + c < slots
                want[s0 + c] = (n, a + 64 * c, min(64, ln - 64 * c))
        assert {s: x for s in range(slots) if (x := _slot_chunk(cu, s, T))} == want


def test_bad_offsets_stay_inside():
    r = random.Random(1)
    for case in range(400):
        T, N = r.randint(1, 700), r.randint(1, 12)
        cu = [r.choice([r.randint(-900, 1500), -2 ** 31, 2 ** 31 - 1]) for _ in range(N + 1)]
        slots = gdr._lib().gdr_slots(1, T, N, 1)
        for n in range(N):
            a, ln, s0 = _seq_span(cu, n, T)
            assert 0 <= a and a + ln <= T and 0 <= s0 and s0 + -(-ln // 64) <= slots
        for s in range(slots):
            x = _slot_chunk(cu, s, T)
            if x:
                assert 0 <= x[1] and 1 <= x[2] <= 64 and x[1] + x[2] <= T


@needs_no_gpu
def test_sizes_that_no_launch_takes_are_refused():
    """A launch holds fewer than 2^32 threads."""
    assert _fwd(T=2 ** 23, H=64, Hk=1, B=1) == ERR_SHAPE                # 2^17 chunks of 64 heads
    assert _fwd(B=2 ** 20, T=1, H=2) == ERR_SHAPE                       # sequences times heads
    assert _fwd(T=1, H=2 ** 17, Hk=1) == ERR_SHAPE                      # a chunk's rows past 31 bits
    s = gdr._lib().gdr_step
    assert s(2 ** 20, 1, 1, 4, 64, 64, 1, *map(fake, range(5)), fake(5), 1, 0.1, fake(6), fake(7), fake(8),
             None) == ERR_SHAPE
    ln = lnorm._lib().ln_fwd
    for C, G in ((2 ** 27, 2 ** 17), (2 ** 21, 2 ** 21)):
        assert ln(1, C, G, 0, 0, 0, fake(0), None, None, 1e-5, fake(1), None, None, None) == ERR_SHAPE
    assert gdr._lib().gdr_ckpt_bytes(1, 2 ** 23, 1, 64, 64, 64, 0, 0) == 0


@needs_no_gpu
def test_ln_alignment_goes_by_the_parts():
    """Rows of parts of a multiple of 8 values go by vectors; others value by value."""
    f = lnorm._lib().ln_fwd
    assert f(4, 64, 1, 1, 1, 0, fake(0) + 2, None, None, 1e-5, fake(1), None, None, None) == ERR_ALIGN
    assert f(4, 63, 1, 1, 1, 0, fake(0) + 1, None, None, 1e-5, fake(1), None, None, None) == ERR_ALIGN
    assert f(4, 63, 1, 1, 1, 0, fake(0), fake(2) + 2, None, 1e-5, fake(1), None, None, None) == ERR_ALIGN


def test_workspace_of_a_training_forward():
    """The checkpoints hold T and the gates, so that a forward that leaves them needs the planes of fp32 inputs only."""
    lib = gdr._lib()
    train = [lib.gdr_fwd_train_workspace_bytes(2, 65, 2, 4, 64, 128, dt, 0, 0) for dt in (0, 1)]
    assert train == [2 * 3 * 2 * (2 * 65 * 2 * 64), 256]
    assert train[0] == lib.gdr_fwd_workspace_bytes(2, 65, 2, 4, 64, 128, 0, 0, 0) - 16 * 3392 * 4
    assert lib.gdr_fwd_train_workspace_bytes(2, 65, 3, 4, 64, 128, 0, 0, 0) == 0


@needs_no_gpu
def test_workspace_of_a_training_forward_is_checked():
    assert _fwd(wsb=255) == ERR_WS and _fwd(ck=None, wsb=256) == ERR_WS
    n = gdr._lib().gdr_fwd_train_workspace_bytes(1, 64, 1, 2, 64, 64, 0, 0, 0)
    assert n > 256 and _fwd(dt=0, wsb=n - 1) == ERR_WS
    assert _fwd(ws=fake(6) + 64) == ERR_ALIAS                           # inside ckpt

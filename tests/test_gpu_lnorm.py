"""The layer norm on the GPU against its definition in 64 bits.

Tolerances (rel-L2): the result's rounding (2^-8 for bf16, 2^-24 for fp32), plus fp32
sums over D channels, at most D 2^-24 of their terms' sizes each, through the mean and the
variance (2 D), in the backward two more (4 D), and over the rows for the
weight's gradients.  Where a row lies far from zero the mean takes away |mean| / std
of the digits: the bound grows by that factor."""
import pytest
import torch

import linear_rnn_lm_amd as L
from tests.gdr_util import ref_norm, rel
from tests.gpu_util import note

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
BF, F32 = torch.bfloat16, torch.float32
EPS = 2.0 ** -24


def half_step(dt):
    return 2.0 ** -8 if dt == BF else EPS


def make(rows, C, xd, yd, wd, seed=0):
    gen = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    x = (rn(rows, C) * torch.exp(0.5 * rn(rows, 1)) + 0.3 * rn(1, C)).to(xd)
    return x, (1 + 0.1 * rn(C)).to(wd), (0.1 * rn(C)).to(wd), rn(rows, C).to(yd)


def check(x, w, b, dy, groups, eps=1e-5, grow=1.0):
    D = x.shape[1] // groups
    dev = [None if t is None else t.to(DEV) for t in (x, w, b, dy)]
    y, mean, rstd = L.ln_fwd(dev[0], dev[1], dev[2], groups=groups, eps=eps, out_dtype=dy.dtype)
    dx, dw, db = L.ln_bwd(dev[3], dev[0], dev[1], mean, rstd, groups=groups)
    torch.cuda.synchronize()
    want = ref_norm(x, w, b, groups, eps, dy)
    fwd = grow * (2 * D + 4) * EPS
    tols = {"y": half_step(dy.dtype) + fwd, "dx": half_step(x.dtype) + 2 * fwd, "dweight": (x.shape[0] + 4) * EPS + fwd,
            "dbias": (x.shape[0] + 4) * EPS}
    # dx = rstd (e - s1 - xh s2): each term and their sum are rounded by at most EPS of a term's
    # size, |s1| and |xh s2| being at most e's over the part, so dx is off by a few EPS of
    # rstd e, not of dx itself; for parts of two channels the terms cancel almost wholly
    # (xh is +-1, dx all but 0).
    e = dy.double() * (1.0 if w is None else w.double())
    size = (e.view(x.shape[0], groups, D) * rstd.double().cpu().unsqueeze(-1)).norm().item()
    tols["dx"] = half_step(x.dtype) + 2 * fwd * max(1.0, size / max(want["dx"].norm().item(), 1e-300))
    for n, t in zip(("y", "dx", "dweight", "dbias"), (y, dx, dw, db)):
        assert rel(t, want[n]) <= tols[n], (n, rel(t, want[n]), tols[n])
    return y, mean, rstd, dx, dw, db


TYPES = [(BF, BF, BF), (BF, BF, F32), (F32, F32, F32), (F32, BF, BF)]


@pytest.mark.parametrize("xd,yd,wd", TYPES)
@pytest.mark.parametrize("rows,C,groups", [
    (1, 2, 1), (3, 7, 1), (5, 8, 1), (130, 64, 1), (17, 100, 1), (40, 384, 1), (9, 257, 1), (33, 1000, 1),
    (2, 1025, 1), (6, 2531, 1), (12, 4096, 1), (3, 5000, 1), (2, 8192, 1), (2, 16384, 1), (2, 16383, 1),
    (300, 2048, 32), (35, 384, 6), (7, 96, 3), (4, 130, 2), (11, 24, 3), (2, 12, 4), (9, 1536, 2), (3, 16640, 5)])
def test_shapes(rows, C, groups, xd, yd, wd):
    note(f"ln rows{rows} C{C} G{groups} {xd} {yd} {wd}")
    check(*make(rows, C, xd, yd, wd, seed=C), groups)


@pytest.mark.parametrize("C,groups", [(64, 1), (384, 6), (4096, 1), (333, 1)])
def test_many_rows(C, groups):
    note(f"ln 5000 rows C{C} G{groups}")
    check(*make(5000, C, BF, BF, F32, seed=1), groups)


@pytest.mark.parametrize("D", [1, 24, 64, 384, 520, 768, 1032, 2056, 2048, 6144, 9000, 16])
def test_every_team_shape(D):
    note(f"ln D{D}")
    check(*make(50, 2 * D, F32, F32, F32, seed=D), 2)


def test_no_weights_and_partial_gradients():
    note("ln without weights")
    x, w, b, dy = make(20, 128, F32, F32, F32)
    full = check(x, None, None, dy, 2)
    check(x, w, None, dy, 2)
    args = (dy.to(DEV), x.to(DEV), None, full[1], full[2])
    dx, dw, db = L.ln_bwd(*args, groups=2, want_dw=False)
    assert dw is None and db is None and torch.equal(dx, full[3])
    dx, dw, db = L.ln_bwd(*args, groups=2, want_dx=False)
    assert dx is None and torch.equal(dw, full[4]) and torch.equal(db, full[5])
    y, mean, rstd = L.ln_fwd(x.to(DEV), groups=2, want_stats=False)
    assert mean is None and rstd is None and torch.equal(y, full[0])


def test_constant_far_and_tiny_rows():
    note("ln constant rows, far means, tiny values")
    x, w, b, dy = make(12, 512, F32, F32, F32)
    x[3] = 2.5                                   # no spread: y = bias exactly
    y = L.ln_fwd(x.to(DEV), w.to(DEV), b.to(DEV))[0].cpu()
    assert torch.equal(y[3], b)
    x, w, b, dy = make(12, 512, F32, F32, F32)
    check(x + 1000, w, b, dy, 1, grow=2000)      # |mean| / std is up to about 2000 here
    check(x * 1e-4, w, b, dy, 1, eps=1e-12)
    check(x * 1e15, w, b, dy, 1)


def test_nan_and_inf_stay_in_their_part():
    note("ln NaN")
    x, w, b, dy = make(6, 128, F32, F32, F32)
    clean = check(x, w, b, dy, 2)
    bad = x.clone()
    bad[2, 5], bad[4, 100] = float("nan"), float("inf")
    y, mean, rstd = L.ln_fwd(bad.to(DEV), w.to(DEV), b.to(DEV), groups=2)
    dx = L.ln_bwd(dy.to(DEV), bad.to(DEV), w.to(DEV), mean, rstd, groups=2)[0]
    torch.cuda.synchronize()
    part = torch.zeros(6, 2, dtype=torch.bool, device=DEV)
    part[2, 0] = part[4, 1] = True
    for t, c in ((y, clean[0]), (dx, clean[3])):
        t, c = t.view(6, 2, 64), c.view(6, 2, 64)
        assert torch.isnan(t[part]).all() and torch.equal(t[~part], c[~part])


def test_shapes_of_x_and_repeat():
    note("ln (B, T, C), two runs")
    x, w, b, dy = make(24, 320, BF, BF, BF)
    a = check(x, w, b, dy, 5)
    y, mean, rstd = L.ln_fwd(x.view(2, 3, 4, 320).to(DEV), w.to(DEV), b.to(DEV), groups=5)
    assert torch.equal(y.view(24, 320), a[0]) and mean.shape == (24, 5)
    for s, t in zip(a, check(x, w, b, dy, 5)):
        assert torch.equal(s, t)


def test_graph_and_stream():
    note("ln graph")
    x, w, b, dy = (t.to(DEV) for t in make(700, 384, BF, BF, F32))

    def both():
        y, mean, rstd = L.ln_fwd(x, w, b)
        return [y, *L.ln_bwd(dy, x, w, mean, rstd)]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        first = both()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = both()
    for i in range(4):
        x.mul_(1.5)
        graph.replay()
        got = [t.clone() for t in outs]
        torch.cuda.synchronize()
        want = both()
        torch.cuda.synchronize()
        assert all(torch.equal(a, c) for a, c in zip(got, want)), i
    assert all(torch.isfinite(t).all() for t in first)


def test_autograd_op():
    note("LN autograd")
    x, w, b, dy = make(30, 96, F32, BF, BF)
    leaves = [t.to(DEV).requires_grad_() for t in (x, w, b)]
    y = L.LN.apply(*leaves, 3, 1e-5, BF)
    assert y.dtype == BF
    y.backward(dy.to(DEV))
    want = ref_norm(x, w, b, 3, 1e-5, dy)
    for t, n in zip(leaves, ("dx", "dweight", "dbias")):
        assert t.grad.dtype == t.dtype and rel(t.grad, want[n]) <= half_step(t.dtype) + (4 * 32 + 34) * EPS
    x1 = x.to(DEV).requires_grad_()
    L.LN.apply(x1).sum().backward()
    frozen = L.LN.apply(x.to(DEV), leaves[1])
    assert torch.isfinite(x1.grad).all() and frozen.requires_grad


def test_norm_of_the_recurrences_output():
    """The recurrence's fp32 output through its per-head norm into bf16, as a layer does."""
    from linear_rnn_lm_amd.inputs import make_inputs
    note("wkv7 fwd + ln")
    t = make_inputs(2, 40, 3, BF, seed=3)
    y, _, _ = L.fwd(*[a.to(DEV) for a in t.tensors()])
    w = torch.randn(192, generator=torch.Generator().manual_seed(1))
    z = L.ln_fwd(y.view(2, 40, 192), w.to(DEV), groups=3, eps=64e-5, out_dtype=BF, want_stats=False)[0]
    want = ref_norm(y.view(80, 192).cpu(), w, None, 3, 64e-5)["y"]
    assert z.dtype == BF and rel(z.view(80, 192), want) <= 2.0 ** -8 + 140 * EPS


def test_offsets_past_31_bits():
    """The last rows of a tensor of more than 2^31 values, against the same rows alone."""
    note("ln, long offsets")
    rows, C, n = (1 << 20) + 5, 2056, 7
    gen = torch.Generator().manual_seed(9)
    xs, ds = (torch.randn(n, C, generator=gen).to("cuda", torch.bfloat16) for _ in range(2))
    x, dy = (torch.zeros(rows, C, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    x[-n:], dy[-n:] = xs, ds
    assert x.numel() > 2 ** 31
    y, mean, rstd = L.ln_fwd(x)
    ys, ms, rs = L.ln_fwd(xs)
    dx, dw, db = L.ln_bwd(dy, x, None, mean, rstd)
    dxs, dws, dbs = L.ln_bwd(ds, xs, None, ms, rs)
    torch.cuda.synchronize()
    assert torch.equal(y[-n:], ys) and torch.equal(mean[-n:], ms) and torch.equal(dx[-n:], dxs)
    # n terms of at most 5 max abs(dy) (xh stays below 5 here), summed in another order: n roundings of their
    # total at most, on either side
    for a, b in ((dw, dws), (db, dbs)):
        assert (a - b).abs().max() <= 2 * n * 2.0 ** -24 * n * ds.abs().max().float() * 5


@pytest.mark.parametrize("C,groups", [(333, 1), (36, 3)])
def test_views_at_odd_addresses(C, groups):
    note(f"ln views C{C}")
    x, w, b, dy = make(9, C, BF, BF, BF, seed=4)
    x, w, b, dy = (t.to(DEV) for t in (x, w, b, dy))
    xs, ds = x[1:], dy[1:]
    assert xs.data_ptr() % 16
    got = L.ln_fwd(xs, w, b, groups=groups)
    want = L.ln_fwd(xs.clone(), w, b, groups=groups)
    gg = L.ln_bwd(ds, xs, w, got[1], got[2], groups=groups)
    gw = L.ln_bwd(ds.clone(), xs.clone(), w, want[1], want[2], groups=groups)
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip((*got, *gg), (*want, *gw)))

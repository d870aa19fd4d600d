"""The block norm on the GPU against its definition in 64 bits (tolerances: mix_util)."""
import pytest
import torch

import linear_rnn_lm_amd as L
from tests.gpu_util import note
from tests.mix_util import E, WS, half_step, ref_rn, rel

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
BF, F32 = torch.bfloat16, torch.float32


def make(rows, C, od=F32, iod=F32, rd=F32, wd=F32, seed=0, gate=True, res=True, ws=WS, norm2=True):
    gen = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    p = dict(o=(rn(rows, C) * torch.exp(0.5 * rn(rows, 1)) + 0.3 * rn(1, C)).to(od), gate=rn(rows, C).to(iod) if gate else None,
             res=rn(rows, C).to(rd) if res else None)
    for n in WS:
        w = ((0 if "bias" in n else 1) + 0.3 * rn(C)).to(wd)
        p[n] = w if n in ws and (norm2 or not n.endswith("2")) else None
    p["dr"], p["dh"] = rn(rows, C).to(rd if res else iod), rn(rows, C).to(iod) if norm2 else None
    return p


def check(p, groups=1, norm="layer", norm2="layer", act="silu", eps=1e-5, eps2=1e-5, grow=1.0):
    d = {n: None if t is None else t.to(DEV) for n, t in p.items()}
    ws, kw = {n: d[n] for n in WS}, dict(groups=groups, norm=norm, norm2=norm2, act=act)
    iod = p["dh"].dtype if p["dh"] is not None else p["gate"].dtype if p["gate"] is not None else p["dr"].dtype
    r, h, stats = L.rn_fwd(d["o"], d["gate"], d["res"], **ws, **kw, eps=eps, eps2=eps2, out_dtype=iod)
    names = ("o", "gate", "res", *WS)
    got = dict(zip(names, L.rn_bwd(d["dr"], d["dh"], d["o"], d["gate"], d["res"], stats, **ws, **kw)))
    torch.cuda.synchronize()
    v = {n: None if p[n] is None else p[n].double().requires_grad_() for n in names}
    wr, wh = ref_rn(v, groups, norm, norm2, act, eps, eps2)
    outs, cots = [], []
    for t, g in ((wr, p["dr"]), (wh, p["dh"])):
        if g is not None:
            outs.append(t)
            cots.append(g.double())
    rows, C = p["o"].shape
    fwd = grow * (4 * C + 20) * E
    assert rel(r, wr) <= half_step(r.dtype) + fwd
    if norm2 is None:
        assert h is None
    else:
        assert rel(h, wh) <= half_step(h.dtype) + fwd
    want = dict(zip([n for n in names if v[n] is not None],
                    torch.autograd.grad(outs, [t for t in v.values() if t is not None], cots, allow_unused=True)))
    # A norm's gradient is rstd (e - mean(e) - xh mean(e xh)): each term and the sum are rounded by E of rstd e, not
    # of the result, which is smaller where parts have few channels; `size` is that of e rstd over the
    # result's for o, with e the gradient that reaches norm1's output, formed here in 64 bits.
    u = p["o"].double().unflatten(-1, (groups, -1))
    if norm == "layer":
        u = u - u.mean(-1, keepdim=True)
    rstd = 1 / torch.sqrt((u * u).mean(-1, keepdim=True) + eps)
    g = p["gate"].double() if p["gate"] is not None else None
    e = want["res"] if p["res"] is not None else None
    for n, t in got.items():
        if v[n] is None:
            assert t is None, n
            continue
        w = want[n] if want[n] is not None else torch.zeros_like(v[n])
        tol = half_step(t.dtype) + 2 * fwd + (rows * E if n in WS else 0)
        if n == "o" and e is not None:
            a = 1.0 if g is None else (torch.sigmoid(g) * (g if act == "silu" else 1.0))
            en = e * a * (1.0 if p["scale"] is None else p["scale"].double()) * (1.0 if p["weight"] is None else p["weight"].double())
            size = (en.unflatten(-1, (groups, -1)) * rstd).norm().item()
            tol = half_step(t.dtype) + 2 * fwd * max(1.0, size / max(w.norm().item(), 1e-300))
        assert rel(t, w) <= tol, (n, rel(t, w), tol)
    return r, h, stats, got


TYPES = [(F32, F32, F32, F32), (BF, BF, BF, BF), (F32, BF, BF, F32), (BF, BF, F32, F32), (F32, BF, F32, BF)]


@pytest.mark.parametrize("od,iod,rd,wd", TYPES)
@pytest.mark.parametrize("rows,C,groups", [
    (1, 8, 1), (3, 7, 1), (2, 16, 1), (40, 64, 1), (17, 100, 1), (33, 128, 2), (5, 200, 1), (9, 257, 1), (20, 384, 6),
    (7, 512, 1), (6, 1000, 1), (3, 1024, 8), (4, 1030, 1), (3, 1536, 12), (5, 2048, 32), (2, 2560, 20), (3, 4096, 1),
    (2, 4099, 1), (2, 8192, 1), (2, 8192, 16), (1, 8191, 1)])
def test_shapes(rows, C, groups, od, iod, rd, wd):
    note(f"rn rows{rows} C{C} G{groups} {od} {iod} {rd} {wd}")
    check(make(rows, C, od, iod, rd, wd, seed=C), groups)


@pytest.mark.parametrize("od,iod,rd,wd", [TYPES[0], TYPES[2]])
@pytest.mark.parametrize("rows,C", [(50, 9), (33, 15), (20, 71), (9, 129), (40, 255), (7, 513), (5, 1027), (6, 2051), (3, 4101), (2, 8189)])
def test_last_vector_overlaps(rows, C, od, iod, rd, wd):
    """Rows whose last eight channels begin inside another lane's: each channel counts once, in teams of every size."""
    note(f"rn ragged rows{rows} C{C} {od} {iod}")
    check(make(rows, C, od, iod, rd, wd, seed=C), norm="rms", norm2="rms")
    check(make(rows, C, od, iod, rd, wd, seed=C + 1))


@pytest.mark.parametrize("C", range(1, 9))
def test_few_channels(C):
    """Root-mean-square norms of 1 to 8 channels, and nothing is written beside the rows."""
    note(f"rn C{C}")
    for dtype in (F32, BF):
        rows = 300
        p = make(rows, C, dtype, dtype, dtype, seed=C)
        d = {n: None if t is None else t.to(DEV) for n, t in p.items()}
        bufs = [torch.full((rows * C + 64,), 7.0, dtype=dtype, device=DEV) for _ in range(2)]
        r, h = (b[32:32 + rows * C].view(rows, C) for b in bufs)
        if C == 8:
            assert r.data_ptr() % 16 == 0
        L.rn_fwd(d["o"], d["gate"], d["res"], **{n: d[n] for n in WS}, norm="rms", norm2="rms", r=r, h=h)
        torch.cuda.synchronize()
        wr, wh = ref_rn({n: None if p[n] is None else p[n].double() for n in ("o", "gate", "res", *WS)}, norm="rms", norm2="rms")
        # a root mean square of a row loses nothing by cancellation; r's sum may, of terms of a few times its size
        assert rel(r, wr) <= half_step(dtype) + 64 * E and rel(h, wh) <= half_step(dtype) + 256 * E
        assert all((b[:32] == 7).all() and (b[-32:] == 7).all() for b in bufs)


@pytest.mark.parametrize("norm", ["layer", "rms"])
@pytest.mark.parametrize("norm2", ["layer", "rms", None])
@pytest.mark.parametrize("act", ["silu", "sigmoid", None])
@pytest.mark.parametrize("res", [True, False])
@pytest.mark.parametrize("C,groups", [(192, 3), (77, 1), (2304, 9)])
def test_kinds(norm, norm2, act, res, C, groups):
    note(f"rn {norm} {norm2} {act} res{res} C{C} G{groups}")
    check(make(13, C, seed=2, gate=act is not None, res=res, norm2=norm2 is not None), groups, norm, norm2, act or "silu")


@pytest.mark.parametrize("ws", [(), ("weight",), ("scale", "bias2"), ("bias", "weight2")])
def test_missing_weights(ws):
    note(f"rn weights {ws}")
    check(make(9, 256, BF, BF, BF, F32, seed=3, ws=ws), 4)


@pytest.mark.parametrize("groups", [1, 2, 4, 8])
def test_parts_of_512_to_64(groups):
    note(f"rn parts {groups}")
    check(make(700, 512, BF, BF, F32, F32, seed=4), groups, "rms", "layer", "sigmoid")


def test_many_rows():
    note("rn 5000 rows")
    check(make(5000, 72, F32, F32, F32, F32, seed=5))
    check(make(3001, 384, BF, BF, BF, BF, seed=6), 6)


def test_one_gradient_and_not_wanted():
    note("rn dr or dh alone")
    p = make(11, 128, seed=7)
    check(dict(p, dr=None), 2)
    d = {k: t.to(DEV) for k, t in p.items()}
    ws, kw = {k: d[k] for k in WS}, dict(groups=2, norm2="layer")
    _, _, stats = L.rn_fwd(d["o"], d["gate"], d["res"], **ws, **kw)
    zero = torch.zeros_like(d["o"])
    for dr, dh in ((d["dr"], None), (None, d["dh"])):
        got = L.rn_bwd(dr, dh, d["o"], d["gate"], d["res"], stats, **ws, **kw)
        full = L.rn_bwd(zero if dr is None else dr, zero if dh is None else dh, d["o"], d["gate"], d["res"], stats, **ws, **kw)
        some = L.rn_bwd(dr, dh, d["o"], d["gate"], d["res"], stats, **ws, **kw, want_do=False, want_dres=False, want_dw=False)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, full))
        assert [t is None for t in some] == [True, False] + [True] * 6 and torch.equal(some[1], got[1])


def test_gradients_against_differences():
    """As for the selective scan: 1e-5 covers central differences with steps of 1e-4."""
    note("rn differences")
    p = make(5, 128, seed=8)
    _, _, _, got = check(p, 2, "layer", "rms")
    gen = torch.Generator().manual_seed(3)

    def f(v):
        r, h = ref_rn(v, 2, "layer", "rms")
        return (r * p["dr"]).sum() + (h * p["dh"]).sum()

    names = ("o", "gate", "res", *WS)
    for n in names:
        v = {k: p[k].double() for k in names}
        dirn = torch.randn(v[n].shape, generator=gen, dtype=torch.float64)
        want = ((f({**v, n: v[n] + 1e-4 * dirn}) - f({**v, n: v[n] - 1e-4 * dirn})) / 2e-4).item()
        have = (got[n].double().cpu() * dirn).sum().item()
        size = got[n].double().cpu().norm().item() * dirn.norm().item()
        assert abs(want - have) <= size * (16 * 128 * E + 1e-5), n


def test_constant_far_and_tiny_rows():
    note("rn constant rows, far means, tiny values")
    p = make(12, 512, seed=9)
    p["o"][3] = 2.5                                        # no spread: norm1 gives 0
    d = {n: t.to(DEV) for n, t in p.items()}
    r, _, _ = L.rn_fwd(d["o"], None, d["res"], weight=d["weight"])
    assert torch.equal(r[3], d["res"][3])
    check(dict(p, o=p["o"] * 1e-4), 2, eps=1e-12)
    # At 1e15 the constant row's mean, 2.5e15, is rounded by up to E of itself, 1.5e8, where its spread is 0 and
    # sqrt(eps) 3e-3: what fp32 sums leave of x - mean is that rounding, whatever it is, and norm1 scales it to at most 1.
    # So that row is held to |norm1| <= 1, the others to the tolerance, and the weights' gradients are
    # compared without what the row alone adds to them (its terms are rounded by E of themselves each).
    far = dict(p, o=p["o"] * 1e15)
    rest = [i for i in range(12) if i != 3]
    cut = lambda q, rows: {n: t if n in WS else t[rows].contiguous() for n, t in q.items()}  # noqa: E731
    _, _, _, alone = check(cut(far, rest), 2)
    d = {n: t.to(DEV) for n, t in far.items()}
    ws, kw = {n: d[n] for n in WS}, dict(groups=2, norm2="layer")
    u, _, _ = L.rn_fwd(d["o"], groups=2)
    assert (u[3].abs() <= 1 + 600 * E).all()
    _, _, stats = L.rn_fwd(d["o"], d["gate"], d["res"], **ws, **kw)
    full = L.rn_bwd(d["dr"], d["dh"], d["o"], d["gate"], d["res"], stats, **ws, **kw)
    one = L.rn_bwd(*(d[n][3:4].contiguous() for n in ("dr", "dh", "o", "gate", "res")), stats[3:4].contiguous(), **ws, **kw)
    torch.cuda.synchronize()
    for i, n in enumerate(("o", "gate", "res", *WS)):
        if n in WS:
            assert rel(full[i] - one[i], alone[n]) <= 12 * E * (1 + one[i].norm() / alone[n].norm()).item() + 12 * E
        else:
            assert torch.equal(full[i][rest], alone[n])
    # the mean takes away |mean| / std, up to about 2000, of the digits
    check(dict(make(12, 512, seed=9), o=make(12, 512, seed=9)["o"] + 1000), 2, grow=2000)


def test_gate_slices():
    note("rn gate slice")
    for C, off in ((64, 8), (63, 5)):
        p = make(30, C, BF, BF, BF, F32, seed=10)
        d = {n: t.to(DEV) for n, t in p.items()}
        wide = torch.full((30, C + 24), float("nan"), dtype=BF, device=DEV)
        wide = wide[:, :C + 24] if C % 8 else torch.full((30, 88), float("nan"), dtype=BF, device=DEV)
        wide[:, off:off + C] = d["gate"]
        view = wide[:, off:off + C]
        ws = {n: d[n] for n in WS}
        a = L.rn_fwd(d["o"], d["gate"], d["res"], **ws, norm2="rms")
        b = L.rn_fwd(d["o"], view, d["res"], **ws, norm2="rms")
        ga = L.rn_bwd(d["dr"], d["dh"], d["o"], d["gate"], d["res"], a[2], **ws, norm2="rms")
        gb = L.rn_bwd(d["dr"], d["dh"], d["o"], view, d["res"], b[2], **ws, norm2="rms")
        torch.cuda.synchronize()
        assert all(torch.equal(s, t) for s, t in zip((*a, *ga), (*b, *gb)))


def test_nan_stays_in_its_row():
    note("rn NaN")
    p = make(6, 128, seed=11)
    clean = check(p, 2)
    for n, bad in (("o", float("nan")), ("gate", float("inf")), ("res", float("nan"))):
        q = {k: t.clone() for k, t in p.items()}
        q[n][2, 70] = bad
        d = {k: t.to(DEV) for k, t in q.items()}
        ws, kw = {k: d[k] for k in WS}, dict(groups=2, norm2="layer")
        r, h, stats = L.rn_fwd(d["o"], d["gate"], d["res"], **ws, **kw)
        do, dgate, dres, *_ = L.rn_bwd(d["dr"], d["dh"], d["o"], d["gate"], d["res"], stats, **ws, **kw)
        torch.cuda.synchronize()
        rest = [0, 1, 3, 4, 5]
        for t, c in ((r, clean[0]), (h, clean[1]), (do, clean[3]["o"]), (dgate, clean[3]["gate"]), (dres, clean[3]["res"])):
            assert torch.equal(t[rest], c[rest]), n
        assert torch.equal(r[2, :64], clean[0][2, :64]) and not torch.isfinite(h[2]).any()


@pytest.mark.parametrize("rows,C", [(1, 8), (700, 256), (3000, 2048), (40, 8192), (9, 1030)])
def test_workspace_of_exactly_its_size(rows, C):
    note(f"rn workspace {rows} {C}")
    p = {n: None if t is None else t.to(DEV) for n, t in make(rows, C, seed=3).items()}
    kw = {n: p[n] for n in WS}
    r, h, stats = L.rn_fwd(p["o"], p["gate"], p["res"], norm2="rms", **kw)
    dr, dh = torch.randn_like(r), torch.randn_like(h)
    want = L.rn_bwd(dr, dh, p["o"], p["gate"], p["res"], stats, norm2="rms", **kw)
    need = L.rnorm._lib().rn_bwd_workspace_bytes(rows, C, 1)
    guard = torch.full((need + 512,), 0xa5, dtype=torch.uint8, device=DEV)
    got = L.rn_bwd(dr, dh, p["o"], p["gate"], p["res"], stats, norm2="rms", workspace=guard[256:256 + need], **kw)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert (guard[:256] == 0xa5).all() and (guard[-256:] == 0xa5).all()


def test_graph_and_same_bits():
    note("rn graph")
    p = make(700, 384, BF, BF, F32, F32, seed=12)
    d = {n: t.to(DEV) for n, t in p.items()}
    ws, kw = {n: d[n] for n in WS}, dict(groups=6, norm2="rms")

    def both():
        r, h, stats = L.rn_fwd(d["o"], d["gate"], d["res"], **ws, **kw)
        return [r, h, *L.rn_bwd(d["dr"], d["dh"], d["o"], d["gate"], d["res"], stats, **ws, **kw)]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        both()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = both()
    for i in range(4):
        d["o"].mul_(1.25)
        graph.replay()
        got = [t.clone() for t in outs]
        torch.cuda.synchronize()
        want = both()
        torch.cuda.synchronize()
        assert all(torch.equal(a, c) for a, c in zip(got, want)), i


def test_autograd_op():
    note("RN autograd")
    p = make(30, 192, F32, BF, BF, BF, seed=13)
    names = ("o", "gate", "res", *WS)
    v = {n: p[n].double().requires_grad_() for n in names}
    wr, wh = ref_rn(v, 3, "layer", "rms")
    want = torch.autograd.grad([wr, wh], list(v.values()), [p["dr"].double(), p["dh"].double()])
    leaves = [p[n].to(DEV).requires_grad_() for n in names]
    r, h = L.RN.apply(*leaves, dict(groups=3, norm2="rms", out_dtype=BF))
    assert r.dtype == BF and h.dtype == BF
    torch.autograd.backward([r, h], [p["dr"].to(DEV), p["dh"].to(DEV)])
    for t, w in zip(leaves, want):
        assert t.grad.dtype == t.dtype and rel(t.grad, w) <= half_step(t.dtype) + (8 * 192 + 70) * E
    # without a second norm, a residual and a gate; at an odd address
    o = torch.empty(30 * 192 + 1, device=DEV)[1:].view(30, 192).copy_(p["o"]).requires_grad_()
    assert o.data_ptr() % 16
    r, h = L.RN.apply(o)
    assert h is None
    r.backward(torch.ones_like(r))
    assert torch.isfinite(o.grad).all()


def test_offsets_past_31_bits():
    note("rn, long offsets")
    rows, C, n = (1 << 20) + 5, 2056, 7
    p = {k: None if t is None else t.to(DEV) for k, t in make(n, C, BF, BF, BF, F32, seed=14, gate=False).items()}
    o, res, dr = (torch.zeros(rows, C, dtype=BF, device=DEV) for _ in range(3))
    o[-n:], res[-n:], dr[-n:] = p["o"], p["res"], p["dr"]
    r, h, stats = L.rn_fwd(o, None, res, weight=p["weight"], norm2="rms")
    rs, hs, ss = L.rn_fwd(p["o"], None, p["res"], weight=p["weight"], norm2="rms")
    do = L.rn_bwd(dr, None, o, None, res, stats, weight=p["weight"], norm2="rms", want_dw=False)[0]
    dos = L.rn_bwd(p["dr"], None, p["o"], None, p["res"], ss, weight=p["weight"], norm2="rms", want_dw=False)[0]
    torch.cuda.synchronize()
    assert torch.equal(r[-n:], rs) and torch.equal(h[-n:], hs) and torch.equal(do[-n:], dos)

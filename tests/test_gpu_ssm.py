"""The selective scan on the GPU against its definition in 64 bits (tolerances: mix_util)."""
import pytest
import torch

import linear_rnn_lm_amd as L
from tests.gpu_util import note
from tests.mix_util import E, GRADS, INS, half_step, make_scan, ref_scan, ref_scan_grads, rel, scan_tol

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
BF, F32 = torch.bfloat16, torch.float32


def to_dev(p):
    return {n: None if t is None else t.to(DEV) for n, t in p.items()}


def run(p, softplus=True, cu=None, train=True):
    """y, hT and a dict of gradients of the device tensors p."""
    kw = dict(dt_bias=p["dt_bias"], softplus=softplus,
              cu_seqlens=None if cu is None else torch.tensor(cu, dtype=torch.int32, device=DEV))
    ins = [p[n] for n in ("x", "dt", "A", "b", "c")]
    y, ckpt, hT = L.ssm_fwd(*ins, p["D"], p["z"], p["h0"], want_ckpt=train, **kw)
    if not train:
        return y, hT, None
    return y, hT, dict(zip(GRADS, L.ssm_bwd(p["dy"], *ins, ckpt, p["D"], p["z"], p["dhT"], want_dh0=p["h0"] is not None, **kw)))


def check(p, softplus=True, cu=None, ref_on="cpu"):
    y, hT, got = run(to_dev(p), softplus, cu)
    torch.cuda.synchronize()
    wy, wh, want = ref_scan_grads(p, softplus, cu, ref_on)
    dt, S, T = p["x"].dtype, p["A"].shape[1], p["x"].shape[1]
    tokens = p["x"].shape[0] * T
    steps = T if cu is None else max(b - a for a, b in zip(cu, cu[1:]))
    assert rel(y, wy) <= scan_tol(steps, S, dt)
    assert rel(hT, wh) <= scan_tol(steps, S, F32)
    for n, g in got.items():
        if want[n] is None:
            assert g is None, n
            continue
        many = n in ("dA", "dD", "ddt_bias")
        tol = scan_tol(steps, S, F32 if many or n == "dh0" else dt, tokens if many else p["x"].shape[2] if n in ("db", "dc") else 0,
                       True)
        assert rel(g, want[n]) <= tol, (n, rel(g, want[n]), tol)
    return y, hT, got


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("B,T,C,S,G", [
    (1, 1, 16, 16, 1), (1, 2, 1, 16, 1), (2, 15, 5, 16, 1), (1, 16, 64, 16, 1), (3, 17, 65, 16, 1), (2, 33, 128, 16, 2),
    (1, 100, 200, 16, 1), (1, 70, 192, 16, 3), (1, 1, 64, 32, 1), (2, 31, 40, 32, 1), (1, 48, 320, 32, 5),
    (1, 3, 33, 64, 1), (2, 40, 128, 64, 2), (1, 35, 31, 64, 1)])
def test_shapes(B, T, C, S, G, dtype):
    note(f"ssm B{B} T{T} C{C} S{S} G{G} {dtype}")
    check(make_scan(B, T, C, S, G, dtype, seed=C + T))


@pytest.mark.parametrize("z,D,bias,h0,softplus", [
    (False, True, True, True, True), (True, False, True, False, True), (False, False, False, False, True),
    (True, True, False, True, False)])
def test_optional_inputs(z, D, bias, h0, softplus):
    note(f"ssm z{z} D{D} bias{bias} h0{h0} softplus{softplus}")
    p = make_scan(2, 37, 48, 16, 1, F32, seed=5, z=z, D=D, bias=bias, h0=h0)
    if not softplus:
        p["dt"] = p["dt"].abs() * 0.2
    check(p, softplus)


@pytest.mark.parametrize("dtype,S,G,C", [(F32, 16, 1, 70), (BF, 32, 2, 128), (BF, 64, 1, 40)])
@pytest.mark.parametrize("cu,T", [([0, 5, 5, 38, 39, 90], 90), ([3, 20, 20, 64], 70), ([0, 0, 0], 9), ([0, 32, 48, 64], 64)])
def test_packed(cu, T, dtype, S, G, C):
    note(f"ssm packed {cu} of {T} S{S} G{G} {dtype}")
    y, _, got = check(make_scan(1, T, C, S, G, dtype, seed=T, N=len(cu) - 1), cu=cu)
    for t in (y, got["dx"], got["ddt"], got["dz"], got["db"], got["dc"]):
        assert (t[:, :cu[0]] == 0).all() and (t[:, cu[-1]:] == 0).all()


def test_rows_outside_stay_and_are_not_read():
    note("ssm rows outside")
    cu, T, C, S = [4, 21, 40], 50, 24, 16
    p = to_dev(make_scan(1, T, C, S, 1, F32, seed=1, N=2))
    cut = torch.tensor(cu, dtype=torch.int32, device=DEV)
    want_y, want_h, want = run(p, cu=cu)
    for n in ("x", "dt", "b", "c", "z", "dy"):
        p[n][:, :4], p[n][:, 40:] = float("nan"), float("inf")
    ins, kw = [p[n] for n in ("x", "dt", "A", "b", "c")], dict(dt_bias=p["dt_bias"], cu_seqlens=cut)
    y = torch.full((1, T, C), 7.0, device=DEV)
    out = [torch.full(t.shape, 7.0, device=DEV) for t in list(want.values())[:8]]
    _, ckpt, hT = L.ssm_fwd(*ins, p["D"], p["z"], p["h0"], y=y, **kw)
    dh0 = L.ssm_bwd(p["dy"], *ins, ckpt, p["D"], p["z"], p["dhT"], out=out, **kw)[-1]
    torch.cuda.synchronize()
    assert torch.equal(hT, want_h) and torch.equal(dh0, want["dh0"])
    for t, w in ((y, want_y), *zip(out, list(want.values())[:8])):
        if t.dim() > 2:
            assert (t[:, :4] == 7).all() and (t[:, 40:] == 7).all()
            t, w = t[:, 4:40], w[:, 4:40]
        assert torch.equal(t, w)


def test_longer_sequences():
    note("ssm T600")
    check(make_scan(1, 600, 20, 16, 1, F32, seed=2))
    check(make_scan(2, 300, 36, 64, 1, BF, seed=3))


@pytest.mark.parametrize("B,T,C,S,dtype,what", [
    (1, 70, 12289, 16, BF, "two segments"), (3, 40, 4111, 16, F32, "one segment, not enough waves to fill the chip"),
    (1, 70, 13401, 16, BF, "forward with two states to a lane, backward in two segments"),
    (3, 40, 4501, 16, F32, "the same, one segment"),
    (1, 900, 4096, 16, BF, "15 segments, their sums with four states to a lane"),
    (2, 330, 48, 32, F32, "6 segments of 32 states"), (1, 257, 70, 64, BF, "5 segments of 64 states")])
def test_variants_of_a_launch(B, T, C, S, dtype, what):
    """Sizes at which a launch deals its work out in each of its ways."""
    note(f"ssm B{B} T{T} C{C} S{S} {dtype}: {what}")
    check(make_scan(B, T, C, S, 1, dtype, seed=T), ref_on=DEV)


@pytest.mark.parametrize("S,G,C,dtype", [(16, 1, 40, F32), (32, 2, 128, BF), (64, 1, 33, F32)])
def test_packed_long_and_many(S, G, C, dtype):
    """Sequences of several segments beside empty and short ones; more sequences than a wave has lanes."""
    note(f"ssm packed long S{S}")
    cu = [2, 132, 133, 133, 480, 500]
    check(make_scan(1, 510, C, S, G, dtype, seed=20, N=5), cu=cu, ref_on=DEV)
    gen = torch.Generator().manual_seed(21)
    lens = torch.randint(0, 9, (90,), generator=gen).tolist()
    lens[50] = 200
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    check(make_scan(1, cu[-1] + 3, C, S, G, dtype, seed=22, N=90), cu=cu, ref_on=DEV)


@pytest.mark.parametrize("dtype", [F32, BF])
def test_slices_of_wider_rows(dtype):
    """x, dt, z, b and c as slices at odd places of wider rows give what dense copies give."""
    note(f"ssm slices {dtype}")
    B, T, C, S = 2, 21, 37, 16
    p = to_dev(make_scan(B, T, C, S, 1, dtype, seed=4))
    want_y, want_h, want = run(p)
    wide = {}
    for n, off in (("x", 1), ("dt", 3), ("z", 37), ("b", 5), ("c", 0)):
        t = p[n]
        buf = torch.full((B, T, t[0, 0].numel() + off + 3), float("nan"), dtype=dtype, device=DEV)
        view = buf[..., off:off + t[0, 0].numel()]
        view.copy_(t.flatten(2))
        wide[n] = view.unflatten(-1, t.shape[2:]) if t.dim() > 3 else view
        assert not wide[n].is_contiguous()
    y, h, got = run({**p, **wide})
    torch.cuda.synchronize()
    assert torch.equal(y, want_y) and torch.equal(h, want_h)
    assert all(torch.equal(got[n], want[n]) for n in GRADS)


def test_gradients_against_differences():
    """Along random directions: <gradient, v> against central differences of the 64-bit definition.  With
    step e the difference is off by e^2 / 6 of a third derivative and 2^-52 / e of the value: 1e-6
    at e = 1e-4 for values and derivatives of this size; the kernel's gradient has its own tolerance."""
    note("ssm differences")
    p = make_scan(1, 19, 6, 16, 1, F32, seed=7)
    _, _, got = run(to_dev(p))
    gen = torch.Generator().manual_seed(1)

    def f(v):
        y, hT = ref_scan(v)
        return (y * p["dy"]).sum() + (hT * p["dhT"]).sum()

    for n, g in zip(INS, GRADS):
        v = {k: None if p[k] is None else p[k].double() for k in INS}
        dirn = torch.randn(v[n].shape, generator=gen, dtype=torch.float64)
        e = 1e-4
        up, dn = f({**v, n: v[n] + e * dirn}), f({**v, n: v[n] - e * dirn})
        want, have = ((up - dn) / (2 * e)).item(), (got[g].double().cpu() * dirn).sum().item()
        size = got[g].double().cpu().norm().item() * dirn.norm().item()
        assert abs(want - have) <= size * (scan_tol(19, 16, F32, 19, True) + 1e-5), (n, want, have)


def test_far_steps_and_decays():
    """Steps from 0 to 30, decays that clear a state at once and such that keep it."""
    note("ssm far steps")
    p = make_scan(1, 40, 24, 16, 1, F32, seed=8, bias=False)
    p["dt"][:, ::3] = 30.0
    p["dt"][:, 1::3] = -30.0
    p["dt"][:, 5] = -float("inf")                          # a step of exactly 0: the token passes the state on
    p["A"][:, 0], p["A"][:, 1] = -1e-6, -1e4
    y, hT, _ = run(to_dev(p), train=False)
    wy, wh = ref_scan({n: None if p[n] is None else p[n].double() for n in INS})
    # a step of 30 takes |delta A| to 3e5: e^(delta A) is 0 then, and below 87 its error is |delta A| 9 E
    # of itself, less than the 6 E of what was there that the tolerance counts
    assert rel(y, wy) <= scan_tol(40, 16, F32) and rel(hT, wh) <= scan_tol(40, 16, F32)
    q = dict(p, x=p["x"][:, 5:6], dt=p["dt"][:, 5:6], b=p["b"][:, 5:6], c=p["c"][:, 5:6], z=p["z"][:, 5:6], dy=p["dy"][:, 5:6])
    q = {n: None if t is None else t.contiguous() for n, t in q.items()}
    assert torch.equal(run(to_dev(q), train=False)[1].cpu(), p["h0"])


def test_nan_and_inf_stay_in_their_channel():
    note("ssm NaN")
    p = make_scan(2, 40, 24, 16, 1, F32, seed=9)
    clean_y, clean_h, clean = run(to_dev(p))
    for n, bad in (("x", float("nan")), ("dt", float("nan")), ("z", float("nan")), ("x", float("inf"))):
        q = {k: None if t is None else t.clone() for k, t in p.items()}
        q[n][1, 20, 5] = bad
        y, hT, got = run(to_dev(q))
        torch.cuda.synchronize()
        hit = ~(y == clean_y)
        seen = torch.zeros_like(hit)
        seen[1, 20:, 5] = True
        assert hit[1, 20, 5] and not (hit & ~seen).any(), n
        seen = torch.zeros_like(seen)
        seen[1, :, 5] = True
        for g in ("dx", "ddt", "dz"):
            assert not (~(got[g] == clean[g]) & ~seen).any(), (n, g)
        other = torch.ones(24, dtype=torch.bool, device=DEV)
        other[5] = False
        assert torch.equal(got["dA"][other], clean["dA"][other]) and torch.equal(got["dD"][other], clean["dD"][other])
        assert torch.equal(hT[0], clean_h[0]) and torch.equal(hT[1][other], clean_h[1][other])
        assert torch.equal(got["db"][0], clean["db"][0]) and torch.equal(got["dc"][:, :20][0], clean["dc"][:, :20][0])


def test_graph_replays_with_other_inputs_and_offsets():
    note("ssm graph")
    T, N = 90, 3
    p = to_dev(make_scan(1, T, 70, 16, 1, BF, seed=10, N=N))
    cu = torch.tensor([0, 30, 64, 90], dtype=torch.int32, device=DEV)
    ins, kw = [p[n] for n in ("x", "dt", "A", "b", "c")], dict(dt_bias=p["dt_bias"], cu_seqlens=cu)

    def both():
        y, ckpt, hT = L.ssm_fwd(*ins, p["D"], p["z"], p["h0"], **kw)
        return [y, hT, *L.ssm_bwd(p["dy"], *ins, ckpt, p["D"], p["z"], p["dhT"], **kw)]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        both()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = both()
    for i, offs in enumerate(([0, 30, 64, 90], [0, 0, 90, 90], [5, 6, 40, 77], [0, 88, 89, 90])):
        p["x"].mul_(0.9)
        cu.copy_(torch.tensor(offs, dtype=torch.int32))
        graph.replay()
        got = [t.clone() for t in outs]
        torch.cuda.synchronize()
        want = both()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)), i


def test_same_bits_and_two_streams():
    note("ssm repeat")
    p = to_dev(make_scan(2, 130, 130, 16, 1, BF, seed=11))
    q = to_dev(make_scan(1, 77, 64, 32, 1, BF, seed=12))
    a, b = run(p), run(q)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s1):
        a2 = run(p)
    with torch.cuda.stream(s2):
        b2 = run(q)
    torch.cuda.synchronize()
    for u, v in ((a, a2), (b, b2)):
        assert torch.equal(u[0], v[0]) and torch.equal(u[1], v[1])
        assert all(torch.equal(u[2][n], v[2][n]) for n in GRADS)


def test_state_in_place_and_carried():
    """A prompt in two calls, hT over h0, gives the states and outputs of one call."""
    note("ssm carried state")
    p = to_dev(make_scan(2, 50, 40, 16, 1, F32, seed=13))
    y, hT, _ = run(p, train=False)
    h = p["h0"].clone()
    ys = []
    for s in (slice(0, 16), slice(16, 33), slice(33, 50)):
        part = [p[n][:, s] for n in ("x", "dt", "b", "c", "z")]     # views: rows at one distance only for B = 1
        part = [t.contiguous() for t in part]
        yy, _, hh = L.ssm_fwd(part[0], part[1], p["A"], part[2], part[3], p["D"], part[4], h, dt_bias=p["dt_bias"],
                              want_ckpt=False, hT=h)
        assert hh is h
        ys.append(yy)
    torch.cuda.synchronize()
    assert torch.equal(torch.cat(ys, 1), y) and torch.equal(h, hT)


@pytest.mark.parametrize("cu,B,T", [(None, 2, 300), ([0, 3, 290, 300], 1, 300)])
def test_long_state_in_place(cu, B, T):
    """hT over h0 where a sequence has several segments: each of them starts from h0."""
    note(f"ssm in place T{T} {cu}")
    p = to_dev(make_scan(B, T, 40, 16, 1, F32, seed=23, N=B if cu is None else 3))
    y, hT, _ = run(p, cu=cu, train=False)
    kw = dict(dt_bias=p["dt_bias"], want_ckpt=False, cu_seqlens=None if cu is None else torch.tensor(cu, dtype=torch.int32, device=DEV))
    ins = [p[n] for n in ("x", "dt", "A", "b", "c")]
    for _ in range(3):
        h = p["h0"].clone()
        y2, _, _ = L.ssm_fwd(*ins, p["D"], p["z"], h, hT=h, **kw)
        torch.cuda.synchronize()
        assert torch.equal(y2, y) and torch.equal(h, hT)
    zero = torch.zeros_like(p["h0"])
    y3, _, _ = L.ssm_fwd(*ins, p["D"], p["z"], zero, **kw)
    y4, _, none = L.ssm_fwd(*ins, p["D"], p["z"], want_hT=False, **kw)     # neither of them
    torch.cuda.synchronize()
    assert torch.equal(y3, y4) and none is None


@pytest.mark.parametrize("B,T,C,S,cu", [(2, 300, 40, 16, None), (1, 50, 70, 64, None), (1, 300, 64, 32, [0, 100, 300])])
def test_workspace_of_exactly_its_size(B, T, C, S, cu):
    note(f"ssm workspace B{B} T{T} C{C} S{S} {cu}")
    N = 0 if cu is None else len(cu) - 1
    p = to_dev(make_scan(B, T, C, S, 1, BF, seed=24, N=N or B))
    want = run(p, cu=cu)
    lib = L.ssm._lib()
    dims = (B, T, C, S, 1, N, int(N > 0))
    ins = [p[n] for n in ("x", "dt", "A", "b", "c")]
    kw = dict(dt_bias=p["dt_bias"], cu_seqlens=None if cu is None else torch.tensor(cu, dtype=torch.int32, device=DEV))

    def guarded(n):
        buf = torch.full((n + 512,), 0xa5, dtype=torch.uint8, device=DEV)
        return buf, buf[256:256 + n]

    guards = [guarded(lib.ssm_fwd_workspace_bytes(*dims)), guarded(lib.ssm_bwd_workspace_bytes(*dims)),
              guarded(lib.ssm_ckpt_bytes(*dims))]
    ckpt = guards[2][1].view(F32).view(-1, C, S)
    y, _, hT = L.ssm_fwd(*ins, p["D"], p["z"], p["h0"], workspace=guards[0][1], ckpt=ckpt, **kw)
    got = L.ssm_bwd(p["dy"], *ins, ckpt, p["D"], p["z"], p["dhT"], workspace=guards[1][1], **kw)
    torch.cuda.synchronize()
    assert torch.equal(y, want[0]) and torch.equal(hT, want[1])
    assert all(torch.equal(a, want[2][n]) for n, a in zip(GRADS, got))
    assert all((b[:256] == 0xa5).all() and (b[-256:] == 0xa5).all() for b, _ in guards)


def test_two_graphs_at_once():
    """Two captured training passes, replayed beside each other and with eager work between the replays."""
    note("ssm two graphs")
    ps = [to_dev(make_scan(2, 200, 70, 16, 1, BF, seed=s)) for s in (25, 26)]
    want = [run(p) for p in ps]
    graphs, outs = [], []
    for p in ps:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            outs.append(run(p))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        run(ps[0])
        for o, w in zip(outs, want):
            assert torch.equal(o[0], w[0]) and torch.equal(o[1], w[1])
            assert all(torch.equal(o[2][n], w[2][n]) for n in GRADS)


# ------------------------------------------------------------------ step
@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("B,T,C,S,G", [(1, 1, 1, 16, 1), (3, 1, 65, 16, 1), (2, 4, 100, 32, 1), (5, 1, 128, 64, 2),
                                       (2, 3, 192, 16, 3), (70, 1, 17, 16, 1)])
def test_step(B, T, C, S, G, dtype):
    note(f"ssm step B{B} T{T} C{C} S{S} G{G} {dtype}")
    p = make_scan(B, T, C, S, G, dtype, seed=B + C)
    d = to_dev(p)
    state = d["h0"].clone()
    y = L.ssm_step(d["x"], d["dt"], d["A"], d["b"], d["c"], state, d["D"], d["z"], dt_bias=d["dt_bias"])
    torch.cuda.synchronize()
    wy, wh = ref_scan({n: None if p[n] is None else p[n].double() for n in INS})
    assert rel(y, wy) <= scan_tol(T, S, dtype) and rel(state, wh) <= scan_tol(T, S, F32)


def test_step_slots_padding_and_repeats():
    """Slots in any order, padding (whose inputs are NaN), two rows of one slot, another pool for the results."""
    note("ssm step slots")
    B, T, C, S, P = 7, 2, 40, 16, 9
    p = to_dev(make_scan(B, T, C, S, 1, F32, seed=14))
    pool = torch.randn(P, C, S, generator=torch.Generator().manual_seed(1)).to(DEV)
    slots = torch.tensor([4, -1, 0, 4, 9, 8, 4], dtype=torch.int32, device=DEV)
    for n in ("x", "dt", "b", "c", "z"):
        p[n][1], p[n][4] = float("nan"), float("nan")
    nxt = torch.full_like(pool, 7.0)
    before = pool.clone()
    args = lambda r: [p[n][r].contiguous() for n in ("x", "dt")] + [p["A"]] + [p[n][r].contiguous() for n in ("b", "c")]  # noqa: E731
    y = L.ssm_step(*args(slice(None)), pool, p["D"], p["z"], dt_bias=p["dt_bias"], slots=slots, state_out=nxt)
    torch.cuda.synchronize()
    assert torch.equal(pool, before)
    want = before.clone()
    for r, s in enumerate(slots.tolist()):
        if not 0 <= s < P:
            assert (y[r] == 0).all()
            continue
        st = want[s:s + 1].clone()
        yr = L.ssm_step(*args(slice(r, r + 1)), st, p["D"], p["z"][r:r + 1].contiguous(), dt_bias=p["dt_bias"])
        assert torch.equal(y[r:r + 1], yr), r
        want[s] = st[0]
    used = [0, 4, 8]
    assert torch.equal(nxt[used], want[used])
    assert (nxt[[1, 2, 3, 5, 6, 7]] == 7).all()
    y2 = L.ssm_step(*args(slice(None)), pool, p["D"], p["z"], dt_bias=p["dt_bias"], slots=slots)
    torch.cuda.synchronize()
    assert torch.equal(y2, y) and torch.equal(pool, want)


def test_step_graph_with_other_slots():
    """A captured step, replayed with other slots, padding and repeated slots."""
    note("ssm step graph")
    B, C, S, P = 5, 70, 16, 6
    p = to_dev(make_scan(B, 1, C, S, 1, BF, seed=27))
    pool = torch.randn(P, C, S, generator=torch.Generator().manual_seed(2)).to(DEV)
    slots = torch.arange(B, dtype=torch.int32, device=DEV)
    step = lambda state: L.ssm_step(*[p[n] for n in ("x", "dt", "A", "b", "c")], state, p["D"], p["z"], dt_bias=p["dt_bias"],  # noqa: E731
                                    slots=slots)
    step(pool.clone())
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = step(pool)
    for ids in ([0, 1, 2, 3, 4], [5, 5, 0, 5, -1], [3, 2, 1, 0, 9], [-1] * 5):
        slots.copy_(torch.tensor(ids, dtype=torch.int32))
        other = pool.clone()
        graph.replay()
        torch.cuda.synchronize()
        want = step(other)
        torch.cuda.synchronize()
        assert torch.equal(y, want) and torch.equal(pool, other), ids


def test_steps_continue_a_prompt():
    note("ssm prompt then steps")
    p = make_scan(3, 30, 50, 16, 1, F32, seed=15)
    d = to_dev(p)
    cut = lambda a, b: [d[n][:, a:b].contiguous() for n in ("x", "dt")] + [d["A"]] + [d[n][:, a:b].contiguous() for n in ("b", "c")]  # noqa: E731
    z = lambda a, b: d["z"][:, a:b].contiguous()  # noqa: E731
    y0, _, state = L.ssm_fwd(*cut(0, 24), d["D"], z(0, 24), d["h0"], dt_bias=d["dt_bias"], want_ckpt=False)
    ys = [y0] + [L.ssm_step(*cut(t, t + 1), state, d["D"], z(t, t + 1), dt_bias=d["dt_bias"]) for t in range(24, 30)]
    torch.cuda.synchronize()
    wy, wh = ref_scan({n: None if p[n] is None else p[n].double() for n in INS})
    assert rel(torch.cat(ys, 1), wy) <= scan_tol(30, 16, F32) and rel(state, wh) <= scan_tol(30, 16, F32)


# ------------------------------------------------------------------ autograd
def test_autograd_op():
    note("SSM autograd")
    p = make_scan(2, 21, 128, 16, 2, BF, seed=16)
    _, _, want = ref_scan_grads(p)
    leaves = {n: p[n].to(DEV).requires_grad_() for n in INS}
    order = ("x", "dt", "A", "b", "c", "D", "z", "dt_bias", "h0")
    y, hT = L.SSM.apply(*[leaves[n] for n in order])
    torch.autograd.backward([y, hT], [p["dy"].to(DEV), p["dhT"].to(DEV)])
    for n, g in zip(INS, GRADS):
        assert leaves[n].grad.dtype == p[n].dtype
        assert rel(leaves[n].grad, want[g]) <= scan_tol(21, 16, p[n].dtype, 42 + 128, True), n
    x = p["x"].to(DEV).transpose(0, 1).contiguous().transpose(0, 1).requires_grad_()      # a layout that no call takes
    y2, _ = L.SSM.apply(x, *[leaves[n].detach() for n in order[1:]])
    assert torch.equal(y2, y)
    y2.backward(p["dy"].to(DEV))                           # hT has no gradient: zero
    q = dict(p, dhT=None)
    assert rel(x.grad, ref_scan_grads(q)[2]["dx"]) <= scan_tol(21, 16, BF, 0, True)
    with pytest.raises(RuntimeError):
        g = torch.autograd.grad(L.SSM.apply(x, *[leaves[n] for n in order[1:]])[0].sum(), x, create_graph=True)[0]
        g.sum().backward()


def test_offsets_past_31_bits():
    """The last rows of an x of more than 2^31 values, against the same rows alone: another batch may deal the
    states to other lanes and sum y in another order, so each is within its tolerance of the same value."""
    note("ssm, long offsets")
    B, T, C, S, n = 70, 8192, 4096, 16, 40
    assert B * T * C > 2 ** 31
    p = to_dev(make_scan(1, n, C, S, 1, BF, seed=17, z=False, h0=False))
    big = {k: torch.zeros(B, T, *p[k].shape[2:], dtype=BF, device=DEV) for k in ("x", "dt", "b", "c")}
    for k in big:
        big[k][-1, :n] = p[k][0]
    y, _, hT = L.ssm_fwd(big["x"], big["dt"], p["A"], big["b"], big["c"], p["D"], dt_bias=p["dt_bias"], want_ckpt=False)
    ys, _, _ = L.ssm_fwd(p["x"], p["dt"], p["A"], p["b"], p["c"], p["D"], dt_bias=p["dt_bias"], want_ckpt=False)
    torch.cuda.synchronize()
    assert rel(y[-1, :n], ys[0]) <= 2 * scan_tol(n, S, BF) and (y[0] == 0).all()

"""The short convolution on the GPU against its definition in 64 bits (tolerances: mix_util)."""
import pytest
import torch

import linear_rnn_lm_amd as L
from tests.gpu_util import note
from tests.mix_util import conv_tol, make_conv, ref_conv, ref_conv_grads, rel

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
BF, F32 = torch.bfloat16, torch.float32


def to_dev(p):
    return {n: None if t is None else t.to(DEV) for n, t in p.items()}


def run(p, silu=True, cu=None):
    cu = None if cu is None else torch.tensor(cu, dtype=torch.int32, device=DEV)
    y, hT = L.conv_fwd(p["x"], p["weight"], p["bias"], p["h0"], silu=silu, cu_seqlens=cu)
    got = L.conv_bwd(p["dy"], p["x"], p["weight"], p["bias"], p["h0"], p["dhT"], silu=silu, cu_seqlens=cu)
    return y, hT, dict(zip(("dx", "dweight", "dbias", "dh0"), got))


def check(p, silu=True, cu=None):
    y, hT, got = run(to_dev(p), silu, cu)
    torch.cuda.synchronize()
    wy, wh, want = ref_conv_grads(p, silu, cu)
    dt, W, tokens = p["x"].dtype, p["weight"].shape[1], p["x"].shape[0] * p["x"].shape[1]
    assert rel(y, wy) <= conv_tol(W, dt)
    assert torch.equal(hT.cpu().double(), wh)
    for n, w in want.items():
        many = n in ("dweight", "dbias")
        tol = conv_tol(W, F32 if many else dt, tokens if many else 0, True)
        assert rel(got[n], w) <= tol, (n, rel(got[n], w), tol)
    return y, hT, got


@pytest.mark.parametrize("dtype,wdtype", [(F32, F32), (BF, F32), (BF, BF), (F32, BF)])
@pytest.mark.parametrize("B,T,C,W", [(1, 1, 1, 2), (1, 1, 8, 4), (2, 2, 16, 4), (1, 3, 5, 4), (3, 16, 64, 3), (2, 17, 40, 4),
                                     (1, 100, 9, 2), (2, 33, 264, 4), (1, 50, 100, 4), (1, 259, 24, 3)])
def test_shapes(B, T, C, W, dtype, wdtype):
    note(f"conv B{B} T{T} C{C} W{W} {dtype} {wdtype}")
    check(make_conv(B, T, C, W, dtype, seed=T + C, wdtype=wdtype))


@pytest.mark.parametrize("bias,h0,silu", [(False, True, True), (True, False, True), (True, True, False), (False, False, False)])
def test_optional_inputs(bias, h0, silu):
    note(f"conv bias{bias} h0{h0} silu{silu}")
    check(make_conv(2, 37, 48, 4, F32, seed=3, bias=bias, h0=h0), silu)
    check(make_conv(2, 2, 48, 4, F32, seed=4, bias=bias, h0=h0), silu)


@pytest.mark.parametrize("C", [24, 25])
@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("cu,T", [([0, 5, 5, 38, 39, 90], 90), ([3, 4, 6, 9, 9, 41], 50), ([0, 0, 0], 9), ([0, 16, 32, 64], 64)])
def test_packed(cu, T, W, C):
    note(f"conv packed {cu} of {T} W{W} C{C}")
    for dtype in (F32, BF):
        y, _, got = check(make_conv(1, T, C, W, dtype, seed=T, N=len(cu) - 1), cu=cu)
        for t in (y, got["dx"]):
            assert (t[:, :cu[0]] == 0).all() and (t[:, cu[-1]:] == 0).all()


def test_rows_outside_stay_and_are_not_read():
    note("conv rows outside")
    cu, T, C = [4, 21, 40], 50, 24
    p = to_dev(make_conv(1, T, C, 4, BF, seed=1, N=2))
    want = run(p, cu=cu)
    for n in ("x", "dy"):
        p[n][:, :4], p[n][:, 40:] = float("nan"), float("inf")
    cut = torch.tensor(cu, dtype=torch.int32, device=DEV)
    y, dx = (torch.full((1, T, C), 7.0, dtype=BF, device=DEV) for _ in range(2))
    dw, db = torch.empty(C, 4, device=DEV), torch.empty(C, device=DEV)
    _, hT = L.conv_fwd(p["x"], p["weight"], p["bias"], p["h0"], cu_seqlens=cut, y=y)
    *_, dh0 = L.conv_bwd(p["dy"], p["x"], p["weight"], p["bias"], p["h0"], p["dhT"], cu_seqlens=cut, out=(dx, dw, db))
    torch.cuda.synchronize()
    for t, w in ((y, want[0]), (dx, want[2]["dx"])):
        assert (t[:, :4] == 7).all() and (t[:, 40:] == 7).all() and torch.equal(t[:, 4:40], w[:, 4:40])
    assert torch.equal(hT, want[1]) and torch.equal(dh0, want[2]["dh0"])
    assert torch.equal(dw, want[2]["dweight"]) and torch.equal(db, want[2]["dbias"])


@pytest.mark.parametrize("C,off,dtype", [(32, 8, BF), (32, 3, BF), (20, 4, F32), (21, 1, F32)])
def test_slices_of_wider_rows(C, off, dtype):
    note(f"conv slice C{C} off{off} {dtype}")
    p = to_dev(make_conv(2, 40, C, 4, dtype, seed=5))
    want = run(p)
    buf = torch.full((2, 40, C + 32), float("nan"), dtype=dtype, device=DEV)
    buf[..., off:off + C] = p["x"]
    got = run({**p, "x": buf[..., off:off + C]})
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    # by values and by vectors the sums over runs are the same sums
    assert all(torch.equal(got[2][n], want[2][n]) for n in want[2])


def test_weights_at_any_address_and_workspace_of_its_size():
    note("conv odd weights, exact workspace")
    B, T, C, W = 2, 300, 64, 4
    for wdtype in (F32, BF):
        p = to_dev(make_conv(B, T, C, W, BF, seed=7, wdtype=wdtype))
        want = run(p)
        buf = torch.empty(C * W + 1, dtype=wdtype, device=DEV)
        buf[1:] = p["weight"].flatten()
        got = run({**p, "weight": buf[1:].view(C, W)})
        need = L.conv._lib().conv_bwd_workspace_bytes(B, T, C, W, 0, 0)
        guard = torch.full((need + 512,), 0xa5, dtype=torch.uint8, device=DEV)
        tight = L.conv_bwd(p["dy"], p["x"], p["weight"], p["bias"], p["h0"], p["dhT"], workspace=guard[256:256 + need])
        torch.cuda.synchronize()
        assert torch.equal(got[0], want[0]) and all(torch.equal(got[2][n], want[2][n]) for n in want[2])
        assert all(torch.equal(a, b) for a, b in zip(tight, want[2].values()))
        assert (guard[:256] == 0xa5).all() and (guard[-256:] == 0xa5).all()


def test_nan_and_inf_reach_their_window_only():
    """A value that is no number in one input or gradient: only the tokens whose windows hold it see it,
    and never another channel, row or sequence."""
    note("conv NaN")
    p = make_conv(2, 40, 24, 4, F32, seed=8)
    clean = run(to_dev(p))
    for n, t, bad in (("x", 20, float("nan")), ("x", 39, float("inf")), ("dy", 20, float("nan")), ("dhT", 2, float("nan"))):
        q = {k: None if v is None else v.clone() for k, v in p.items()}
        q[n][1, t, 5] = bad
        y, hT, got = run(to_dev(q))
        torch.cuda.synchronize()
        first = 0 if n == "dhT" else t
        seen = torch.zeros(2, 40, 24, dtype=torch.bool, device=DEV)
        seen[1, first:first + 4, 5] = n == "x"
        assert not (~(y == clean[0]) & ~seen).any(), n
        seen[1, 37 + t if n == "dhT" else max(t - 3, 0):, 5] = True
        seen[1, (t if n == "dy" else 39 if n == "dhT" else t + 3) + 1:, 5] = False
        assert not (~(got["dx"] == clean[2]["dx"]) & ~seen).any(), n
        other = torch.arange(24, device=DEV) != 5
        assert torch.equal(got["dweight"][other], clean[2]["dweight"][other])
        assert torch.equal(got["dh0"][0], clean[2]["dh0"][0]) and torch.equal(hT[0], clean[1][0])


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("B,T,C,W", [(1, 9001, 1003, 4), (2, 4100, 1024, 3), (1, 33000, 261, 2)])
def test_many_tokens_by_vectors(B, T, C, W, dtype):
    """Enough work for vectors of channels: multiples of them, and rows whose last vector overlaps the one before.  The first
    and last tokens, and every sum, against the definition on the GPU."""
    note(f"conv vectors B{B} T{T} C{C} W{W} {dtype}")
    p = make_conv(B, T, C, W, dtype, seed=9)
    y, hT, got = run(to_dev(p))
    torch.cuda.synchronize()
    wy, wh, want = ref_conv_grads(to_dev(p))
    assert rel(y, wy) <= conv_tol(W, dtype) and torch.equal(hT.double(), wh)
    for n, w in want.items():
        many = n in ("dweight", "dbias")
        assert rel(got[n], w) <= conv_tol(W, F32 if many else dtype, B * T if many else 0, True), n
        assert rel(got[n][..., -9:] if n in ("dx", "dh0") else got[n][-9:], w[..., -9:] if n in ("dx", "dh0") else w[-9:]) <= \
            conv_tol(W, F32 if many else dtype, B * T if many else 0, True), n


@pytest.mark.parametrize("C,W,dtype", [(1003, 4, BF), (1024, 3, F32), (1000, 2, BF)])
def test_packed_by_vectors(C, W, dtype):
    """Many sequences, empty, of one token and long, in a row long enough for vectors of channels."""
    note(f"conv packed vectors C{C} W{W} {dtype}")
    gen = torch.Generator().manual_seed(10)
    cu = [3]
    for n in [0, 1, 2, 3, 700, 0, 31, 32, 33, 9] + torch.randint(0, 900, (20,), generator=gen).tolist():
        cu.append(cu[-1] + n)
    T = max(cu[-1] + 5, 9000)
    p = make_conv(1, T, C, W, dtype, seed=11, N=len(cu) - 1)
    y, hT, got = run(to_dev(p), cu=cu)
    torch.cuda.synchronize()
    wy, wh, want = ref_conv_grads(to_dev(p), cu=cu)
    assert rel(y, wy) <= conv_tol(W, dtype) and torch.equal(hT.double(), wh)
    for n, w in want.items():
        many = n in ("dweight", "dbias")
        assert rel(got[n], w) <= conv_tol(W, F32 if many else dtype, T if many else 0, True), n


@pytest.mark.parametrize("C", [9, 12, 37, 1029])
def test_step_in_place_with_overlapping_vectors(C):
    """Channels that two threads work on are written by one of them: many rows, several tokens, states in place."""
    note(f"conv step in place C{C}")
    for dtype in (F32, BF):
        p = to_dev(make_conv(60, 3, C, 4, dtype, seed=C))
        wy, wh = L.conv_fwd(p["x"], p["weight"], p["bias"], p["h0"])
        state = p["h0"].clone()
        y = L.conv_step(p["x"], p["weight"], p["bias"], state)
        torch.cuda.synchronize()
        assert torch.equal(y, wy) and torch.equal(state, wh)


def test_long_runs_and_same_bits():
    """Enough tokens for longer runs, against the first row alone in shorter ones."""
    note("conv long")
    p = to_dev(make_conv(4, 9001, 1024, 4, BF, seed=6))
    a, b = run(p), run(p)
    torch.cuda.synchronize()
    assert torch.equal(a[0], b[0]) and all(torch.equal(a[2][n], b[2][n]) for n in a[2])
    few = {n: t if n in ("weight", "bias") else t[:1].contiguous() for n, t in p.items()}
    c = run(few)
    assert torch.equal(c[0], a[0][:1]) and torch.equal(c[2]["dx"], a[2]["dx"][:1]) and torch.equal(c[1], a[1][:1])
    wy, _, want = ref_conv_grads({n: None if t is None else t.cpu() for n, t in few.items()})
    assert rel(c[0], wy) <= conv_tol(4, BF)
    assert rel(c[2]["dweight"], want["dweight"]) <= conv_tol(4, F32, 9001, True)


def test_gradients_against_differences():
    """As for the selective scan: 1e-5 covers central differences with steps of 1e-4."""
    note("conv differences")
    p = make_conv(1, 11, 6, 4, F32, seed=7)
    _, _, got = run(to_dev(p))
    gen = torch.Generator().manual_seed(2)

    def f(v):
        y, hT = ref_conv(v)
        return (y * p["dy"]).sum() + (hT * p["dhT"]).sum()

    for n, g in (("x", "dx"), ("weight", "dweight"), ("bias", "dbias"), ("h0", "dh0")):
        v = {k: p[k].double() for k in ("x", "weight", "bias", "h0")}
        dirn = torch.randn(v[n].shape, generator=gen, dtype=torch.float64)
        up, dn = f({**v, n: v[n] + 1e-4 * dirn}), f({**v, n: v[n] - 1e-4 * dirn})
        want, have = ((up - dn) / 2e-4).item(), (got[g].double().cpu() * dirn).sum().item()
        size = got[g].double().cpu().norm().item() * dirn.norm().item()
        assert abs(want - have) <= size * (conv_tol(4, F32, 11, True) + 1e-5), n


def test_nan_stays_with_its_channel_and_readers():
    note("conv NaN")
    p = make_conv(1, 40, 16, 4, F32, seed=8)
    a = run(to_dev(p))
    p["x"][0, 20, 5] = float("nan")
    b = run(to_dev(p))
    torch.cuda.synchronize()
    hit = torch.zeros(40, 16, dtype=torch.bool, device=DEV)
    hit[20:24, 5] = True
    assert torch.equal(~(a[0][0] == b[0][0]), hit)
    hit[17:24, 5] = True                                   # the tokens whose gradients pass the four readers
    assert torch.equal(~(a[2]["dx"][0] == b[2]["dx"][0]), hit)


def test_graph_and_offsets():
    note("conv graph")
    p = to_dev(make_conv(1, 90, 40, 4, BF, seed=9, N=3))
    cu = torch.tensor([0, 30, 64, 90], dtype=torch.int32, device=DEV)

    def both():
        y, hT = L.conv_fwd(p["x"], p["weight"], p["bias"], p["h0"], cu_seqlens=cu)
        return [y, hT, *L.conv_bwd(p["dy"], p["x"], p["weight"], p["bias"], p["h0"], p["dhT"], cu_seqlens=cu)]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        both()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = both()
    for i, offs in enumerate(([0, 30, 64, 90], [0, 0, 90, 90], [5, 6, 40, 77])):
        p["x"].mul_(0.9)
        cu.copy_(torch.tensor(offs, dtype=torch.int32))
        graph.replay()
        got = [t.clone() for t in outs]
        torch.cuda.synchronize()
        want = both()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)), i


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("B,T,C,W", [(1, 1, 1, 2), (3, 1, 40, 4), (2, 5, 24, 3), (5, 2, 4100, 4), (70, 1, 17, 4)])
def test_step(B, T, C, W, dtype):
    note(f"conv step B{B} T{T} C{C} W{W} {dtype}")
    p = make_conv(B, T, C, W, dtype, seed=B)
    d = to_dev(p)
    state = d["h0"].clone()
    y = L.conv_step(d["x"], d["weight"], d["bias"], state)
    torch.cuda.synchronize()
    wy, wh = ref_conv({n: None if p[n] is None else p[n].double() for n in ("x", "weight", "bias", "h0")})
    assert rel(y, wy) <= conv_tol(W, dtype) and torch.equal(state.cpu().double(), wh)


def test_step_slots_padding_and_repeats():
    note("conv step slots")
    B, T, C, P = 7, 2, 40, 9
    p = to_dev(make_conv(B, T, C, 4, BF, seed=10))
    pool = torch.randn(P, 3, C, generator=torch.Generator().manual_seed(1)).to(DEV, BF)
    slots = torch.tensor([4, -1, 0, 4, 9, 8, 4], dtype=torch.int32, device=DEV)
    p["x"][1], p["x"][4] = float("nan"), float("nan")
    nxt, before = torch.full_like(pool, 7.0), pool.clone()
    y = L.conv_step(p["x"], p["weight"], p["bias"], pool, slots=slots, state_out=nxt)
    torch.cuda.synchronize()
    assert torch.equal(pool, before)
    want = before.clone()
    for r, s in enumerate(slots.tolist()):
        if not 0 <= s < P:
            assert (y[r] == 0).all()
            continue
        st = want[s:s + 1].clone()
        assert torch.equal(y[r:r + 1], L.conv_step(p["x"][r:r + 1].contiguous(), p["weight"], p["bias"], st)), r
        want[s] = st[0]
    assert torch.equal(nxt[[0, 4, 8]], want[[0, 4, 8]]) and (nxt[[1, 2, 3, 5, 6, 7]] == 7).all()
    y2 = L.conv_step(p["x"], p["weight"], p["bias"], pool, slots=slots)
    torch.cuda.synchronize()
    assert torch.equal(y2, y) and torch.equal(pool, want)


def test_autograd_op():
    note("CONV autograd")
    p = make_conv(2, 21, 24, 4, BF, seed=11)
    _, _, want = ref_conv_grads(p)
    leaves = {n: p[n].to(DEV).requires_grad_() for n in ("x", "weight", "bias", "h0")}
    y, hT = L.CONV.apply(*leaves.values())
    torch.autograd.backward([y, hT], [p["dy"].to(DEV), p["dhT"].to(DEV)])
    for n, g in (("x", "dx"), ("weight", "dweight"), ("bias", "dbias"), ("h0", "dh0")):
        assert leaves[n].grad.dtype == p[n].dtype
        assert rel(leaves[n].grad, want[g]) <= conv_tol(4, p[n].dtype, 42, True), n
    x = p["x"].to(DEV).transpose(0, 1).contiguous().transpose(0, 1).requires_grad_()
    y2, _ = L.CONV.apply(x, *[leaves[n].detach() for n in ("weight", "bias", "h0")])
    assert torch.equal(y2, y)
    y2.backward(p["dy"].to(DEV))
    assert rel(x.grad, ref_conv_grads(dict(p, dhT=None))[2]["dx"]) <= conv_tol(4, BF, 0, True)


def test_offsets_past_31_bits():
    note("conv, long offsets")
    B, T, C, n = 70, 8192, 4096, 40
    p = to_dev(make_conv(1, n, C, 4, BF, seed=12, h0=False))
    x = torch.zeros(B, T, C, dtype=BF, device=DEV)
    x[-1, -n:] = p["x"][0]
    y, hT = L.conv_fwd(x, p["weight"], None)
    ys, hs = L.conv_fwd(p["x"], p["weight"], None)
    torch.cuda.synchronize()
    assert torch.equal(y[-1, -n:], ys[0]) and torch.equal(hT[-1], hs[0]) and (y[0] == 0).all()

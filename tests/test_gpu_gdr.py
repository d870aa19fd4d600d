"""The gated delta rule on the GPU against its definition in 64 bits."""
import pytest
import torch

import linear_rnn_lm_amd as L
from linear_rnn_lm_amd import gdr
from tests.gdr_util import make, ref_norm, reference, rel, tol_bwd, tol_fwd
from tests.gpu_util import note

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
BF, F32 = torch.bfloat16, torch.float32
GRADS = ("dq", "dk", "dv", "dg", "dbeta", "dh0")


def dev(*xs):
    return [None if x is None else x.to(DEV) for x in xs]


def cu_of(cu):
    return None if cu is None else torch.tensor(cu, dtype=torch.int32, device=DEV)


def check_all(got, want, K, V, dtype):
    for n, x in got.items():
        low = x.dtype == BF
        tol = (tol_bwd(K, V, BF if low else F32) if n in GRADS else tol_fwd(K, BF if low else F32))
        e = rel(x, want[n])
        assert e <= tol, f"{n}: {e:.3e} over {tol:.3e}"


def run(x, cu=None, scale=None, **kw):
    q, k, v, g, beta, h0, do, dhT = dev(*x)
    c = cu_of(cu)
    o, ck, hT = L.gdr_fwd(q, k, v, g, beta, h0, cu_seqlens=c, scale=scale, **kw)
    out = L.gdr_bwd(do, q, k, v, g, beta, ck, dhT, cu_seqlens=c, scale=scale)
    torch.cuda.synchronize()
    return {"o": o, "hT": hT, **dict(zip(GRADS, out))}


HEADS = [(64, 64), (64, 128), (128, 64), (128, 128)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("K,V", HEADS)
@pytest.mark.parametrize("B,T,Hk,H,h0", [(1, 1, 1, 1, True), (2, 63, 1, 2, False), (1, 64, 2, 2, True),
                                         (2, 65, 1, 3, True), (1, 200, 3, 6, True), (3, 129, 2, 2, False)])
def test_dense(B, T, Hk, H, h0, K, V, dtype):
    note(f"gdr dense B{B} T{T} Hk{Hk} H{H} K{K} V{V} {dtype}")
    x = make(B, T, Hk, H, K, V, dtype, seed=T, h0=h0)
    check_all(run(x), reference(*x), K, V, dtype)


PACKED = [([0, 70], 70), ([0, 1, 1, 65, 193], 193), ([0, 0, 64, 64, 128, 130, 130], 130), ([3, 67, 140], 150),
          ([5, 5], 9), ([0, 1, 2, 3, 4, 5, 6, 7], 8), ([64, 128, 129], 200)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("K,V", [(64, 64), (128, 128)])
@pytest.mark.parametrize("cu,T", PACKED)
def test_packed(cu, T, K, V, dtype):
    note(f"gdr packed {cu} T{T} K{K} V{V} {dtype}")
    x = make(1, T, 1, 2, K, V, dtype, seed=len(cu), N=len(cu) - 1)
    check_all(run(x, cu), reference(*x, cu=cu), K, V, dtype)


@pytest.mark.parametrize("B,Hk,H,V", [(2, 2, 2, 64), (33, 1, 4, 64), (40, 4, 8, 128), (70, 2, 8, 64)])
def test_head_counts(B, Hk, H, V):
    """From a few heads to more than there are compute units: every launch shape of the scans."""
    note(f"gdr heads B{B} Hk{Hk} H{H} V{V}")
    for K in (64, 128):
        x = make(B, 70, Hk, H, K, V, BF, seed=B)
        check_all(run(x), reference(*x), K, V, BF)


def test_scale_and_long():
    note("gdr scale, 700 tokens")
    x = make(1, 700, 1, 1, 64, 64, F32, seed=4)
    check_all(run(x, scale=0.7), reference(*x, scale=0.7), 64, 64, F32)


@pytest.mark.parametrize("kind", ["g_zero", "g_inf", "g_large", "beta_zero", "beta_one_same_keys", "beta_small"])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_edges(kind, dtype):
    note(f"gdr edge {kind} {dtype}")
    q, k, v, g, beta, h0, do, dhT = make(1, 150, 1, 2, 64, 64, dtype, seed=9)
    if kind == "g_zero":
        g = torch.zeros_like(g)
    elif kind == "g_inf":          # the state is cleared before tokens 0, 40 and 64 .. 66
        g[:, [0, 40, 64, 65, 66]] = -float("inf")
    elif kind == "g_large":
        g = -30 * torch.rand(g.shape, generator=torch.Generator().manual_seed(1))
    elif kind == "beta_zero":
        beta[:, 20:90] = 0
    elif kind == "beta_small":
        beta = 1e-6 * beta
    else:                          # (I + A) as far from I as it gets
        beta, g = torch.ones_like(beta), torch.zeros_like(g)
        k = k[:, :1].expand_as(k).contiguous()
    x = (q, k, v, g, beta, h0, do, dhT)
    want = reference(q, k, v, g.clamp(min=-1e4), beta, h0, do, dhT)
    got = run(x)
    # |k| is 1 up to its rounding: with one key throughout, a token's error along k is
    # replaced, not added to, so the tolerances hold as they are.  dg under decays of e^-30
    # is a difference of row sums that all but cancel: it is held to the size of those
    # sums (dg's own plus q dq and k dk).
    for n, t in got.items():
        tol = tol_bwd(64, 64, t.dtype) if n in GRADS else tol_fwd(64, t.dtype)
        d = (t.double().cpu() - want[n]).norm().item()
        size = want[n].norm().item()
        if n == "dg":
            rows = (q.double() * want["dq"]).sum(-1).norm() + (k.double() * want["dk"]).sum(-1).norm()
            size += rows.item()
        assert torch.isfinite(t).all() and d <= tol * size, f"{n}: {d / size:.3e} over {tol:.3e}"


def test_nan_stays_in_its_sequence():
    note("gdr NaN in one packed sequence")
    cu, T = [0, 70, 130, 200], 200
    x = list(make(1, T, 1, 2, 64, 64, BF, seed=2, N=3))
    clean = run(x, cu)
    x[2] = x[2].clone()
    x[2][0, 100] = float("nan")
    x[0] = x[0].clone()
    x[0][0, 129] = float("inf")    # the last token of the sequence, beside the next one's first
    got = run(x, cu)
    for n in ("o", "dq", "dk", "dv", "dg", "dbeta"):
        for a, b in ((0, 70), (130, 200)):
            assert torch.equal(got[n][0, a:b], clean[n][0, a:b]), n
    for n in ("hT", "dh0"):
        for s in (0, 2):
            assert torch.equal(got[n][s], clean[n][s]), n
    assert torch.isnan(got["o"][0, 100]).all()   # its chunk's other tokens are unspecified


def test_rows_outside_the_sequences():
    note("gdr rows outside")
    cu, T = [10, 80], 100
    q, k, v, g, beta, h0, do, dhT = dev(*make(1, T, 1, 2, 64, 64, BF, seed=3, N=1))
    c = cu_of(cu)
    o = torch.full_like(v, 7.0)
    _, ck, _ = L.gdr_fwd(q, k, v, g, beta, h0, cu_seqlens=c, o=o)
    out = [torch.full_like(t, 7.0) for t in (q, k, v, g, beta)]
    L.gdr_bwd(do, q, k, v, g, beta, ck, dhT, cu_seqlens=c, out=out)
    fresh = L.gdr_fwd(q, k, v, g, beta, h0, cu_seqlens=c)[0]
    fresh_g = L.gdr_bwd(do, q, k, v, g, beta, ck, dhT, cu_seqlens=c)[:5]
    torch.cuda.synchronize()
    for kept, new in zip([o, *out], [fresh, *fresh_g]):
        assert torch.equal(kept[:, 10:80], new[:, 10:80])
        for a, b in ((0, 10), (80, T)):
            assert (kept[:, a:b] == 7).all() and (new[:, a:b] == 0).all()


def test_bad_offsets_only_give_bad_results():
    """Offsets out of range or decreasing: clamped, nothing outside the tensors is touched
    (the arithmetic is checked on the CPU in test_gdr_checks)."""
    note("gdr bad offsets")
    T = 130
    q, k, v, g, beta, h0, do, dhT = dev(*make(1, T, 1, 2, 64, 64, BF, seed=3, N=3))
    for cu in ([0, 500, 90, 130], [-5, 20, 2 ** 31 - 1, 130], [130, 100, 50, 0]):
        c = cu_of(cu)
        guard = torch.full((3, T, 2, 64), 7.0, dtype=BF, device=DEV)
        _, ck, _ = L.gdr_fwd(q, k, v, g, beta, h0, cu_seqlens=c, o=guard[1:2])
        L.gdr_bwd(do, q, k, v, g, beta, ck, dhT, cu_seqlens=c)
        torch.cuda.synchronize()
        assert (guard[0] == 7).all() and (guard[2] == 7).all()


def test_outputs_are_fully_written_and_repeat():
    note("gdr prefilled outputs, two runs")
    q, k, v, g, beta, h0, do, dhT = dev(*make(2, 70, 2, 4, 128, 64, BF, seed=5))
    nan = float("nan")
    runs = []
    for fill in (nan, 3.0):
        full = lambda t: torch.full_like(t, fill)  # noqa: E731
        hT = torch.full((2, 4, 64, 128), fill, device=DEV)
        ws = torch.full((gdr._lib().gdr_fwd_workspace_bytes(2, 70, 2, 4, 128, 64, 1, 0, 0) // 4,), fill, device=DEV)
        o, ck, hT = L.gdr_fwd(q, k, v, g, beta, h0, o=full(v), hT=hT, workspace=ws)
        out = [full(t) for t in (q, k, v, g, beta)]
        wb = torch.full((gdr._lib().gdr_bwd_workspace_bytes(2, 70, 2, 4, 128, 64, 1, 0, 0) // 4,), fill, device=DEV)
        dh0 = L.gdr_bwd(do, q, k, v, g, beta, ck, dhT, out=out, workspace=wb)[5]
        runs.append([o, hT, ck, *out, dh0])
    torch.cuda.synchronize()
    for a, b in zip(*runs):
        assert torch.isfinite(a).all() and torch.equal(a, b)


def test_in_place_state_and_wanted_outputs():
    note("gdr hT in place of h0")
    q, k, v, g, beta, h0, *_ = dev(*make(2, 90, 2, 2, 64, 64, BF, seed=6))
    o, ck, hT = L.gdr_fwd(q, k, v, g, beta, h0)
    s = h0.clone()
    o2, ck2, hT2 = L.gdr_fwd(q, k, v, g, beta, s, hT=s, want_ckpt=False)
    o3, ck3, hT3 = L.gdr_fwd(q, k, v, g, beta, h0, want_o=False, want_ckpt=False)
    torch.cuda.synchronize()
    assert ck2 is None and ck3 is None and o3 is None and hT2 is s
    assert torch.equal(o, o2) and torch.equal(hT, s) and torch.equal(hT, hT3)


def test_differences():
    """A directional derivative from the forward itself (fp32 inputs) against the backward:
    the central difference over +-h is off by the rounding of o and hT over h (about
    2^-22 |L| / h) and by h^2 / 6 of the third derivative."""
    note("gdr central differences")
    x = make(1, 130, 1, 2, 64, 64, F32, seed=8)
    q, k, v, g, beta, h0, do, dhT = dev(*x)
    got = run(x)
    gen = torch.Generator().manual_seed(3)
    h = 2.0 ** -6
    for i, (t, n) in enumerate(zip((q, k, v, g, beta, h0), GRADS)):
        d = torch.randn(t.shape, generator=gen).to(DEV)
        d = d / d.norm() * t.norm() * 0.25

        def loss(sign):
            ins = [q, k, v, g, beta, h0]
            ins[i] = t + sign * h * d
            o, _, hT = L.gdr_fwd(*ins, want_ckpt=False)
            return ((o.double() * do.double()).sum() + (hT.double() * dhT.double()).sum()).item()

        num, ana = (loss(1) - loss(-1)) / (2 * h), (got[n].double() * d.double()).sum().item()
        size = got[n].double().norm().item() * d.double().norm().item()
        assert abs(num - ana) <= 2e-3 * size + 1e-3 * abs(ana), (n, num, ana, size)


def test_other_stream_and_graph():
    """A forward and backward captured once and replayed with other offsets and inputs, against eager calls."""
    note("gdr stream and graph")
    T, N = 200, 4
    x = make(1, T, 1, 2, 64, 64, BF, seed=11, N=N)
    q, k, v, g, beta, h0, do, dhT = dev(*x)
    offsets = [[0, 64, 64, 130, 200], [0, 1, 2, 3, 150], [0, 200, 200, 200, 200]]
    c = cu_of(offsets[0])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())

    def both():
        o, ck, hT = L.gdr_fwd(q, k, v, g, beta, h0, cu_seqlens=c)
        return [o, hT, *L.gdr_bwd(do, q, k, v, g, beta, ck, dhT, cu_seqlens=c)]

    with torch.cuda.stream(side):
        first = both()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = both()
    for i in range(6):
        c.copy_(cu_of(offsets[i % 3]))
        v.mul_(1.25)
        graph.replay()
        got = [t.clone() for t in outs]
        torch.cuda.synchronize()
        want = both()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)), i
    assert all(torch.isfinite(t).all() for t in first)


def test_autograd_op_and_norm():
    """The layer as it is used: a norm before, the rule, a per-head norm after it; every gradient
    against 64-bit autograd on the definitions."""
    note("GDR + LN autograd")
    B, T, Hk, H, K, V = 2, 75, 2, 4, 64, 64
    q, k, v, g, beta, h0, *_ = make(B, T, Hk, H, K, V, F32, seed=12)
    gen = torch.Generator().manual_seed(2)
    w1, b1, w2 = (torch.randn(n, generator=gen) for n in (H * V, H * V, H * V))
    cot = torch.randn(B, T, H * V, generator=gen)
    leaves = [t.to(DEV).requires_grad_() for t in (q, k, v, g, beta, h0, w1, b1, w2)]
    Q, Kk, Vv, G, Bt, S0, W1, B1, W2 = leaves
    xn = L.LN.apply(Vv.reshape(B, T, H * V), W1, B1)
    o, hT = L.GDR.apply(Q, Kk, xn.view(B, T, H, V), G, Bt, S0)
    y = L.LN.apply(o.reshape(B, T, H * V), W2, None, H)
    loss = (y * cot.to(DEV)).sum() + hT.square().sum()
    got = torch.autograd.grad(loss, leaves)

    ref = [t.detach().double().cpu().requires_grad_() for t in leaves]
    rq, rk, rv, rg, rb, rs, rw1, rb1, rw2 = ref

    def norm(z, w, b, n):
        p = z.reshape(B, T, n, -1)
        c = p - p.mean(-1, keepdim=True)
        return (c / (c.square().mean(-1, keepdim=True) + 1e-5).sqrt()).reshape(B, T, -1) * w + b

    from tests.gdr_util import ref_dense
    ro, rhT = ref_dense(rq, rk, norm(rv, rw1, rb1, 1).view(B, T, H, V), rg, rb, rs, K ** -0.5)
    ry = norm(ro, rw2, 0.0, H)
    want = torch.autograd.grad((ry * cot.double()).sum() + rhT.square().sum(), ref)
    # the norms add a sum over H V channels forward and backward, and divide by the
    # spread of o's parts, which amplifies o's error by |o| / spread (about 1 here)
    tol = 2 * tol_bwd(K, V, F32) + 2 * H * V * 2.0 ** -24
    for n, a, b in zip("q k v g beta h0 w1 b1 w2".split(), got, want):
        assert rel(a, b) <= tol, (n, rel(a, b), tol)


def test_autograd_types_and_missing_gradients():
    note("GDR autograd, bf16, unused hT, packed tail")
    q, k, v, g, beta, h0, *_ = dev(*make(1, 40, 1, 2, 64, 64, BF, seed=13, N=1))
    for t in (q, k, v):
        t.requires_grad_()
    gb = g.to(BF).requires_grad_()
    o, hT = L.GDR.apply(q, k, v, gb, beta, None, cu_of([0, 30]), 0.5)
    o.float().square().sum().backward()
    assert q.grad.dtype == BF and gb.grad.dtype == BF and (q.grad[:, 30:] == 0).all() and (gb.grad[:, 30:] == 0).all()
    assert (o[:, 30:] == 0).all() and torch.isfinite(k.grad).all()
    with torch.no_grad():
        o2, _ = L.GDR.apply(q, k, v, gb, beta, None, cu_of([0, 30]), 0.5)
    assert torch.equal(o, o2)
    q.grad = None
    o, hT = L.GDR.apply(q, k, v, g, beta)
    hT.sum().backward()                                    # o unused
    assert (q.grad == 0).all() and k.grad.abs().sum() > 0


# ---------------------------------------------------------------------------- the recurrent step
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("K,V", HEADS)
@pytest.mark.parametrize("B,T,Hk,H", [(1, 1, 1, 1), (3, 1, 2, 6), (2, 4, 1, 2), (70, 1, 2, 2)])
def test_step(B, T, Hk, H, K, V, dtype):
    note(f"gdr step B{B} T{T} Hk{Hk} H{H} K{K} V{V} {dtype}")
    q, k, v, g, beta, h0, *_ = make(B, T, Hk, H, K, V, dtype, seed=B)
    want = reference(q, k, v, g, beta, h0)
    dq = dev(q, k, v, g, beta)
    s = h0.to(DEV)
    o = L.gdr_step(*dq, s)
    out = torch.full_like(s, 5.0)
    o2 = L.gdr_step(*dq, h0.to(DEV), state_out=out)
    torch.cuda.synchronize()
    assert rel(o, want["o"]) <= tol_fwd(K, dtype) and rel(s, want["hT"]) <= tol_fwd(K, F32)
    assert torch.equal(o, o2) and torch.equal(s, out)


def test_step_slots():
    """Slots in any order, padding rows, and rows that share a slot: consecutive tokens of one sequence."""
    note("gdr step slots")
    B, T, Hk, H, K, V, P = 8, 2, 1, 2, 64, 128, 9
    q, k, v, g, beta, h0, *_ = make(B, T, Hk, H, K, V, BF, seed=1, N=P)
    slots = [4, -1, 0, 4, P, 8, 0, 4]
    state = h0.to(DEV)
    o = L.gdr_step(*dev(q, k, v, g, beta), state, slots=torch.tensor(slots, dtype=torch.int32, device=DEV))
    torch.cuda.synchronize()
    want, wo = h0.double().clone(), torch.zeros(B, T, H, V, dtype=torch.float64)
    for b, s in enumerate(slots):
        if 0 <= s < P:
            r = reference(*[x[b:b + 1] for x in (q, k, v, g, beta)], want[s:s + 1])
            wo[b], want[s] = r["o"][0], r["hT"][0]
    assert rel(o, wo) <= tol_fwd(K, BF) and rel(state, want) <= tol_fwd(K, F32)
    assert (o[1] == 0).all() and (o[4] == 0).all()
    for s in (1, 2, 3, 5, 6, 7):
        assert torch.equal(state[s].cpu(), h0[s])


def test_step_edges_and_graph():
    note("gdr step, g = -inf, beta = 0, graph")
    B, H = 3, 2
    q, k, v, g, beta, h0, *_ = make(B, 1, H, H, 64, 64, BF, seed=21)
    g[0], beta[1] = -float("inf"), 0.0
    want = reference(q, k, v, g.clamp(min=-1e4), beta, h0)
    ins, s = dev(q, k, v, g, beta), h0.to(DEV)
    slots = torch.tensor([2, 0, 1], dtype=torch.int32, device=DEV)
    pool = h0[[1, 2, 0]].to(DEV)
    o = L.gdr_step(*ins, s)
    assert rel(o, want["o"]) <= tol_fwd(64, BF) and rel(s, want["hT"]) <= tol_fwd(64, F32)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        og = L.gdr_step(*ins, pool, slots=slots)
    eager = pool.clone()
    for i in range(4):
        slots.copy_(torch.tensor([[2, 0, 1], [1, 1, -1], [0, 2, 2], [7, 0, 1]][i], dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        oe = L.gdr_step(*ins, eager, slots=slots)
        torch.cuda.synchronize()
        assert torch.equal(og, oe) and torch.equal(pool, eager), i


def test_prompt_then_steps_then_norm():
    """Serving as a whole: packed prompts fill a pool, tokens follow one at a time, each output goes
    through the per-head norm."""
    note("gdr prompt + steps + norm")
    Hk, H, K, V, P = 1, 2, 128, 128, 5
    lens, new = [65, 1, 0, 130], 5
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    q, k, v, g, beta, *_ = make(1, cu[-1], Hk, H, K, V, BF, seed=31, N=4)
    nq, nk, nv, ng, nb, *_ = make(4, new, Hk, H, K, V, BF, seed=32)
    w = torch.randn(H * V, generator=torch.Generator().manual_seed(5))
    pool = torch.zeros(P, H, V, K, device=DEV)
    slots = torch.tensor([3, 0, 4, 1], dtype=torch.int32, device=DEV)
    _, _, hT = L.gdr_fwd(*dev(q, k, v, g, beta), cu_seqlens=cu_of(cu), want_ckpt=False)
    pool[slots.long()] = hT
    ys, os_ = [], []
    for t in range(new):
        o = L.gdr_step(*dev(*[x[:, t:t + 1].contiguous() for x in (nq, nk, nv, ng, nb)]), pool, slots=slots)
        os_.append(o)
        ys.append(L.ln_fwd(o.view(4, H * V), w.to(DEV), groups=H, want_stats=False)[0])
    torch.cuda.synchronize()
    for n in range(4):
        a, b = cu[n], cu[n + 1]
        full = [torch.cat([x[:, a:b], y[n:n + 1]], 1) for x, y in zip((q, k, v, g, beta), (nq, nk, nv, ng, nb))]
        r = reference(*full)
        o = torch.cat([x[n:n + 1] for x in os_], 1)
        assert rel(o, r["o"][:, b - a:]) <= tol_fwd(K, BF)
        assert rel(pool[slots[n].item()], r["hT"][0]) <= tol_fwd(K, F32)
        for t in range(new):
            want = ref_norm(os_[t][n].reshape(1, -1).cpu(), w, None, H, 1e-5)["y"]
            assert rel(ys[t][n:n + 1], want) <= 2.0 ** -8 + 2 * V * 2.0 ** -24


def test_step_many_rows_of_one_slot():
    """More rows than a workgroup has threads, with the rows of a slot far apart and next to each other."""
    note("gdr step, 600 rows, 300 slots")
    B, H, P = 600, 1, 300
    q, k, v, g, beta, h0, *_ = make(B, 1, 1, H, 64, 64, BF, seed=41, N=P)
    slots = [b % P for b in range(B)]
    slots[257], slots[258], slots[599] = 256, 256, 0
    state = h0.to(DEV)
    o = L.gdr_step(*dev(q, k, v, g, beta), state, slots=torch.tensor(slots, dtype=torch.int32, device=DEV))
    torch.cuda.synchronize()
    want, wo = h0.double().clone(), torch.zeros(B, 1, H, 64, dtype=torch.float64)
    for s in range(P):
        rows = [b for b in range(B) if slots[b] == s]
        if rows:
            r = reference(*[x[rows].transpose(0, 1).contiguous() for x in (q, k, v, g, beta)], want[s:s + 1])
            wo[rows], want[s] = r["o"].transpose(0, 1), r["hT"][0]
    assert rel(o, wo) <= tol_fwd(64, BF) and rel(state, want) <= tol_fwd(64, F32)


def test_two_streams_at_once():
    """Two forwards and backwards in flight together, each on its own stream, against one after the other."""
    note("gdr, two streams")
    sets = [dev(*make(2, 300, 2, 4, 64, 128, BF, seed=s)) for s in (51, 52)]

    def both(x):
        q, k, v, g, beta, h0, do, dhT = x
        o, ck, hT = L.gdr_fwd(q, k, v, g, beta, h0)
        return [o, hT, *L.gdr_bwd(do, q, k, v, g, beta, ck, dhT)]

    want = [both(x) for x in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [None, None]
    for _ in range(3):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i] = both(sets[i])
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_captured_training_step():
    """Norm, rule and norm with their backward captured through autograd, on leaves that no eager graph
    uses, replayed with other values and checked against eager passes on other leaves."""
    note("gdr + ln autograd in a graph")
    B, T, H, K = 2, 70, 2, 64
    vals = [t.to(DEV) for t in make(B, T, H, H, K, K, BF, seed=61)[:5]] + [torch.ones(H * K, device=DEV)]
    cot = torch.randn(B, T, H * K, generator=torch.Generator().manual_seed(3)).to(DEV, BF)

    def grads(leaves):
        q, k, v, g, beta, w = leaves
        xn = L.LN.apply(v.reshape(B, T, H * K), w)
        o, _ = L.GDR.apply(q, k, xn.view(B, T, H, K), g, beta)
        y = L.LN.apply(o.reshape(B, T, H * K), w, None, H)
        return torch.autograd.grad(y, leaves, cot)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        grads([x.clone().requires_grad_() for x in vals])
    torch.cuda.current_stream().wait_stream(side)
    leaves = [x.clone().requires_grad_() for x in vals]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = grads(leaves)
    for i in range(4):
        with torch.no_grad():
            for x, y in zip(leaves, vals):
                x.copy_(y)
            leaves[2].mul_(1.0 + 0.5 * i)
        graph.replay()
        got = [t.clone() for t in outs]
        want = grads([x.detach().clone().requires_grad_() for x in leaves])
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)), i


def test_offsets_past_31_and_32_bits():
    """A short sequence at the end of a row so long that token and checkpoint offsets pass 2^31 and 2^32, and a
    step on the last states of a pool of more than 2^32 values, against the same calls on short tensors."""
    note("gdr, long offsets")
    H, K, V, n = 16, 64, 128, 100
    T = (1 << 20) + 200
    x = dev(*make(1, n, H, H, K, V, BF, seed=71, N=1))
    q, k, v, g, beta, h0, do, dhT = x
    o, ck, hT = L.gdr_fwd(q, k, v, g, beta, h0)
    want = [o, *L.gdr_bwd(do, q, k, v, g, beta, ck, dhT)]

    def tail(t):
        big = torch.empty(1, T, *t.shape[2:], dtype=t.dtype, device=DEV)
        big[:, T - n:] = t
        return big

    bq, bk, bv, bg, bb, bdo = [tail(t) for t in (q, k, v, g, beta, do)]
    assert bv.numel() > 2 ** 31
    cu = cu_of([T - n, T])
    bo, bck, bhT = L.gdr_fwd(bq, bk, bv, bg, bb, h0, cu_seqlens=cu)
    assert bck.numel() > 2 ** 32
    got = [bo, *L.gdr_bwd(bdo, bq, bk, bv, bg, bb, bck, dhT, cu_seqlens=cu)]
    torch.cuda.synchronize()
    assert torch.equal(bhT, hT)
    for a, b in zip(got[:-1], want):
        assert torch.equal(a[:, T - n:], b) and not a[:, :T - n:4099].any()
    assert torch.equal(got[-1], want[-1])
    del bq, bk, bv, bg, bb, bdo, bo, bck, got

    P = (1 << 32) // (H * V * K) + 2
    pool = torch.empty(P, H, V, K, device=DEV)
    pool[P - 1], pool[1] = h0[0], h0[0]
    row = [t[:, :1].contiguous().expand(2, 1, *t.shape[2:]).contiguous() for t in (q, k, v, g, beta)]
    os_ = L.gdr_step(*row, pool, slots=torch.tensor([P - 1, 1], dtype=torch.int32, device=DEV))
    torch.cuda.synchronize()
    assert torch.equal(os_[0], os_[1]) and torch.equal(pool[P - 1], pool[1]) and not torch.equal(pool[1], h0[0])


def test_no_gradient_of_the_gradient():
    note("gdr + ln, second derivative refused")
    q, k, v, g, beta, *_ = dev(*make(1, 5, 1, 1, 64, 64, F32, seed=81))
    v.requires_grad_()
    for y in (L.GDR.apply(q, k, v, g, beta)[0], L.LN.apply(v.reshape(5, 64))):
        dv, = torch.autograd.grad(y.square().sum(), v, create_graph=True)
        with pytest.raises(RuntimeError):
            torch.autograd.grad(dv.sum(), v)


@pytest.mark.parametrize("N,H", [(64, 2), (65, 2), (5, 300)])
def test_packed_many_sequences(N, H):
    """Around the number of sequences that the scans take by length, with equal and empty ones, and with more
    workgroups than that is done for."""
    note(f"gdr packed N{N} H{H}")
    lens = [(7 * i * i) % 90 if i % 5 else 64 for i in range(N)]
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    x = make(1, cu[-1], 1, H, 64, 64, BF, seed=91, N=N)
    q, k, v, g, beta, h0, do, dhT = x
    got = run(x, cu)
    for n in range(N):
        a, b = cu[n], cu[n + 1]
        if a == b:
            assert torch.equal(got["hT"][n].cpu(), h0[n])
            continue
        if n % 9 and n != N - 1:
            continue
        r = reference(*[t[:, a:b] for t in (q, k, v, g, beta)], h0[n:n + 1])
        assert rel(got["o"][:, a:b], r["o"]) <= tol_fwd(64, BF) and rel(got["hT"][n:n + 1], r["hT"]) <= tol_fwd(64, F32)


def test_one_token_views_and_checkpoints_alone():
    """Slices of longer tensors, whose gates lie at odd addresses, and a forward that only leaves checkpoints."""
    note("gdr views")
    q, k, v, g, beta, h0, do, dhT = dev(*make(1, 70, 1, 3, 64, 64, BF, seed=95))
    s, s2 = h0.clone(), h0.clone()
    for t in range(3):
        cut = [x[:, t:t + 1] for x in (q, k, v, g, beta)]
        o = L.gdr_step(*cut, s)
        o2 = L.gdr_step(*[x.clone() for x in cut], s2)
        assert torch.equal(o, o2) and torch.equal(s, s2)
    cut = [x[:, 1:68] for x in (q, k, v, g, beta)]
    assert cut[3].data_ptr() % 16
    o, ck, hT = L.gdr_fwd(*cut, h0)
    o2, ck2, hT2 = L.gdr_fwd(*[x.clone() for x in cut], h0)
    none, ck3, none2 = L.gdr_fwd(*cut, h0, want_o=False, want_hT=False)
    a, b = (L.gdr_bwd(do[:, 1:68].contiguous(), *c, x, dhT) for c, x in ((cut, ck3), ([x.clone() for x in cut], ck2)))
    torch.cuda.synchronize()
    assert none is None and none2 is None
    assert torch.equal(o, o2) and torch.equal(hT, hT2) and all(torch.equal(x, y) for x, y in zip(a, b))

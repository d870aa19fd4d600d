"""The convolution, the selective scan and the block norm run together, as one layer of a model
uses them: input projection, convolution, projections of its output to steps and matrices, scan,
norm and gate with the residual and the next norm.  Training, a prompt with single tokens
after it, packed sequences, and a captured step.

Tolerances.  A stage adds its own error (mix_util's; a product over K values: K E of its terms'
sizes) and passes on what it got.  How much larger that may become is bounded by the terms' sizes
beside the results': norms divide by a row's own size and the other stages' weights are made to keep
it, so each of the seven stages at most doubles it, and half of them do for any one value: 2^4 of
the sum of all stages' errors.
"""
import pytest
import torch

import linear_rnn_lm_amd as L
from tests.gpu_util import note
from tests.mix_util import E, conv_tol, ref_conv, ref_rn, ref_scan, rel, scan_tol

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
BF, F32 = torch.bfloat16, torch.float32
OPT = dict(groups=2, norm="rms", norm2="rms")


def make(C, S, R, W, dtype, seed=0):
    gen = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    return dict(win=(rn(C, 2 * C) / C ** 0.5).to(dtype), wx=(rn(C, R + 2 * S) / C ** 0.5).to(dtype),
                wdt=(rn(R, C) / R ** 0.5).to(dtype), conv_w=(rn(C, W) / W ** 0.5).to(dtype), conv_b=(0.1 * rn(C)).to(dtype),
                A=-torch.exp(0.5 * rn(C, S)), D=1 + 0.1 * rn(C), dt_bias=rn(C) - 2, weight=1 + 0.1 * rn(C),
                scale=1 + 0.1 * rn(C), weight2=1 + 0.1 * rn(C))


def layer(p, u, res, conv_state, state, cu=None, slots=None, ref=False):
    """u: (B, T, C) in the layer's type, res fp32.  Returns r, h and both states.  With `ref` from the
    definitions; with `slots` single steps, the states updated in place."""
    C, S = p["A"].shape
    R, W = p["wdt"].shape[0], p["conv_w"].shape[1]
    mm = lambda a, w: (a.flatten(0, -2) @ w).unflatten(0, a.shape[:-1])  # noqa: E731
    xz = mm(u, p["win"])
    x, z = xz[..., :C], xz[..., C:]
    cut = cu if ref or cu is None else torch.tensor(cu, dtype=torch.int32, device=DEV)
    if ref:
        x, conv_out = ref_conv(dict(x=x, weight=p["conv_w"], bias=p["conv_b"], h0=conv_state), cu=cu)
    elif slots is None:
        x, conv_out = L.CONV.apply(x, p["conv_w"], p["conv_b"], conv_state, cut)
    else:
        x, conv_out = L.conv_step(x, p["conv_w"], p["conv_b"], conv_state, slots=slots), conv_state
    dbc = mm(x, p["wx"])
    dt = mm(dbc[..., :R].contiguous(), p["wdt"])
    b, c = (t.unsqueeze(-2) for t in dbc[..., R:].split(S, -1))
    if ref:
        y, out = ref_scan(dict(x=x, dt=dt, A=p["A"], b=b, c=c, D=p["D"], z=None, dt_bias=p["dt_bias"], h0=state), cu=cu)
        r, h = ref_rn(dict(o=y, gate=z, res=res, weight=p["weight"], bias=None, scale=p["scale"], weight2=p["weight2"],
                           bias2=None), **OPT)
        return r, h, conv_out, out
    if slots is None:
        y, out = L.SSM.apply(x, dt, p["A"], b, c, p["D"], None, p["dt_bias"], state, cut)
        r, h = L.RN.apply(y, z, res, p["weight"], None, p["scale"], p["weight2"], None, OPT)
    else:
        y, out = L.ssm_step(x, dt, p["A"], b, c, state, p["D"], dt_bias=p["dt_bias"], slots=slots), state
        r, h, _ = L.rn_fwd(y, z, res, weight=p["weight"], scale=p["scale"], weight2=p["weight2"], want_stats=False, **OPT)
    return r, h, conv_out, out


def tol(T, C, S, W, grad=False):
    ops = conv_tol(W, F32, T if grad else 0, grad) + scan_tol(T, S, F32, T if grad else 0, grad)
    return 16 * (ops + 4 * C * E + (8 if grad else 4) * C * E)


def test_training_pass():
    note("mix: training")
    B, T, C, S, R, W = 2, 45, 128, 16, 8, 4
    p = make(C, S, R, W, F32)
    gen = torch.Generator().manual_seed(1)
    u, res, dr, dh = (torch.randn(B, T, C, generator=gen) for _ in range(4))
    names = list(p)
    got = {n: t.to(DEV).requires_grad_() for n, t in {**p, "u": u, "res": res}.items()}
    r, h, _, _ = layer(got, got["u"], got["res"], None, None)
    torch.autograd.backward([r, h], [dr.to(DEV), dh.to(DEV)])
    want = {n: t.double().requires_grad_() for n, t in {**p, "u": u, "res": res}.items()}
    wr, wh, _, _ = layer(want, want["u"], want["res"], None, None, ref=True)
    torch.autograd.backward([wr, wh], [dr.double(), dh.double()])
    assert rel(r, wr) <= tol(T, C, S, W) and rel(h, wh) <= tol(T, C, S, W)
    for n in names + ["u", "res"]:
        assert rel(got[n].grad, want[n].grad) <= tol(B * T, C, S, W, True), n


def test_prompt_then_tokens():
    """Packed prompts, their states put into pools, then single tokens in another order of rows."""
    note("mix: prompt and tokens")
    C, S, R, W, P, more = 128, 16, 8, 4, 5, 4
    p = make(C, S, R, W, F32, seed=2)
    cu = [0, 7, 40, 41]
    gen = torch.Generator().manual_seed(3)
    u, res = torch.randn(1, cu[-1], C, generator=gen), torch.randn(1, cu[-1], C, generator=gen)
    u2, res2 = torch.randn(3, more, C, generator=gen), torch.randn(3, more, C, generator=gen)
    d = {n: t.to(DEV) for n, t in p.items()}
    with torch.no_grad():
        r, h, cs, st = layer(d, u.to(DEV), res.to(DEV), None, None, cu=cu)
        pools = [torch.zeros(P, W - 1, C, device=DEV), torch.zeros(P, C, S, device=DEV)]
        at = [4, 0, 2]
        for pool, s in zip(pools, (cs, st)):
            pool[at] = s
        order = [2, 0, 1]                                  # row i of a step is sequence order[i]; the last row is padding
        slots = torch.tensor([at[i] for i in order] + [-1], dtype=torch.int32, device=DEV)
        rows = [layer(d, torch.cat([u2[order, t:t + 1], u2[:1, :1]]).to(DEV), torch.cat([res2[order, t:t + 1], res2[:1, :1]]).to(DEV),
                      *pools, slots=slots)[:2] for t in range(more)]
    torch.cuda.synchronize()
    v = {n: t.double() for n, t in p.items()}
    for i, (a, b) in enumerate(zip(cu, cu[1:])):
        whole = [torch.cat([t[:, a:b], t2[i:i + 1]], 1).double() for t, t2 in ((u, u2), (res, res2))]
        wr, wh, wc, ws = layer(v, *whole, None, None, ref=True)
        lim = tol(b - a + more, C, S, W)
        assert rel(r[:, a:b], wr[:, :b - a]) <= lim and rel(h[:, a:b], wh[:, :b - a]) <= lim
        row = order.index(i)
        assert rel(torch.cat([q[0][row:row + 1] for q in rows], 1), wr[:, b - a:]) <= lim
        assert rel(torch.cat([q[1][row:row + 1] for q in rows], 1), wh[:, b - a:]) <= lim
        assert rel(pools[0][at[i]], wc[0]) <= lim and rel(pools[1][at[i]], ws[0]) <= lim
    assert (pools[0][[1, 3]] == 0).all() and (pools[1][[1, 3]] == 0).all()


@pytest.mark.parametrize("dtype", [F32, BF])
def test_captured_token(dtype):
    """A layer's step captured into a graph: every replay gives the eager step's bits, states too."""
    note(f"mix: captured token {dtype}")
    B, C, S, R, W, P = 3, 128, 16, 8, 3, 4
    d = {n: t.to(DEV) for n, t in make(C, S, R, W, dtype, seed=4).items()}
    gen = torch.Generator().manual_seed(5)
    u, res = torch.randn(B, 1, C, generator=gen).to(dtype).to(DEV), torch.randn(B, 1, C, generator=gen).to(DEV)
    slots = torch.tensor([3, 0, 1], dtype=torch.int32, device=DEV)
    pools = [torch.zeros(P, W - 1, C, dtype=dtype, device=DEV), torch.zeros(P, C, S, device=DEV)]
    with torch.no_grad():
        step = lambda q: layer(d, u, res, *q, slots=slots)[:2]  # noqa: E731
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step([q.clone() for q in pools])
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs = step(pools)
        for i in range(4):
            u.copy_(torch.randn(B, 1, C, generator=gen).to(dtype))
            slots.copy_(torch.tensor([[3, 0, 1], [1, 1, 2], [-1, 3, 0], [2, 0, 4]][i], dtype=torch.int32))
            other = [q.clone() for q in pools]
            graph.replay()
            torch.cuda.synchronize()
            want = step(other)
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip((*outs, *pools), (*want, *other))), i


@pytest.mark.parametrize("C,dtype", [(64, F32), (67, BF), (66, BF), (21, F32)])
def test_new_rows_outside_sequences_are_zero(C, dtype):
    """New outputs in memory that held other values: most of the row is padding, before and behind the sequences."""
    note(f"mix: rows outside C{C} {dtype}")
    T, S, cu = 400, 16, torch.tensor([37, 60, 60, 131], dtype=torch.int32, device=DEV)
    gen = torch.Generator().manual_seed(6)
    rn = lambda *s: torch.randn(*s, generator=gen).to(dtype).to(DEV)  # noqa: E731
    x, dt, z, dy, b, c = rn(1, T, C), rn(1, T, C), rn(1, T, C), rn(1, T, C), rn(1, T, 1, S), rn(1, T, 1, S)
    A, w = -torch.rand(C, S, generator=gen).to(DEV), rn(C, 4)
    torch.cuda.synchronize()
    stale = [torch.full((1, T, n), float("nan"), dtype=dtype, device=DEV) for n in (C, C, C, C, C, C, S, S)]
    del stale
    y, ckpt, _ = L.ssm_fwd(x, dt, A, b, c, None, z, cu_seqlens=cu)
    dx, ddt, _, db, dc, _, dz, _, _ = L.ssm_bwd(dy, x, dt, A, b, c, ckpt, None, z, cu_seqlens=cu)
    v, _ = L.conv_fwd(x, w, cu_seqlens=cu)
    dv = L.conv_bwd(dy, x, w, cu_seqlens=cu)[0]
    torch.cuda.synchronize()
    for n, t in dict(y=y, dx=dx, ddt=ddt, dz=dz, db=db, dc=dc, v=v, dv=dv).items():
        assert (t[:, :37] == 0).all() and (t[:, 131:] == 0).all() and t.isfinite().all() and t[:, 37:131].any(), n

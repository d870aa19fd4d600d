"""More calls of the selective scan, the short convolution and the block norm on the GPU, against
their definitions in 64 bits (tolerances: mix_util, or derived beside the test)."""
import pytest
import torch

import linear_rnn_lm_amd as L
from tests.gpu_util import note
from tests.mix_util import (E, GRADS, INS, conv_tol, half_step, make_conv, make_scan, ref_conv_grads, ref_scan, ref_scan_grads,
                            rel, scan_tol)
from tests.test_gpu_rnorm import check as check_rn
from tests.test_gpu_rnorm import make as make_rn
from tests.test_gpu_ssm import check as check_scan

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
BF, F32 = torch.bfloat16, torch.float32

# Activations, value by value.  e^-v is good to 5 E: the exponential's last place (2 E), the corrected argument (2^t e^r
# is one rounding, the constant ln 2 gives |v| E / 20, below 4.5 E at 88; the roundings of r itself are
# smaller still): at most 5 E up to |v| of 30 and 7.5 E beyond, where 1 + e^-v and the logarithm add next to nothing of
# their own.  Below 30 the sum 1 + e^-v adds E and the reciprocal's last place 2 E: 8 E; the logarithm's last place
# 2 E and the product with ln 2 E: 8 E.
SPANS = [(-86, -60), (-60, -30), (-30, -10), (-10, -7), (-7, -4), (-4, -1), (-1, 1), (1, 20), (20, 80)]


def spread(lo, hi, n):
    return torch.rand(n, generator=torch.Generator().manual_seed(1), dtype=torch.float64) * (hi - lo) + lo


@pytest.mark.parametrize("lo,hi", SPANS)
def test_steps_keep_their_bits(lo, hi):
    """softplus alone: a state of zero, x = b = 1 and no decay leave delta as the state."""
    note(f"mix: softplus {lo} {hi}")
    v = spread(lo, hi, 1 << 16).float().view(1, 1, -1)
    C = v.shape[2]
    one, b = torch.ones(1, 1, C, device=DEV), torch.ones(1, 1, 1, 16, device=DEV)
    state = torch.zeros(1, C, 16, device=DEV)
    L.ssm_step(one, v.to(DEV), torch.zeros(C, 16, device=DEV), b, b, state)
    _, _, hT = L.ssm_fwd(one, v.to(DEV), torch.zeros(C, 16, device=DEV), b, b, want_ckpt=False)
    torch.cuda.synchronize()
    want = torch.logaddexp(v.double(), torch.zeros(1, dtype=torch.float64)).view(1, C, 1)
    for h in (state, hT):
        err = ((h.double().cpu() - want).abs() / want).max().item()
        assert err <= 8 * E, (lo, hi, err / E)


@pytest.mark.parametrize("lo,hi", SPANS)
def test_gates_keep_their_bits(lo, hi):
    """silu and sigmoid alone: a filter of one tap gives s = x, a scan of y = D x = 1 its gate, a norm of
    1 / sqrt(1 + 0) its activation; each adds at most two roundings to the sigmoid's 8 E."""
    note(f"mix: sigmoid {lo} {hi}")
    v = spread(lo, hi, 1 << 16).float()
    v[v == 0] = 1.0
    C, g = v.numel(), v.to(DEV)
    w = torch.zeros(C, 2, device=DEV)
    w[:, 1] = 1
    y, _ = L.conv_fwd(g.view(1, 1, C), w, want_hT=False)
    one, zero, S0 = torch.ones(1, 1, C, device=DEV), torch.zeros(1, 1, 1, 16, device=DEV), torch.zeros(C, 16, device=DEV)
    gated, _, _ = L.ssm_fwd(one, one, S0, zero, zero, torch.ones(C, device=DEV), g.view(1, 1, C), want_ckpt=False, want_hT=False)
    rows = lambda act: L.rn_fwd(torch.ones(C // 64, 64, device=DEV), g.view(-1, 64), norm="rms", act=act, eps=0.0)[0]  # noqa: E731
    torch.cuda.synchronize()
    s = torch.sigmoid(v.double())
    for got, want in ((y, s * v), (gated, s * v), (rows("silu"), s * v), (rows("sigmoid"), s)):
        err = ((got.double().cpu().flatten() - want).abs() / want.abs()).max().item()
        assert err <= 10 * E, (lo, hi, err / E)


def test_activations_of_no_numbers():
    """Infinities keep the activations' limits where those are numbers, and NaN stays NaN."""
    note("mix: activations of infinities")
    inf, nan = float("inf"), float("nan")
    v = torch.tensor([inf, -inf, nan, 3e38, -3e38, 1e30, -1e30, 200.0, -200.0], device=DEV)
    n = v.numel()
    one, b = torch.ones(1, 1, n, device=DEV), torch.ones(1, 1, 1, 16, device=DEV)
    _, _, hT = L.ssm_fwd(one, v.view(1, 1, n), torch.zeros(n, 16, device=DEV), b, b, want_ckpt=False)
    keep = [1, 3, 4, 5, 6, 7, 8]                           # no decay: e^0, but an infinite step of A = 0 is no number
    want = torch.tensor([0, 3e38, 0, 1e30, 0, 200.0, 0], device=DEV)
    torch.cuda.synchronize()
    assert torch.equal(hT[0, keep, 0], want) and torch.isnan(hT[0, 2]).all() and not torch.isfinite(hT[0, 0]).any()
    gate = v.view(n, 1).expand(n, 8).contiguous()
    r = L.rn_fwd(torch.ones(n, 8, device=DEV), gate, norm="rms", act="sigmoid", eps=0.0)[0]
    torch.cuda.synchronize()
    want = torch.tensor([1, 0, nan, 1, 0, 1, 0, 1, 0.0], device=DEV).view(n, 1).expand(n, 8)
    assert torch.equal(torch.isnan(r), torch.isnan(want)) and torch.equal(torch.nan_to_num(r), torch.nan_to_num(want))


@pytest.mark.parametrize("dtype", [F32, BF])
def test_last_tokens_of_long_rows(dtype):
    """Views x[:, -1:] whose rows lie more than 2^24 values apart: a step takes them, SSM copies them, ssm_fwd refuses."""
    note(f"ssm far rows {dtype}")
    B, T, C, S = 2, 4099, 4096, 16
    p = {n: None if t is None else t.to(DEV) for n, t in make_scan(B, 1, C, S, 1, dtype, seed=3).items()}
    big = {n: torch.full((B, T if n != "b" else 2 ** 20 + 1, *p[n].shape[2:]), float("nan"), dtype=dtype, device=DEV) for n in "xzb"}
    for n, t in big.items():
        t[:, -1:] = p[n]
        big[n] = t[:, -1:]
        assert t.stride(0) > 2 ** 24
    x, z, b = big["x"], big["z"], big["b"]
    state, alone = p["h0"].clone(), p["h0"].clone()
    y = L.ssm_step(x, p["dt"], p["A"], b, p["c"], state, p["D"], z, dt_bias=p["dt_bias"])
    want = L.ssm_step(p["x"], p["dt"], p["A"], p["b"], p["c"], alone, p["D"], p["z"], dt_bias=p["dt_bias"])
    ya, ha = L.SSM.apply(x, p["dt"], p["A"], b, p["c"], p["D"], z, p["dt_bias"], p["h0"])
    yb, hb = L.SSM.apply(p["x"], p["dt"], p["A"], p["b"], p["c"], p["D"], p["z"], p["dt_bias"], p["h0"])
    torch.cuda.synchronize()
    assert torch.equal(y, want) and torch.equal(state, alone) and torch.equal(ya, yb) and torch.equal(ha, hb)
    with pytest.raises(L.Wkv7Error, match="SHAPE"):
        L.ssm_fwd(x, p["dt"], p["A"], b, p["c"])


def test_millions_of_sequences():
    """More than 2^21 sequences of one token: h = delta x b, y = (c b) delta x + D x."""
    note("ssm 2^21 sequences")
    N, C, S = 2 ** 21 + 5, 8, 16
    gen = torch.Generator(device=DEV).manual_seed(1)
    x, dt, b, c = (torch.randn(N, 1, *s, generator=gen, device=DEV).to(BF) for s in ((C,), (C,), (1, S), (1, S)))
    A, D = -torch.ones(C, S, device=DEV), torch.ones(C, device=DEV)
    cu = torch.arange(N + 1, dtype=torch.int32, device=DEV)
    y, _, hT = L.ssm_fwd(x, dt, A, b, c, D, want_ckpt=False)
    flat = lambda t: t.view(1, N, *t.shape[2:])  # noqa: E731
    yp, _, hp = L.ssm_fwd(flat(x), flat(dt), A, flat(b), flat(c), D, cu_seqlens=cu, want_ckpt=False)
    torch.cuda.synchronize()
    # one token: delta is good to 8 E, its products to 2 more; y is a sum of S + 1 terms, of which the largest are a few times
    # the result's size on average, and is rounded once
    d = torch.nn.functional.softplus(dt.double())[:, 0]
    want = (d * x[:, 0].double())[..., None] * b[:, 0].double()
    err = ((hT.double() - want).norm() / want.norm()).item()
    assert err <= 10 * E
    del hT
    want = (want * c[:, 0].double()).sum(-1) + x[:, 0].double()
    err = ((y[:, 0].double() - want).norm() / want.norm()).item()
    assert err <= half_step(BF) + 4 * (S + 10) * E
    assert torch.equal(yp.view_as(y), y)


@pytest.mark.parametrize("wd,bd", [(BF, F32), (F32, BF)])
def test_convolution_with_weights_of_two_types(wd, bd):
    """A bias of fp32 beside bf16 filters keeps its bits, and the other way; a state of another type than x's is refused."""
    note(f"CONV {wd} {bd}")
    p = make_conv(2, 21, 40, 4, F32, seed=5)
    p["weight"], p["bias"] = p["weight"].to(wd), (p["bias"] + 1000 * E).to(bd)
    wy, wh, want = ref_conv_grads(p)
    leaves = {n: p[n].to(DEV).requires_grad_() for n in ("x", "weight", "bias", "h0")}
    y, hT = L.CONV.apply(*leaves.values())
    torch.autograd.backward([y, hT], [p["dy"].to(DEV), p["dhT"].to(DEV)])
    assert rel(y, wy) <= conv_tol(4, F32) and rel(hT, wh) <= conv_tol(4, F32)
    for (n, t), g in zip(leaves.items(), ("dx", "dweight", "dbias", "dh0")):
        assert t.grad.dtype == p[n].dtype and rel(t.grad, want[g]) <= conv_tol(4, p[n].dtype, 42, True), n
    with pytest.raises(ValueError, match="h0"):
        L.CONV.apply(leaves["x"].to(BF), leaves["weight"], leaves["bias"], leaves["h0"])


def test_without_gradients():
    """SSM and RN in a block without gradients, their weights being parameters: the same outputs, no memory for a backward."""
    note("SSM, RN without gradients")
    B, T, C, S = 1, 4096, 512, 64
    p = {n: None if t is None else t.to(DEV) for n, t in make_scan(B, T, C, S, 1, BF, seed=6, h0=False).items()}
    p["A"].requires_grad_(), p["D"].requires_grad_()
    scan = lambda: L.SSM.apply(*[p[n] for n in ("x", "dt", "A", "b", "c", "D", "z", "dt_bias")])  # noqa: E731
    w = torch.ones(C, device=DEV, requires_grad=True)
    norm = lambda y: L.RN.apply(y, p["z"], None, w, None, None, w, None, dict(norm="rms", norm2="rms"))  # noqa: E731
    want = [t.detach() for t in (*scan(), *norm(p["x"]))]
    with torch.no_grad():
        torch.cuda.synchronize()
        torch.cuda.reset_peak_memory_stats()
        before = torch.cuda.memory_allocated()
        got = scan()
        used = torch.cuda.max_memory_allocated() - before
        got = [*got, *norm(p["x"])]
    lib, dims = L.ssm._lib(), (B, T, C, S, 1, 0, 0)
    assert used < lib.ssm_ckpt_bytes(*dims) / 2
    assert all(torch.equal(a, b) and not a.requires_grad for a, b in zip(got, want))
    with torch.no_grad(), torch.enable_grad():
        y, _ = scan()
    y.backward(p["dy"])
    assert torch.isfinite(p["A"].grad).all() and p["A"].grad.any()


@pytest.mark.parametrize("B,T,C,S", [(2, 5, 24, 16), (1, 300, 40, 16), (3, 33, 40, 32), (1, 35, 33, 64)])
def test_states_without_memory(B, T, C, S):
    """A of -infinity clears a state at every step, as -1e30 does, and tokens behind a sequence's end do not touch it."""
    note(f"ssm A -inf B{B} T{T} C{C} S{S}")
    p = make_scan(B, T, C, S, 1, F32, seed=9)
    p["A"][:, 0], p["A"][3] = -1e30, -1e30                 # every delta is above 1e-5: e^(delta A) is 0 in any precision
    wy, wh, want = ref_scan_grads(p, dev=DEV)
    p["A"][p["A"] < -1e29] = -float("inf")
    d = {n: None if t is None else t.to(DEV) for n, t in p.items()}
    ins = [d[n] for n in ("x", "dt", "A", "b", "c")]
    y, ckpt, hT = L.ssm_fwd(*ins, d["D"], d["z"], d["h0"], dt_bias=d["dt_bias"])
    got = dict(zip(GRADS, L.ssm_bwd(d["dy"], *ins, ckpt, d["D"], d["z"], d["dhT"], dt_bias=d["dt_bias"])))
    state = d["h0"].clone()
    ys = L.ssm_step(*ins, state, d["D"], d["z"], dt_bias=d["dt_bias"])
    torch.cuda.synchronize()
    for a, h in ((y, hT), (ys, state)):
        assert rel(a, wy) <= scan_tol(T, S, F32) and rel(h, wh) <= scan_tol(T, S, F32)
    for n in GRADS:
        assert rel(got[n], want[n]) <= scan_tol(T, S, F32, B * T + C, True), n
    # a step of exactly 0 keeps it
    q = {n: d[n][:, :1].contiguous() for n in ("x", "dt", "b", "c")}
    q["dt"].fill_(-float("inf"))
    _, _, hT = L.ssm_fwd(q["x"], q["dt"], d["A"], q["b"], q["c"], h0=d["h0"], want_ckpt=False)
    state = d["h0"].clone()
    L.ssm_step(q["x"], q["dt"], d["A"], q["b"], q["c"], state)
    torch.cuda.synchronize()
    assert torch.equal(hT, d["h0"]) and torch.equal(state, d["h0"])


def test_positions_near_2_to_31():
    """As many tokens as positions of 32 bits have room for: the ends of segments lie below 2^31 as the sequence's does.  All
    tokens are alike, so y has its limit everywhere but at a sequence's first tokens."""
    note("ssm 2^31 tokens")
    T, S = 2 ** 31 - 1100, 16
    one, b = torch.ones(1, T, 1, dtype=BF, device=DEV), torch.ones(1, T, 1, S, dtype=BF, device=DEV)
    A = -torch.ones(1, S, device=DEV)
    y = torch.empty(1, T, 1, dtype=BF, device=DEV)
    # h = e^-1 h + 1: 1 / (1 - 1 / e) from the 40th token on.  S times that is 25.31163, 580 E of itself from where bf16 rounds
    # the other way (25.3125); the factor's 3 E and the update's 2 leave 5 E of h, the sum of S terms another 16.
    h = 1 / (1 - torch.exp(torch.tensor(-1.0, dtype=torch.float64)))
    want = (S * h).to(BF).item()
    for cu in (None, [0, T - 5, T]):
        y.fill_(float("nan"))
        cut = None if cu is None else torch.tensor(cu, dtype=torch.int32, device=DEV)
        _, _, hT = L.ssm_fwd(one, one, A, b, b, softplus=False, cu_seqlens=cut, y=y, want_ckpt=False)
        torch.cuda.synchronize()
        end = T if cu is None else T - 5
        assert (y[0, 40:end] == want).all() and (y[0, :40] <= want).all()
        assert y[0, 0] == S and (cu is None or y[0, T - 5] == S)
        assert rel(hT[0], h.expand(1, S)) <= scan_tol(40, S, F32)


def test_gates_in_rows_of_fp32():
    """A gate that is a slice of fp32 rows, each at a multiple of 16 bytes, their distance no multiple of eight values."""
    note("rn fp32 gate slice")
    gen = torch.Generator().manual_seed(4)
    rows, C = 30, 64
    o, res, dr, dh = (torch.randn(rows, C, generator=gen).to(DEV) for _ in range(4))
    wide = torch.randn(rows, C + 20, generator=gen).to(DEV)
    gate = wide[:, 4:4 + C]
    assert gate.stride(0) % 8 and gate.data_ptr() % 16 == 0
    kw = dict(norm="rms", norm2="rms")
    got, want = (L.rn_fwd(o, g, res, **kw) for g in (gate, gate.contiguous()))
    grads = [L.rn_bwd(dr, dh, o, g, res, want[2], **kw)[:3] for g in (gate, gate.contiguous())]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip((*got, *grads[0]), (*want, *grads[1])))


# ------------------------------------------------------------------ launches that the smaller tests do not reach
def step_ref(p, pool, slots):
    """Rows one after the other from the definition, on the GPU: y and the pool."""
    pool = pool.double()
    p = {n: None if t is None else t.to(DEV).double() for n, t in p.items()}
    y = torch.zeros(p["x"].shape, dtype=torch.float64, device=DEV)
    for r, s in enumerate(slots):
        if 0 <= s < pool.shape[0]:
            row = {n: p[n] if n in ("A", "D", "dt_bias") or p[n] is None else p[n][r:r + 1] for n in INS}
            y[r:r + 1], h = ref_scan(dict(row, h0=pool[s:s + 1]))
            pool[s] = h[0]
    return y, pool


MANY = [(300, 1, 449, 16, 1), (150, 1, 465, 32, 1), (140, 1, 247, 64, 1), (300, 2, 448, 16, 7), (140, 3, 256, 64, 4),
        (160, 1, 448, 32, 7), (2048, 1, 5, 16, 1)]


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("B,T,C,S,G", MANY)
def test_steps_of_many_rows(B, T, C, S, G, dtype):
    """From 2048 workgroups on a wave has four times the channels: the last of them missing, several groups, several tokens."""
    note(f"ssm step of many rows B{B} T{T} C{C} S{S} G{G} {dtype}")
    assert B * -(-C * S // 1024) >= 2048
    p = make_scan(B, T, C, S, G, dtype, seed=B + C)
    d = {n: None if t is None else t.to(DEV) for n, t in p.items()}
    state = d["h0"].clone()
    y = L.ssm_step(d["x"], d["dt"], d["A"], d["b"], d["c"], state, d["D"], d["z"], dt_bias=d["dt_bias"])
    plain = d["h0"].clone()                                # no z, D or bias; another pool for the results
    out = torch.full_like(plain, 7.0)
    y0 = L.ssm_step(d["x"], d["dt"], d["A"], d["b"], d["c"], plain, state_out=out)
    torch.cuda.synchronize()
    v = {n: d[n].double() for n in INS}
    for (a, h), w in (((y, state), v), ((y0, out), dict(v, z=None, D=None, dt_bias=None))):
        wy, wh = ref_scan(w)
        assert rel(a, wy) <= scan_tol(T, S, dtype) and rel(h, wh) <= scan_tol(T, S, F32)
    assert torch.equal(plain, d["h0"])


@pytest.mark.parametrize("dtype,C,S,T", [(F32, 449, 16, 1), (BF, 247, 64, 2)])
def test_steps_of_many_rows_in_a_pool(dtype, C, S, T):
    """Slots in any order, padding whose inputs are NaN, repeated slots, all inputs slices at odd places; into the pool
    and into another one."""
    note(f"ssm step of many rows, slots C{C} S{S} {dtype}")
    B, P = 300, 310
    gen = torch.Generator().manual_seed(8)
    p = make_scan(B, T, C, S, 1, dtype, seed=18)
    slots = torch.randperm(P, generator=gen)[:B]
    slots[17], slots[120], slots[299] = slots[3], slots[3], slots[200]
    slots[50], slots[51], slots[298] = -1, P, 2 ** 31 - 1
    for n in ("x", "dt", "b", "c", "z"):
        p[n][50:52], p[n][298] = float("nan"), float("nan")
    d = {n: None if t is None else t.to(DEV) for n, t in p.items()}
    for n, off in (("x", 1), ("dt", 3), ("z", 5), ("b", 7), ("c", 1)):
        t = d[n].flatten(2)
        buf = torch.full((B, T, t.shape[2] + off + 2), float("nan"), dtype=dtype, device=DEV)
        buf[..., off:off + t.shape[2]] = t
        d[n] = buf[..., off:off + t.shape[2]].unflatten(-1, d[n].shape[2:])
    pool = torch.randn(P, C, S, generator=gen).to(DEV)
    wy, want = step_ref(p, pool, slots.tolist())
    ids = slots.to(torch.int32).to(DEV)
    nxt, before = torch.full_like(pool, 7.0), pool.clone()
    step = lambda **kw: L.ssm_step(d["x"], d["dt"], d["A"], d["b"], d["c"], pool, d["D"], d["z"], dt_bias=d["dt_bias"],  # noqa: E731
                                   slots=ids, **kw)
    y = step(state_out=nxt)
    torch.cuda.synchronize()
    assert torch.equal(pool, before)
    used = sorted({s for s in slots.tolist() if 0 <= s < P})
    rest = [s for s in range(P) if s not in used]
    assert rel(y, wy) <= scan_tol(3 * T, S, dtype) and (y[[50, 51, 298]] == 0).all()
    assert rel(nxt[used], want[used]) <= scan_tol(3 * T, S, F32) and (nxt[rest] == 7).all()
    y2 = step()
    torch.cuda.synchronize()
    assert torch.equal(y2, y) and torch.equal(pool[used], nxt[used]) and torch.equal(pool[rest], before[rest])


@pytest.mark.parametrize("B,T,C,S,dtype", [(2, 130, 16801, 16, F32), (1, 129, 8501, 64, BF), (3, 150, 6001, 32, BF)])
def test_gradients_in_two_segments(B, T, C, S, dtype):
    """Between 2 and 3 waves per SIMD the gradient goes by two segments, the forward by one."""
    note(f"ssm two segments B{B} T{T} C{C} S{S} {dtype}")
    assert 2048 < B * -(-C // 16) * (S // 16) <= 3 * 1024
    check_scan(make_scan(B, T, C, S, 1, dtype, seed=T), ref_on=DEV)


@pytest.mark.parametrize("N,C,S,dtype", [(17, 4090, 16, BF), (17, 1024, 64, F32), (9, 4096, 16, F32)])
def test_many_packed_sequences_in_quarters(N, C, S, dtype):
    """Where packed sequences are enough to fill the chip only those of more than a quarter of all tokens are cut."""
    note(f"ssm packed quarters N{N} C{C} S{S} {dtype}")
    waves = N * -(-C // 16) * (S // 16)
    assert waves > 2048 and (waves > 4096 or N == 9)
    lens = [3, 0, 231, 1, 16, 17] + [5] * (N - 7) + [40]
    cu = [2]
    for n in lens:
        cu.append(cu[-1] + n)
    check_scan(make_scan(1, cu[-1] + 4, C, S, 1, dtype, seed=N, N=N), cu=cu, ref_on=DEV)


@pytest.mark.parametrize("rows,C,groups,od,iod,rd", [
    (17001, 96, 1, F32, F32, F32), (9001, 500, 1, BF, BF, BF), (4003, 2048, 32, F32, BF, BF), (1201, 3001, 1, F32, F32, F32),
    (1500, 8184, 1, BF, BF, F32)])
def test_weights_of_norms_over_many_rows(rows, C, groups, od, iod, rd):
    """More rows than the gradient has teams for twice: a team adds up several, and not all of them equally many."""
    note(f"rn many rows {rows} x {C} {od} {iod} {rd}")
    check_rn(make_rn(rows, C, od, iod, rd, F32, seed=C), groups, norm2="rms")


@pytest.mark.parametrize("B,T,C,S,G,dtype", [(1, 300, 40, 16, 1, BF), (2, 200, 128, 32, 2, F32), (1, 300, 70, 64, 1, BF)])
def test_slices_in_several_segments(B, T, C, S, G, dtype):
    """As slices at odd places of wider rows, what is not theirs being NaN, in sequences of several segments."""
    note(f"ssm slices in segments B{B} T{T} C{C} S{S} {dtype}")
    p = {n: None if t is None else t.to(DEV) for n, t in make_scan(B, T, C, S, G, dtype, seed=30).items()}
    wide = dict(p)
    for n, off in (("x", 1), ("dt", 3), ("z", 7), ("b", 5), ("c", 0)):
        t = p[n].flatten(2)
        buf = torch.full((B, T, t.shape[2] + off + 3), float("nan"), dtype=dtype, device=DEV)
        buf[..., off:off + t.shape[2]] = t
        wide[n] = buf[..., off:off + t.shape[2]].unflatten(-1, p[n].shape[2:])
    got = []
    for q in (p, wide):
        ins = [q[n] for n in ("x", "dt", "A", "b", "c")]
        y, ckpt, hT = L.ssm_fwd(*ins, q["D"], q["z"], q["h0"], dt_bias=q["dt_bias"])
        got.append([y, hT, *L.ssm_bwd(q["dy"], *ins, ckpt, q["D"], q["z"], q["dhT"], dt_bias=q["dt_bias"])])
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(*got))


@pytest.mark.parametrize("C,dtype", [(1024, BF), (1029, BF), (1001, F32)])
def test_convolution_of_slices_by_vectors(C, dtype):
    """Vectors of channels at odd addresses: slices of wider rows, filters and biases in bf16 behind an odd value."""
    note(f"conv slices by vectors C{C} {dtype}")
    T, W = 9000, 4
    p = {n: None if t is None else t.to(DEV) for n, t in make_conv(1, T, C, W, dtype, seed=31, wdtype=BF).items()}
    odd = dict(p)
    buf = torch.full((1, T, C + 5), float("nan"), dtype=dtype, device=DEV)
    buf[..., 3:3 + C] = p["x"]
    odd["x"] = buf[..., 3:3 + C]
    for n in ("weight", "bias"):
        flat = torch.full((p[n].numel() + 1,), float("nan"), dtype=BF, device=DEV)
        flat[1:] = p[n].flatten()
        odd[n] = flat[1:].view(p[n].shape)
    got = []
    for q in (p, odd):
        y, hT = L.conv_fwd(q["x"], q["weight"], q["bias"], q["h0"])
        got.append([y, hT, *L.conv_bwd(q["dy"], q["x"], q["weight"], q["bias"], q["h0"], q["dhT"])])
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(*got))


def test_broadcast_inputs_and_gradients():
    """Inputs that are one value for many rows or channels, and gradients that are (a sum's): as their dense copies give."""
    note("mix: broadcast")
    B, T, C, S = 2, 21, 64, 16
    p = {n: None if t is None else t.to(DEV) for n, t in make_scan(B, T, C, S, 1, F32, seed=32).items()}
    thin = {"x": p["x"], "dt": p["dt"][:, :, :1], "b": p["b"][:, :1], "z": p["z"][:1], "A": p["A"][:1]}
    full = {"x": (B, T, C), "dt": (B, T, C), "b": (B, T, 1, S), "z": (B, T, C), "A": (C, S)}
    w, o = torch.randn(C, 4, generator=torch.Generator().manual_seed(1)).to(DEV), torch.ones(C, device=DEV)

    def layer(dense):
        leaves = {n: t.clone().requires_grad_() for n, t in thin.items()}
        v = {n: t.expand(full[n]) for n, t in leaves.items()}
        if dense:
            v = {n: t.contiguous() for n, t in v.items()}
        x, _ = L.CONV.apply(v["x"], w, None)
        y, hT = L.SSM.apply(x, v["dt"], v["A"], v["b"], p["c"], o, v["z"])
        r, h = L.RN.apply(y, v["z"], v["x"], o, None, None, o, None, dict(norm="rms", norm2="rms"))
        (r.sum() + h.sum() + hT.sum()).backward()
        return [r, h, *(t.grad for t in leaves.values())]

    for a, b in zip(layer(False), layer(True)):
        assert torch.equal(a, b) and torch.isfinite(a).all()


@pytest.mark.parametrize("lo,hi", SPANS)
def test_slopes_keep_their_bits(lo, hi):
    """The gradient of a raw step alone: one token, no decay, x = b = c = dy = 1, so ddt is S times the step's slope, of which S
    and the sum are exact and one rounding is added."""
    note(f"mix: slope {lo} {hi}")
    v = spread(lo, hi, 1 << 16).float().view(1, 1, -1)
    C = v.shape[2]
    one, b = torch.ones(1, 1, C, device=DEV), torch.ones(1, 1, 1, 16, device=DEV)
    ins = (one, v.to(DEV), torch.zeros(C, 16, device=DEV), b, b)
    _, ckpt, _ = L.ssm_fwd(*ins)
    ddt = L.ssm_bwd(one, *ins, ckpt)[1]
    torch.cuda.synchronize()
    want = 16 * torch.sigmoid(v.double())
    err = ((ddt.double().cpu() - want).abs() / want).max().item()
    assert err <= 9 * E, (lo, hi, err / E)

"""What the selective scan, its short convolution and the fused block norm are measured on.

Six kinds of call, in plain torch where `own` is false and through the
package's entry points where it is true:

  scan        ssm_fwd              outputs and final states of whole prompts
  scan_train  ssm_fwd + ssm_bwd    a training step's outputs and gradients
  scan_step   ssm_step             one or a few new tokens per sequence, states in a pool
  conv        conv_fwd             the causal convolution over prompts
  conv_train  conv_fwd + conv_bwd  with its gradients
  conv_step   conv_step            new tokens, the last inputs of every sequence in a pool
  norm        rn_fwd (+ rn_bwd)    norm, gate, scaled residual and the next norm, with gradients

Definitions.  Selective scan: per channel S states h; token t with input x, step
delta = softplus(dt + dt_bias), A (per channel and state), b and c (S each, shared
by the channels of a group):

    h <- exp(delta A) h + delta x b;  y = (sum_s c_s h_s + D x) silu(z)

Convolution over W tokens, x before a sequence's first token being its state:

    y_t = silu(bias + sum_j w_j x_(t - W + 1 + j))

Block norm, over rows of C channels, norm1 over each of `groups` equal parts:

    r = res + scale act(gate) (norm1(o) w1 + b1);  h = norm2(r) w2 + b2
"""
import math
import random

import torch

own = False

CHUNK = 64
EPS1, EPS2 = 64e-5, 1e-5
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # a serving batch of prompts of many lengths in one row, some continuing from a state; a wide state
        dict(name="scan_packed", op="scan", B=1, T=8193, C=2048, S=64, G=4, dtype="bf16", packed=17, h0=True, z=False),
        # one long document through the widest layer: few channels for the chip, many tokens in a row
        dict(name="scan_long", op="scan", B=1, T=16384, C=4096, S=16, G=1, dtype="bf16", packed=0, h0=False, z=True),
        # the 36M training layer's batch: 12 rows of 1024 tokens, 384 channels expanded twofold
        dict(name="scan_train_36m", op="scan_train", B=12, T=1024, C=768, S=16, G=1, dtype="bf16", packed=0, h0=False,
             z=True),
        # a 1.5B-class training layer: 4096 tokens, 2048 channels expanded twofold
        dict(name="scan_train_1b5", op="scan_train", B=4, T=4096, C=4096, S=16, G=1, dtype="bf16", packed=0, h0=False,
             z=True),
        # fp32, packed sequences of odd lengths that carry their states, several groups
        dict(name="scan_train_fp32", op="scan_train", B=1, T=999, C=320, S=32, G=5, dtype="fp32", packed=6, h0=True,
             z=True),
        # a decoding step of a large batch
        dict(name="step_batch", op="scan_step", B=256, T=1, C=4096, S=16, G=1, dtype="bf16", pool=0, z=True),
        # a few chat sequences out of a pool of states: latency
        dict(name="step_few", op="scan_step", B=5, T=1, C=2048, S=16, G=1, dtype="bf16", pool=16, z=True),
        # the convolution of the 1.5B-class layer, with its gradients
        dict(name="conv_train_1b5", op="conv_train", B=8, T=4096, C=4096, W=4, dtype="bf16", packed=0, h0=False,
             bias=True),
        # prompts of many lengths in one row, continuing from their last inputs
        dict(name="conv_packed", op="conv", B=1, T=12289, C=2048, W=4, dtype="bf16", packed=23, h0=True, bias=True),
        # the convolution's part of a decoding step
        dict(name="conv_step", op="conv_step", B=256, T=1, C=4096, W=4, dtype="bf16", pool=300, bias=True),
        # the end of a time mix while decoding: gated root-mean-square norm, residual, next norm
        dict(name="norm_decode", op="norm", rows=256, C=4096, groups=1, dtype="bf16", odtype="bf16", rdtype="bf16",
             norm="rms", norm2="rms", gate="silu", res=True, scale=False, grad=False),
        # the end of a time mix in the 1.5B-class layer: per-head norm of the fp32 output, gate, scaled residual, norm
        dict(name="norm_train_1b5", op="norm", rows=32768, C=2048, groups=32, dtype="bf16", odtype="fp32",
             rdtype="bf16", norm="layer", norm2="layer", gate="sigmoid", res=True, scale=True, grad=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["scan", "scan_train", "scan_step", "conv", "conv_train", "conv_step", "norm"])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    if op == "norm":
        groups, C = rng.choice([(1, _log(rng, 8, 8192)), (rng.randint(2, 32), 0)])
        C = C or groups * rng.choice([64, 64, 128, 256])
        rows = _log(rng, 1, max(2, min(30000, 30_000_000 // C)))
        res = rng.random() < 0.7
        return dict(op=op, rows=rows, C=C, groups=groups, dtype=dtype, odtype=rng.choice([dtype, dtype, "fp32"]),
                    rdtype=rng.choice([dtype, "fp32"]), norm=rng.choice(["layer", "rms"]),
                    norm2=rng.choice(["layer", "rms", None]), gate=rng.choice(["silu", "sigmoid", None]), res=res,
                    scale=rng.random() < 0.5, grad=rng.random() < 0.6)
    if op in ("scan_step", "conv_step"):
        B, C = _log(rng, 1, 300), _log(rng, 16, 5000)
        case = dict(op=op, B=B, T=rng.choice([1, 1, 1, 2, 3, 5]), C=C, dtype=dtype,
                    pool=rng.choice([0, B + rng.randint(0, 8)]))
        if op == "conv_step":
            return dict(case, W=rng.choice([2, 3, 4, 4]), bias=rng.random() < 0.7)
        S = rng.choice([16, 16, 32, 64])
        if rng.random() < 0.3:
            case.update(C=64 * rng.randint(2, 40), G=2)
            case["C"] -= case["C"] % 128
        return dict(case, S=S, G=case.get("G", 1), z=rng.random() < 0.6)
    C = _log(rng, 16, 4096)
    most = 30_000_000 // C
    if op in ("conv", "conv_train"):
        case = dict(W=rng.choice([2, 3, 4, 4]), bias=rng.random() < 0.7)
    else:
        case = dict(S=rng.choice([16, 16, 32, 64]), G=1, z=rng.random() < 0.6)
        if rng.random() < 0.3:
            case["G"] = rng.randint(2, 6)
            C = case["G"] * 64 * rng.randint(1, 6)
        most = (250_000_000 if op == "scan" else 80_000_000) // (C * case["S"])
    tokens = _log(rng, 2, max(3, min(12000, most)))
    packed = 0
    if rng.random() < 0.5:
        packed, B, T = rng.randint(1, max(2, min(40, tokens // 8))), 1, tokens
    else:
        B = rng.randint(1, min(8, tokens))
        T = max(1, tokens // B)
    return dict(op=op, B=B, T=T, C=C, dtype=dtype, packed=packed, h0=rng.random() < 0.5, **case)


def _lengths(T, n, seed):
    """n sequence lengths with sum T, uneven; the second one is empty where there are three or more."""
    r = random.Random(seed * 7919 + T)
    w = [0.05 + r.random() ** 2 for _ in range(n)]
    if n >= 3:
        w[1] = 0.0
    cuts, s, tot = [0], 0.0, sum(w)
    for x in w:
        s += x
        cuts.append(int(round(T * s / tot)))
    cuts[-1] = T
    return cuts


# ------------------------------------------------------------------ the inputs
def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=gen, device=dev)  # noqa: E731
    dt = DT[case["dtype"]]
    st = dict(case=case)
    if case["op"] == "norm":
        R, C = case["rows"], case["C"]
        w = lambda a: (a + 0.1 * rn(C))  # noqa: E731
        st["o"] = (rn(R, C) * torch.exp(0.5 * rn(R, 1)) + 0.3 * rn(1, C)).to(DT[case["odtype"]])
        st["gate"] = rn(R, C).to(dt) if case["gate"] else None
        st["res"] = (2.0 * rn(R, C)).to(DT[case["rdtype"]]) if case["res"] else None
        st["weight"], st["bias"] = w(1.0), w(0.0) if case["norm"] == "layer" else None
        st["scale"] = w(0.5) if case["scale"] else None
        st["weight2"] = w(1.0) if case["norm2"] else None
        st["bias2"] = w(0.0) if case["norm2"] == "layer" else None
        if case["grad"]:
            st["dr"] = rn(R, C).to(DT[case["rdtype"]] if case["res"] else dt)
            st["dh"] = rn(R, C).to(dt) if case["norm2"] else None
        return st
    B, T, C = case["B"], case["T"], case["C"]
    # what a layer's first projection gives: the mix's input and its gate, side by side
    xz = rn(B, T, 2 * C)
    step = case["op"].endswith("_step")
    N = B
    if step:
        P = case["pool"] or B
        st["slots"] = None
        if case["pool"]:
            at = list(range(P))
            random.Random(seed).shuffle(at)
            st["slots"] = torch.tensor(at[:B], dtype=torch.int32, device=dev)
    else:
        st["cu"], st["longest"] = None, T
        if case["packed"]:
            N = case["packed"]
            cuts = _lengths(T, N, seed)
            st["cu"] = torch.tensor(cuts, dtype=torch.int32, device=dev)
            st["longest"] = max(b - a for a, b in zip(cuts, cuts[1:]))
    if case["op"].startswith("conv"):
        W = case["W"]
        st["x"] = xz.to(dt)[..., :C]
        st["weight"] = rn(C, W) * W ** -0.5
        st["bias"] = 0.1 * rn(C) if case["bias"] else None
        if step:
            st["state"] = rn(P, W - 1, C).to(dt)
            st["next"] = torch.zeros_like(st["state"])
            return st
        st["h0"] = rn(N, W - 1, C).to(dt) if case["h0"] else None
        if case["op"] == "conv_train":
            st["dy"] = rn(B, T, C).to(dt)
            st["dhT"] = rn(N, W - 1, C).to(dt) if case["h0"] else None
        return st
    S, G = case["S"], case["G"]
    xz[..., :C] = torch.nn.functional.silu(xz[..., :C])
    xz = xz.to(dt)
    st["x"] = xz[..., :C].contiguous()                     # the convolution's output
    st["z"] = xz[..., C:] if case["z"] else None
    # what the second projection gives: a low-rank step, b and c side by side
    R = max(1, C // 16)
    p = rn(B, T, R + 2 * G * S).to(dt)
    st["b"], st["c"] = (p[..., R + i * G * S:R + (i + 1) * G * S].unflatten(-1, (G, S)) for i in (0, 1))
    st["dt"] = (0.5 * rn(B, T, C)).to(dt)
    size = torch.exp(torch.empty(C, device=dev).uniform_(math.log(1e-3), math.log(1e-1), generator=gen))
    st["dt_bias"] = size + torch.log(-torch.expm1(-size))  # softplus of it is `size`
    st["A"] = -torch.arange(1, S + 1, device=dev).float() * torch.exp(0.2 * rn(C, S))
    st["D"] = 1 + 0.1 * rn(C)
    if step:
        st["state"] = 0.3 * rn(P, C, S)
        st["next"] = torch.zeros_like(st["state"])
        return st
    st["h0"] = 0.3 * rn(N, C, S) if case["h0"] else None
    if case["op"] == "scan_train":
        st["dy"] = rn(B, T, C).to(dt)
        st["dhT"] = 0.3 * rn(N, C, S) if case["h0"] else None
    return st


# ------------------------------------------------------------------ one pass
def run(st):
    op = st["case"]["op"]
    if op == "norm":
        return _run_norm(st)
    kind, _, rest = op.partition("_")
    return {"scan": {"": _run_scan, "train": _run_scan_train, "step": _run_scan_step},
            "conv": {"": _run_conv, "train": _run_conv_train, "step": _run_conv_step}}[kind][rest](st)


def _run_scan(st):
    if own:
        import linear_rnn_lm_amd as L
        y, _, hT = L.ssm_fwd(st["x"], st["dt"], st["A"], st["b"], st["c"], st["D"], st["z"], st["h0"],
                             dt_bias=st["dt_bias"], cu_seqlens=st["cu"], want_ckpt=False)
        return y, hT
    y, hT = _plain_scan(st, *_scan_floats(st))
    return y.to(st["x"].dtype), hT


def _run_scan_train(st):
    if own:
        import linear_rnn_lm_amd as L
        ins = (st["x"], st["dt"], st["A"], st["b"], st["c"])
        more = dict(dt_bias=st["dt_bias"], cu_seqlens=st["cu"])
        y, ckpt, hT = L.ssm_fwd(*ins, st["D"], st["z"], st["h0"], **more)
        return y, hT, *L.ssm_bwd(st["dy"], *ins, ckpt, st["D"], st["z"], st["dhT"], want_dh0=st["h0"] is not None, **more)
    dt = st["x"].dtype
    leaves = [None if t is None else t.detach().requires_grad_() for t in _scan_floats(st)]
    with torch.enable_grad():
        y, hT = _plain_scan(st, *leaves)
        outs, cots = [y], [st["dy"].float()]
        if st["dhT"] is not None:
            outs.append(hT)
            cots.append(st["dhT"])
        got = iter(torch.autograd.grad(outs, [t for t in leaves if t is not None], cots))
    dx, ddt, dA, db, dc, dD, dz, dbias, dh0 = (None if t is None else next(got) for t in leaves)
    return (y.detach().to(dt), hT.detach(), dx.to(dt), ddt.to(dt), dA, db.to(dt), dc.to(dt), dD,
            None if dz is None else dz.to(dt), dbias, dh0)


def _run_scan_step(st):
    if own:
        import linear_rnn_lm_amd as L
        y = L.ssm_step(st["x"], st["dt"], st["A"], st["b"], st["c"], st["state"], st["D"], st["z"],
                       dt_bias=st["dt_bias"], slots=st["slots"], state_out=st["next"])
        return y, st["next"]
    x, dt, A, b, c, D, z, bias, _ = _scan_floats(st)
    C = x.shape[-1]
    rep = C // b.shape[2]
    at = slice(None) if st["slots"] is None else st["slots"].long()
    h = st["state"][at]
    delta = torch.nn.functional.softplus(dt + bias)
    y = torch.empty_like(x)
    for t in range(x.shape[1]):
        bt, ct = (m[:, t].repeat_interleave(rep, 1) for m in (b, c))
        h = torch.exp(delta[:, t, :, None] * A) * h + (delta[:, t] * x[:, t])[..., None] * bt
        y[:, t] = (h * ct).sum(-1) + D * x[:, t]
    if z is not None:
        y = y * z * torch.sigmoid(z)
    st["next"][at] = h
    return y.to(st["x"].dtype), st["next"]


def _run_conv(st):
    if own:
        import linear_rnn_lm_amd as L
        return L.conv_fwd(st["x"], st["weight"], st["bias"], st["h0"], cu_seqlens=st["cu"])
    y, hT = _plain_conv(st, *(None if st[n] is None else st[n].float() for n in ("x", "weight", "bias", "h0")))
    return y.to(st["x"].dtype), hT.to(st["x"].dtype)


def _run_conv_train(st):
    if own:
        import linear_rnn_lm_amd as L
        y, hT = L.conv_fwd(st["x"], st["weight"], st["bias"], st["h0"], cu_seqlens=st["cu"])
        return y, hT, *L.conv_bwd(st["dy"], st["x"], st["weight"], st["bias"], st["h0"], st["dhT"], cu_seqlens=st["cu"],
                                  want_dh0=st["h0"] is not None)
    dt = st["x"].dtype
    leaves = [None if st[n] is None else st[n].float().detach().requires_grad_() for n in ("x", "weight", "bias", "h0")]
    with torch.enable_grad():
        y, hT = _plain_conv(st, *leaves)
        outs, cots = [y], [st["dy"].float()]
        if st["dhT"] is not None:
            outs.append(hT)
            cots.append(st["dhT"].float())
        got = iter(torch.autograd.grad(outs, [t for t in leaves if t is not None], cots))
    dx, dw, db, dh0 = (None if t is None else next(got) for t in leaves)
    return y.detach().to(dt), hT.detach().to(dt), dx.to(dt), dw, db, None if dh0 is None else dh0.to(dt)


def _run_conv_step(st):
    if own:
        import linear_rnn_lm_amd as L
        y = L.conv_step(st["x"], st["weight"], st["bias"], st["state"], slots=st["slots"], state_out=st["next"])
        return y, st["next"]
    x, w = st["x"].float(), st["weight"]
    W, T = w.shape[1], x.shape[1]
    at = slice(None) if st["slots"] is None else st["slots"].long()
    ext = torch.cat([st["state"][at].float(), x], 1)
    y = sum(ext[:, j:j + T] * w[:, j] for j in range(W))
    if st["bias"] is not None:
        y = y + st["bias"]
    st["next"][at] = ext[:, T:].to(st["next"].dtype)
    return (y * torch.sigmoid(y)).to(st["x"].dtype), st["next"]


def _run_norm(st):
    case = st["case"]
    G, kw = case["groups"], dict(groups=case["groups"], norm=case["norm"], norm2=case["norm2"], act=case["gate"])
    ws = {n: st[n] for n in ("weight", "bias", "scale", "weight2", "bias2")}
    out_dt = DT[case["dtype"]]
    if own:
        import linear_rnn_lm_amd as L
        r, h, stats = L.rn_fwd(st["o"], st["gate"], st["res"], **ws, **kw, eps=EPS1, eps2=EPS2, out_dtype=out_dt,
                               want_stats=case["grad"])
        if not case["grad"]:
            return r, h
        return r, h, *L.rn_bwd(st["dr"], st["dh"], st["o"], st["gate"], st["res"], stats, **ws, **kw)
    o = st["o"].float()
    R, C = o.shape
    part = lambda t: t.view(R, G, C // G)  # noqa: E731

    def norm(v, kind, eps):
        vc = v - v.mean(-1, keepdim=True) if kind == "layer" else v
        rstd = torch.rsqrt((vc * vc).mean(-1, keepdim=True) + eps)
        return vc * rstd, rstd

    def norm_grad(e, vh, rstd, kind):
        e = e - vh * (e * vh).mean(-1, keepdim=True) - (e.mean(-1, keepdim=True) if kind == "layer" else 0.0)
        return e * rstd

    oh, rstd1 = norm(part(o), case["norm"], EPS1)
    oh = oh.reshape(R, C)
    u = oh * st["weight"] + (0.0 if st["bias"] is None else st["bias"])
    a = 1.0
    if case["gate"]:
        gate = st["gate"].float()
        sg = torch.sigmoid(gate)
        a = gate * sg if case["gate"] == "silu" else sg
    s = a * u
    r = s if st["scale"] is None else s * st["scale"]
    if case["res"]:
        r = r + st["res"].float()
    rdt = DT[case["rdtype"]] if case["res"] else out_dt
    h = None
    if case["norm2"]:
        rh, rstd2 = norm(r, case["norm2"], EPS2)
        h = rh * st["weight2"] + (0.0 if st["bias2"] is None else st["bias2"])
    outs = (r.to(rdt), None if h is None else h.to(out_dt))
    if not case["grad"]:
        return outs
    dr = st["dr"].float()
    dw2 = db2 = None
    if case["norm2"]:
        dh = st["dh"].float()
        dw2, db2 = (dh * rh).sum(0), dh.sum(0) if st["bias2"] is not None else None
        dr = dr + norm_grad(dh * st["weight2"], rh, rstd2, case["norm2"])
    ds = dr if st["scale"] is None else dr * st["scale"]
    dscale = None if st["scale"] is None else (dr * s).sum(0)
    du, dgate = ds * a, None
    if case["gate"]:
        slope = sg * (1 + gate * (1 - sg)) if case["gate"] == "silu" else sg * (1 - sg)
        dgate = (ds * u * slope).to(st["gate"].dtype)
    dw, db = (du * oh).sum(0), du.sum(0) if st["bias"] is not None else None
    do = norm_grad(part(du * st["weight"]), part(oh), rstd1, case["norm"]).reshape(R, C)
    return *outs, do.to(st["o"].dtype), dgate, dr.to(rdt) if case["res"] else None, dw, db, dscale, dw2, db2


# ------------------------------------------------------------------ plain forms over whole sequences
def _padded(st, x):
    """Packed sequences as a padded batch; padding is 0."""
    cu = st["cu"].long()
    at = cu[:-1, None] + torch.arange(st["longest"], device=x.device)
    ok = at < cu[1:, None]
    return x[0][at.clamp(max=x.shape[1] - 1)] * ok.view(*ok.shape, *([1] * (x.dim() - 2)))


def _unpadded(st, y, T):
    cu = st["cu"].long()
    pos = torch.arange(T, device=y.device)
    seq = torch.searchsorted(cu[1:], pos, right=True)
    return y[seq, pos - cu[seq]][None]


def _scan_floats(st):
    got = [st["x"], st["dt"], st["A"], st["b"], st["c"], st["D"], st["z"], st["dt_bias"], st.get("h0")]
    return [None if t is None else t.float() for t in got]


def _plain_scan(st, x, dt, A, b, c, D, z, bias, h0):
    """Chunks of 64 tokens: token by token inside all chunks at once, then the states from chunk to chunk.  Padding
    has a step of 0, which changes no state."""
    delta = torch.nn.functional.softplus(dt + bias)
    T = x.shape[1]
    packed = st["cu"] is not None
    xs, bs, cs, ds = (_padded(st, t) if packed else t for t in (x, b, c, delta))
    B, L, C = xs.shape
    NC = -(-L // CHUNK)
    G, S = b.shape[2:]

    def chunks(t):                       # (B, L, ...) -> (chunk length, B, NC, ...)
        t = torch.nn.functional.pad(t, (0, 0) * (t.dim() - 2) + (0, NC * CHUNK - L))
        return t.view(B, NC, CHUNK, *t.shape[2:]).movedim(2, 0)

    n = min(L, CHUNK)
    wide = lambda m: m.repeat_interleave(C // G, -2)  # noqa: E731
    xs, bs, cs, ds = chunks(xs), chunks(bs), chunks(cs), chunks(ds)
    us = ds * xs
    h = torch.zeros(B, NC, C, S, device=x.device)
    ys = []
    for t in range(n):
        h = torch.exp(ds[t][..., None] * A) * h + us[t][..., None] * wide(bs[t])
        ys.append((h * wide(cs[t])).sum(-1))
    total = ds.double().cumsum(0)                                       # sums of steps, in 64 bits
    over = torch.exp((total[n - 1][..., None] * A).float())
    state = torch.zeros(B, C, S, device=x.device) if h0 is None else h0
    entering = []
    for k in range(NC):
        entering.append(state)
        state = over[:, k] * state + h[:, k]
    entering = torch.stack(entering, 1)
    if NC > 1 or h0 is not None:
        ys = [y + (torch.exp((total[t][..., None] * A).float()) * entering * wide(cs[t])).sum(-1)
              for t, y in enumerate(ys)]
    y = torch.stack(ys, 2).reshape(B, NC * n, C)[:, :L]
    if packed:
        y = _unpadded(st, y, T)
    y = y + D * x
    if z is not None:
        y = y * z * torch.sigmoid(z)
    return y, state


def _plain_conv(st, x, w, bias, h0):
    T, C = x.shape[1:]
    W = w.shape[1]
    xs = _padded(st, x) if st["cu"] is not None else x
    N, L = xs.shape[:2]
    ext = torch.cat([torch.zeros(N, W - 1, C, device=x.device) if h0 is None else h0, xs], 1)
    y = sum(ext[:, j:j + L] * w[:, j] for j in range(W))
    if bias is not None:
        y = y + bias
    y = y * torch.sigmoid(y)
    if st["cu"] is None:
        return y, ext[:, L:]
    cu = st["cu"].long()
    last = (cu[1:] - cu[:-1])[:, None] + torch.arange(W - 1, device=x.device)
    return _unpadded(st, y, T), torch.gather(ext, 1, last[..., None].expand(-1, -1, C))


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "norm":
        n = case["rows"] * case["C"]
        eo, er = DT[case["odtype"]].itemsize, DT[case["rdtype"]].itemsize if case["res"] else e
        gate, res, h = e * bool(case["gate"]), er * case["res"], e * bool(case["norm2"])
        size = eo + gate + 2 * res + h if case["res"] else eo + gate + er + h
        if case["grad"]:                                   # dr and dh in; do, dgate and dres out
            size += er + h + eo + gate + res
        return {"bytes": n * size + 20 * case["C"], "flops": n * (60 if case["grad"] else 20)}
    n = case["B"] * case["T"] * case["C"]
    train = case["op"].endswith("_train")
    N = case.get("packed") or case["B"]
    if case["op"].startswith("conv"):
        W = case["W"]
        state = N * (W - 1) * case["C"] * e
        if case["op"] == "conv_step":
            return {"bytes": 2 * n * e + 2 * state + 4 * case["C"] * (W + 1), "flops": n * (2 * W + 4)}
        state *= 2 if case["h0"] else 1
        return {"bytes": (2 * n * e + state) * (2 if train else 1) + 4 * case["C"] * (W + 1),
                "flops": n * (2 * W + 4) * (4 if train else 1)}
    S, G = case["S"], case["G"]
    tokens = n * e * (4 if case["z"] else 3) + 2 * case["B"] * case["T"] * G * S * e
    state = N * case["C"] * S * 4
    if case["op"] == "scan_step":
        return {"bytes": tokens + 2 * state, "flops": n * (7 * S + 30)}
    state *= 2 if case["h0"] else 1
    return {"bytes": (tokens + state) * (2 if train else 1), "flops": n * (7 * S + 30) * (3 if train else 1)}


# ------------------------------------------------------------------ the definitions, token by token, in 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "norm":
        return _exact_norm(st)
    if case["op"].startswith("conv"):
        return _exact_conv(st)
    return _exact_scan(st)


def _spans(st, N):
    """(rows of the batch, tokens, sequences) that are worked on together."""
    if st["case"]["op"].endswith("_step") or st["cu"] is None:
        return [(slice(None), slice(0, st["case"]["T"]), slice(0, N))]
    cu = st["cu"].tolist()
    return [(slice(0, 1), slice(a, b), slice(n, n + 1)) for n, (a, b) in enumerate(zip(cu, cu[1:]))]


def _exact_scan(st):
    case = st["case"]
    x, dt, A, b, c, D = (st[n].double() for n in ("x", "dt", "A", "b", "c", "D"))
    bias, z = st["dt_bias"].double(), None if st["z"] is None else st["z"].double()
    B, T, C = x.shape
    G, S = b.shape[2:]
    v = dt + bias
    delta = torch.log1p(torch.exp(-v.abs())) + v.clamp(min=0)
    per = torch.arange(C, device=x.device) // (C // G)                 # the group of each channel
    train, step = case["op"] == "scan_train", case["op"] == "scan_step"
    N = B if step else case["packed"] or B
    if step:
        at = torch.arange(B, device=x.device) if st["slots"] is None else st["slots"].long()
        h0 = st["state"].double()[at]
    else:
        h0 = torch.zeros(N, C, S, dtype=torch.float64, device=x.device) if st["h0"] is None else st["h0"].double()
    if T * (3 if train else 1) > 60000:
        return None
    y, hT, kept = torch.zeros_like(x), h0.clone(), {}
    spans = _spans(st, N)
    for rows, ts, ns in spans:
        h = h0[ns]
        for t in range(ts.start, ts.stop):
            if train:
                kept[t, ns.start] = h
            h = torch.exp(delta[rows, t, :, None] * A) * h + (delta[rows, t] * x[rows, t])[..., None] * b[rows, t][:, per]
            y[rows, t] = (h * c[rows, t][:, per]).sum(-1)
        hT[ns] = h
    y = y + D * x
    gated = y if z is None else y * z / (1 + torch.exp(-z))
    if step:
        nxt = st["next"].double()
        nxt[at] = hT
        return gated, nxt
    if not train:
        return gated, hT
    dy = st["dy"].double()
    dz = None
    if z is not None:
        s = 1 / (1 + torch.exp(-z))
        dz = dy * y * s * (1 + z * (1 - s))
        dy = dy * z * s
    dx, ddelta, dA, dh0 = dy * D, torch.zeros_like(x), torch.zeros_like(A), torch.zeros_like(h0)
    db, dc = torch.zeros_like(b), torch.zeros_like(c)
    if st["dhT"] is not None:
        dh0 = st["dhT"].double().clone()
    for rows, ts, ns in spans:
        g = dh0[ns]
        for t in range(ts.stop - 1, ts.start - 1, -1):
            dl, xt, bt, ct = delta[rows, t], x[rows, t], b[rows, t][:, per], c[rows, t][:, per]
            a = torch.exp(dl[..., None] * A)
            ah = a * kept.pop((t, ns.start))
            h = ah + (dl * xt)[..., None] * bt
            g = g + ct * dy[rows, t][..., None]
            gb = (g * bt).sum(-1)
            dx[rows, t] += dl * gb
            p = g * ah
            ddelta[rows, t] = xt * gb + (p * A).sum(-1)
            dA += (p * dl[..., None]).sum(0)
            db[rows, t] = (g * (dl * xt)[..., None]).unflatten(1, (G, C // G)).sum(2)
            dc[rows, t] = (h * dy[rows, t][..., None]).unflatten(1, (G, C // G)).sum(2)
            g = a * g
        dh0[ns] = g
    ddt = ddelta / (1 + torch.exp(-v))
    return (gated, hT, dx, ddt, dA, db, dc, (dy * x).sum((0, 1)), dz, ddt.sum((0, 1)),
            dh0 if st["h0"] is not None else None)


def _exact_conv(st):
    case = st["case"]
    x, w = st["x"].double(), st["weight"].double()
    bias = 0.0 if st["bias"] is None else st["bias"].double()
    (B, T, C), W = x.shape, w.shape[1]
    step, train = case["op"] == "conv_step", case["op"] == "conv_train"
    N = B if step else case["packed"] or B
    if step:
        at = torch.arange(B, device=x.device) if st["slots"] is None else st["slots"].long()
        h0 = st["state"].double()[at]
    else:
        h0 = torch.zeros(N, W - 1, C, dtype=torch.float64, device=x.device) if st["h0"] is None else st["h0"].double()
    y, hT = torch.zeros_like(x), h0.clone()
    dx, dw, db, dh0 = torch.zeros_like(x), torch.zeros_like(w), torch.zeros_like(w[:, 0]), torch.zeros_like(h0)
    for rows, ts, ns in _spans(st, N):
        n = ts.stop - ts.start
        ext = torch.cat([h0[ns], x[rows, ts]], 1)
        s = torch.zeros_like(x[rows, ts]) + bias
        for j in range(W):
            s = s + w[:, j] * ext[:, j:j + n]
        sg = 1 / (1 + torch.exp(-s))
        y[rows, ts], hT[ns] = s * sg, ext[:, n:]
        if not train:
            continue
        ds = st["dy"].double()[rows, ts] * sg * (1 + s * (1 - sg))
        dext = torch.zeros_like(ext)
        if st["dhT"] is not None:
            dext[:, n:] = st["dhT"].double()[ns]
        for j in range(W):
            dext[:, j:j + n] += w[:, j] * ds
            dw[:, j] += (ds * ext[:, j:j + n]).sum((0, 1))
        db += ds.sum((0, 1))
        dh0[ns], dx[rows, ts] = dext[:, :W - 1], dext[:, W - 1:]
    if step:
        nxt = st["next"].double()
        nxt[at] = hT
        return y, nxt
    if not train:
        return y, hT
    return y, hT, dx, dw, db if st["bias"] is not None else None, dh0 if st["h0"] is not None else None


def _exact_norm(st):
    case = st["case"]
    names = ("o", "gate", "res", "weight", "bias", "scale", "weight2", "bias2")
    v = {n: None if st[n] is None else st[n].double().requires_grad_(case["grad"]) for n in names}

    def norm(t, kind, eps):
        if kind == "layer":
            var, mean = torch.var_mean(t, -1, correction=0, keepdim=True)
            return (t - mean) / torch.sqrt(var + eps)
        return t / torch.sqrt(t.square().mean(-1, keepdim=True) + eps)

    with torch.set_grad_enabled(case["grad"]):
        r = norm(v["o"].unflatten(-1, (case["groups"], -1)), case["norm"], EPS1).flatten(1) * v["weight"]
        if v["bias"] is not None:
            r = r + v["bias"]
        if case["gate"]:
            r = r / (1 + torch.exp(-v["gate"])) * (v["gate"] if case["gate"] == "silu" else 1.0)
        if v["scale"] is not None:
            r = r * v["scale"]
        if v["res"] is not None:
            r = r + v["res"]
        h = None
        if case["norm2"]:
            h = norm(r, case["norm2"], EPS2) * v["weight2"]
            if v["bias2"] is not None:
                h = h + v["bias2"]
    if not case["grad"]:
        return r, h
    outs, cots = [r], [st["dr"].double()]
    if h is not None:
        outs.append(h)
        cots.append(st["dh"].double())
    leaves = [t for t in v.values() if t is not None]
    got = dict(zip([n for n in names if v[n] is not None], torch.autograd.grad(outs, leaves, cots)))
    return (r.detach(), None if h is None else h.detach(), *(got.get(n) for n in names))

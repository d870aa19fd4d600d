"""What the gated delta rule and the layer norm are measured on.

Four kinds of call, in plain torch where `own` is false and through the
package's entry points where it is true:

  prefill  gdr_fwd             outputs and final state of whole prompts
  train    gdr_fwd + gdr_bwd   a training step's outputs and gradients
  step     gdr_step            one or a few new tokens per sequence, states in a pool
  norm     ln_fwd (+ ln_bwd)   layer norm, or one norm per head, with its gradients

Definitions.  Per value head with state S (V x K), token t with q, k (K), v (V),
log decay g and write strength beta; q and k of H / Hk neighbouring value heads are shared:

    S <- e^g S;  u = beta (v - S k);  S <- S + u k^T;  o = scale S q

Layer norm over each of `groups` equal parts of the C channels of a row:
y = (x - mean) / sqrt(var + eps) * weight + bias.
"""
import math
import random

import torch

own = False

CHUNK = 64
EPS = 1e-5
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # a short prompt for a small model: what one call costs
        dict(name="prefill_short", op="prefill", B=1, T=61, Hk=4, H=4, K=64, V=64, dtype="bf16", packed=0, h0=False),
        # a serving batch of prompts of many lengths, packed, some of them continuing from a state
        dict(name="prefill_packed", op="prefill", B=1, T=12289, Hk=16, H=32, K=128, V=128, dtype="bf16", packed=23,
             h0=True),
        # one long document: few heads, many chunks in a row
        dict(name="prefill_long", op="prefill", B=1, T=32768, Hk=16, H=32, K=128, V=128, dtype="bf16", packed=0,
             h0=False),
        # the 36M training layer: batch 12, 1024 tokens, 6 heads of 64
        dict(name="train_36m", op="train", B=12, T=1024, Hk=6, H=6, K=64, V=64, dtype="bf16", packed=0, h0=False),
        # the 1.5B-class training layer: batch 8, 4096 tokens, 32 heads of 64, with a state carried in
        dict(name="train_1b5", op="train", B=8, T=4096, Hk=32, H=32, K=64, V=64, dtype="bf16", packed=0, h0=True),
        # packed training sequences, heads of 128, two value heads to a key head
        dict(name="train_packed", op="train", B=1, T=8200, Hk=8, H=16, K=128, V=128, dtype="bf16", packed=9, h0=True),
        # fp32 inputs, an odd length, key and value heads of different sizes
        dict(name="train_fp32", op="train", B=3, T=333, Hk=2, H=4, K=64, V=128, dtype="fp32", packed=0, h0=True),
        # one recurrent step of a 7B-class layer, batch 256, 64 heads of 64
        dict(name="step_7b", op="step", B=256, T=1, Hk=64, H=64, K=64, V=64, dtype="bf16", pool=0),
        # a few chat sequences out of a pool of states: latency
        dict(name="step_few", op="step", B=5, T=1, Hk=16, H=32, K=128, V=128, dtype="bf16", pool=16),
        # the norm in front of a layer while decoding
        dict(name="norm_decode", op="norm", rows=256, C=4096, groups=1, dtype="bf16", wdtype="bf16", grad=False),
        # the norm of the 36M training layer, with its gradients
        dict(name="norm_train_36m", op="norm", rows=12288, C=384, groups=1, dtype="bf16", wdtype="fp32", grad=True),
        # the per-head norm of the recurrence's output in the 1.5B-class layer, with its gradients
        dict(name="norm_heads_1b5", op="norm", rows=32768, C=2048, groups=32, dtype="bf16", wdtype="bf16", grad=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["prefill", "train", "step", "norm"])
    if op == "norm":
        groups, C = rng.choice([(1, _log(rng, 64, 8192)), (rng.randint(2, 48), 0)])
        C = C or groups * rng.choice([32, 64, 64, 128])
        rows = _log(rng, 1, max(2, min(40000, 60_000_000 // C)))
        return dict(op=op, rows=rows, C=C, groups=groups, dtype=rng.choice(["bf16", "bf16", "fp32"]),
                    wdtype=rng.choice(["bf16", "fp32"]), grad=rng.random() < 0.6)
    Hk = rng.randint(1, 16)
    H = Hk * rng.choice([1, 1, 2, 3])
    K, V = rng.choice([(64, 64), (128, 128), (64, 128), (128, 64)])
    dtype = rng.choice(["bf16", "bf16", "bf16", "fp32"])
    if op == "step":
        B = _log(rng, 1, 200)
        return dict(op=op, B=B, T=rng.choice([1, 1, 1, 2, 3, 5]), Hk=Hk, H=H, K=K, V=V, dtype=dtype,
                    pool=rng.choice([0, B + rng.randint(0, 8)]))
    tokens = _log(rng, 20, 12000 if op == "prefill" else 5000)
    if rng.random() < 0.5:
        return dict(op=op, B=1, T=tokens, Hk=Hk, H=H, K=K, V=V, dtype=dtype,
                    packed=rng.randint(1, max(2, min(40, tokens // 8))), h0=rng.random() < 0.5)
    B = rng.randint(1, min(8, max(1, tokens // 16)))
    return dict(op=op, B=B, T=max(1, tokens // B), Hk=Hk, H=H, K=K, V=V, dtype=dtype, packed=0,
                h0=rng.random() < 0.5)


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
    if case["op"] == "norm":
        R, C = case["rows"], case["C"]
        wdt = DT[case["wdtype"]]
        x = (rn(R, C) * torch.exp(0.5 * rn(R, 1)) + 0.3 * rn(1, C)).to(dt)
        return dict(case=case, x=x, weight=(1 + 0.1 * rn(C)).to(wdt), bias=(0.1 * rn(C)).to(wdt),
                    dy=rn(R, C).to(dt) if case["grad"] else None)
    B, T, Hk, H, K, V = (case[n] for n in ("B", "T", "Hk", "H", "K", "V"))
    unit = lambda x: x / x.norm(dim=-1, keepdim=True)  # noqa: E731
    common = 0.4 * rn(1, 1, Hk, K)     # keys of one head lean the same way, as learned ones do
    st = dict(case=case, q=unit(rn(B, T, Hk, K)).to(dt), k=unit(rn(B, T, Hk, K) + common).to(dt), v=rn(B, T, H, V).to(dt))
    rate = torch.exp(torch.empty(H, device=dev).uniform_(math.log(0.01), math.log(1.0), generator=gen))
    st["g"] = -rate * torch.nn.functional.softplus(rn(B, T, H))
    st["beta"] = torch.sigmoid(rn(B, T, H))
    if case["op"] == "step":
        P = case["pool"] or B
        st["state"] = 0.1 * rn(P, H, V, K)
        st["next"] = torch.zeros_like(st["state"])
        st["slots"] = None
        if case["pool"]:
            at = list(range(P))
            random.Random(seed).shuffle(at)
            st["slots"] = torch.tensor(at[:B], dtype=torch.int32, device=dev)
        return st
    N = B
    st["cu"] = None
    if case["packed"]:
        N = case["packed"]
        cuts = _lengths(T, N, seed)
        st["cu"] = torch.tensor(cuts, dtype=torch.int32, device=dev)
        st["longest"] = max(b - a for a, b in zip(cuts, cuts[1:]))
    st["h0"] = 0.1 * rn(N, H, V, K) if case["h0"] else None
    if case["op"] == "train":
        st["do"] = rn(B, T, H, V).to(dt)
        st["dhT"] = 0.1 * rn(N, H, V, K) if case["h0"] else None
    return st


# ------------------------------------------------------------------ one pass
def run(st):
    case = st["case"]
    return {"prefill": _run_prefill, "train": _run_train, "step": _run_step, "norm": _run_norm}[case["op"]](st)


def _run_prefill(st):
    if own:
        import linear_rnn_lm_amd as L
        o, _, hT = L.gdr_fwd(st["q"], st["k"], st["v"], st["g"], st["beta"], st["h0"], cu_seqlens=st["cu"],
                             want_ckpt=False)
        return o, hT
    o, hT = _plain(st, *(st[n].float() for n in ("q", "k", "v", "g", "beta")), st["h0"])
    return o.to(st["v"].dtype), hT


def _run_train(st):
    if own:
        import linear_rnn_lm_amd as L
        ins = [st[n] for n in ("q", "k", "v", "g", "beta")]
        o, ckpt, hT = L.gdr_fwd(*ins, st["h0"], cu_seqlens=st["cu"])
        dq, dk, dv, dg, dbeta, dh0 = L.gdr_bwd(st["do"], *ins, ckpt, st["dhT"], cu_seqlens=st["cu"],
                                               want_dh0=st["h0"] is not None)
        return o, hT, dq, dk, dv, dg, dbeta, dh0
    dt = st["v"].dtype
    ins = [st[n].float().detach().requires_grad_() for n in ("q", "k", "v", "g", "beta")]
    h0 = None if st["h0"] is None else st["h0"].detach().requires_grad_()
    with torch.enable_grad():
        o, hT = _plain(st, *ins, h0)
        outs, grads = [o], [st["do"].float()]
        if st["dhT"] is not None:
            outs.append(hT)
            grads.append(st["dhT"])
        got = torch.autograd.grad(outs, ins + ([] if h0 is None else [h0]), grads)
    dq, dk, dv = (x.to(dt) for x in got[:3])
    return o.detach().to(dt), hT.detach(), dq, dk, dv, got[3], got[4], got[5] if h0 is not None else None


def _run_step(st):
    if own:
        import linear_rnn_lm_amd as L
        o = L.gdr_step(st["q"], st["k"], st["v"], st["g"], st["beta"], st["state"], slots=st["slots"],
                       state_out=st["next"])
        return o, st["next"]
    q, k, v, g, beta = (st[n].float() for n in ("q", "k", "v", "g", "beta"))
    rep = v.shape[2] // q.shape[2]
    q, k = q.repeat_interleave(rep, 2), k.repeat_interleave(rep, 2)
    S = st["state"] if st["slots"] is None else st["state"][st["slots"].long()]
    o = torch.empty_like(v)
    scale = q.shape[-1] ** -0.5
    for t in range(q.shape[1]):
        S = S * torch.exp(g[:, t])[..., None, None]
        u = beta[:, t, :, None] * (v[:, t] - torch.matmul(S, k[:, t, :, :, None])[..., 0])
        S = S + u[..., None] * k[:, t, :, None, :]
        o[:, t] = scale * torch.matmul(S, q[:, t, :, :, None])[..., 0]
    if st["slots"] is None:
        st["next"].copy_(S)
    else:
        st["next"][st["slots"].long()] = S
    return o.to(st["v"].dtype), st["next"]


def _run_norm(st):
    case, x = st["case"], st["x"]
    G = case["groups"]
    if own:
        import linear_rnn_lm_amd as L
        y, mean, rstd = L.ln_fwd(x, st["weight"], st["bias"], groups=G, eps=EPS)
        if not case["grad"]:
            return y
        dx, dweight, dbias = L.ln_bwd(st["dy"], x, st["weight"], mean, rstd, groups=G)
        return y, dx, dweight, dbias
    R, C = x.shape
    xs = x.float().view(R, G, C // G)
    w, b = st["weight"].float().view(G, -1), st["bias"].float().view(G, -1)
    xc = xs - xs.mean(-1, keepdim=True)
    rstd = torch.rsqrt((xc * xc).mean(-1, keepdim=True) + EPS)
    xh = xc * rstd
    y = (xh * w + b).view(R, C).to(x.dtype)
    if not case["grad"]:
        return y
    dy = st["dy"].float().view(R, G, -1)
    dxh = dy * w
    dx = rstd * (dxh - dxh.mean(-1, keepdim=True) - xh * (dxh * xh).mean(-1, keepdim=True))
    return y, dx.view(R, C).to(x.dtype), (dy * xh).sum(0).view(C), dy.sum(0).view(C)


# ------------------------------------------------------------------ the gated delta rule in plain torch, chunk by chunk
def _plain(st, q, k, v, g, beta, h0):
    """Packed sequences are laid out as a padded batch first; padding has k = v = g = beta = 0, which changes no state."""
    if st["cu"] is None:
        return _plain_dense(q, k, v, g, beta, h0)
    cu = st["cu"].long()
    T = q.shape[1]
    pos = torch.arange(T, device=q.device)
    seq = torch.searchsorted(cu[1:], pos, right=True)
    at = cu[:-1, None] + torch.arange(st["longest"], device=q.device)
    ok = at < cu[1:, None]
    at = at.clamp(max=T - 1)
    pad = lambda x: x[0][at] * ok.view(*ok.shape, *([1] * (x.dim() - 2)))  # noqa: E731
    o, hT = _plain_dense(pad(q), pad(k), pad(v), pad(g), pad(beta), h0)
    return o[seq, pos - cu[seq]][None], hT


def _plain_dense(q, k, v, g, beta, h0):
    B, T, H, V = v.shape
    K, rep = q.shape[-1], H // q.shape[2]
    C, NC = CHUNK, -(-T // CHUNK)

    def chunks(x):      # (B, T, H, D) -> (B H, NC, C, D)
        x = torch.nn.functional.pad(x, (0, 0, 0, 0, 0, NC * C - T))
        return x.transpose(1, 2).reshape(B * H, NC, C, x.shape[-1])

    q, k, v = chunks(q.repeat_interleave(rep, 2)), chunks(k.repeat_interleave(rep, 2)), chunks(v)
    g, beta = chunks(g[..., None])[..., 0], chunks(beta[..., None])
    G = g.double().cumsum(-1)                                   # sums of log decays, in 64 bits
    lower = torch.ones(C, C, dtype=torch.bool, device=q.device).tril()
    decay = torch.exp(torch.where(lower, G[..., :, None] - G[..., None, :], -math.inf).float())
    kt = k.transpose(-1, -2)
    A = beta * decay * torch.matmul(k, kt) * lower.tril(-1)
    # (I + A)^-1 by blocks of 1, 2, 4, ...: [[X, 0], [Z, Y]]^-1 = [[X', 0], [-Y' Z X', Y']]
    inv = torch.ones(B * H, NC, C, 1, 1, device=q.device)
    for b in (1, 2, 4, 8, 16, 32):
        n = C // (2 * b)
        blocks = A.view(B * H, NC, n, 2 * b, n, 2 * b).diagonal(dim1=2, dim2=4).permute(0, 1, 4, 2, 3)
        X, Y = inv[:, :, 0::2], inv[:, :, 1::2]
        Z = -torch.matmul(torch.matmul(Y, blocks[..., b:, :b]), X)
        inv = torch.cat([torch.cat([X, torch.zeros_like(X)], -1), torch.cat([Z, Y], -1)], -2)
    inv = inv[:, :, 0]
    gamma = torch.exp(G.float())[..., None]
    to_end = torch.exp((G[..., -1:] - G).float())[..., None]
    W = torch.matmul(inv, beta * gamma * k)
    U0 = torch.matmul(inv, beta * v)
    M = decay * torch.matmul(q, kt)
    qg, ke = q * gamma, k * to_end
    S = torch.zeros(B * H, K, V, device=q.device) if h0 is None else h0.reshape(B * H, V, K).transpose(-1, -2)
    outs = []
    for c in range(NC):
        U = U0[:, c] - torch.matmul(W[:, c], S)
        outs.append(torch.matmul(qg[:, c], S) + torch.matmul(M[:, c], U))
        S = gamma[:, c, -1:] * S + torch.matmul(ke[:, c].transpose(-1, -2), U)
    o = torch.stack(outs, 1).view(B, H, NC * C, V)[:, :, :T].transpose(1, 2) * K ** -0.5
    return o, S.transpose(-1, -2).reshape(B, H, V, K)


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "norm":
        n, w = case["rows"] * case["C"], case["C"] * (2 if case["wdtype"] == "bf16" else 4)
        if not case["grad"]:
            return {"bytes": 2 * n * e + 2 * w, "flops": 8 * n}
        return {"bytes": 4 * n * e + 2 * w + 8 * case["C"], "flops": 20 * n}
    B, T, Hk, H, K, V = (case[n] for n in ("B", "T", "Hk", "H", "K", "V"))
    qk, vo, gates, state = 2 * B * T * Hk * K * e, 2 * B * T * H * V * e, 2 * B * T * H * 4, H * V * K * 4
    if case["op"] == "step":
        return {"bytes": qk + vo + gates + 2 * B * state, "flops": 7 * B * T * H * K * V}
    N = case["packed"] or B
    states = N * state * (2 if case["h0"] else 1)
    if case["op"] == "prefill":
        return {"bytes": qk + vo + gates + states, "flops": 7 * B * T * H * K * V}
    return {"bytes": 2 * (qk + vo + gates + states), "flops": 21 * B * T * H * K * V}


# ------------------------------------------------------------------ the definitions, token by token, in 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "norm":
        return _exact_norm(st)
    H = case["H"]
    wide = lambda x: x.double().repeat_interleave(H // x.shape[2], 2)  # noqa: E731
    q, k, v, g, beta = wide(st["q"]), wide(st["k"]), st["v"].double(), st["g"].double(), st["beta"].double()
    if case["op"] == "step":
        at = torch.arange(case["B"], device=q.device) if st["slots"] is None else st["slots"].long()
        o, S, _ = _exact_fwd(q, k, v, g, beta, st["state"].double()[at], False)
        nxt = st["next"].double()
        nxt[at] = S
        return o, nxt
    N = case["packed"] or case["B"]
    h0 = torch.zeros(N, H, case["V"], case["K"], dtype=torch.float64, device=q.device)
    if st["h0"] is not None:
        h0 = st["h0"].double()
    if st["cu"] is None:
        spans = [(slice(None), slice(0, case["T"]), slice(0, case["B"]))]
    else:
        cu = st["cu"].tolist()
        spans = [(slice(0, 1), slice(a, b), slice(n, n + 1)) for n, (a, b) in enumerate(zip(cu, cu[1:]))]
    train = case["op"] == "train"
    if sum(s[1].stop - s[1].start for s in spans) * (3 if train else 1) > 60000:
        return None
    o, hT = torch.zeros_like(v), h0.clone()
    dq, dk, dv, dg, db, dh0 = (torch.zeros_like(x) for x in (q, k, v, g, beta, h0))
    for bs, ts, ns in spans:
        if ts.start == ts.stop:
            if train and st["dhT"] is not None:
                dh0[ns] = st["dhT"].double()[ns]
            continue
        part = [x[bs, ts] for x in (q, k, v, g, beta)]
        o[bs, ts], hT[ns], kept = _exact_fwd(*part, h0[ns], train)
        if train:
            dS = torch.zeros_like(h0[ns]) if st["dhT"] is None else st["dhT"].double()[ns]
            got = _exact_bwd(st["do"].double()[bs, ts], *part, kept, dS)
            for to, x in zip((dq, dk, dv, dg, db), got):
                to[bs, ts] = x
            dh0[ns] = got[5]
    if not train:
        return o, hT
    Hk = case["Hk"]
    dq, dk = (x.view(*x.shape[:2], Hk, H // Hk, -1).sum(3) for x in (dq, dk))
    return o, hT, dq, dk, dv, dg, db, dh0 if st["h0"] is not None else None


def _exact_fwd(q, k, v, g, beta, S, keep):
    o, kept = torch.empty_like(v), []
    scale = q.shape[-1] ** -0.5
    for t in range(q.shape[1]):
        if keep:
            kept.append(S)
        S = S * g[:, t].exp()[..., None, None]
        u = beta[:, t, :, None] * (v[:, t] - (S * k[:, t, :, None, :]).sum(-1))
        S = S + u[..., None] * k[:, t, :, None, :]
        o[:, t] = scale * (S * q[:, t, :, None, :]).sum(-1)
    return o, S, kept


def _exact_bwd(do, q, k, v, g, beta, kept, dS):
    dq, dk, dv, dg, db = (torch.empty_like(x) for x in (q, k, v, g, beta))
    scale = q.shape[-1] ** -0.5
    for t in range(q.shape[1] - 1, -1, -1):
        a, b = g[:, t].exp()[..., None, None], beta[:, t, :, None]
        kr, qr = k[:, t, :, None, :], q[:, t, :, None, :]
        D = a * kept[t]
        p = v[:, t] - (D * kr).sum(-1)
        u = b * p
        dq[:, t] = scale * ((D + u[..., None] * kr) * do[:, t, ..., None]).sum(-2)
        dS = dS + scale * do[:, t, ..., None] * qr
        du = (dS * kr).sum(-1)
        db[:, t] = (du * p).sum(-1)
        dp = b * du
        dv[:, t] = dp
        dD = dS - dp[..., None] * kr
        dk[:, t] = (dS * u[..., None]).sum(-2) - (D * dp[..., None]).sum(-2)
        dg[:, t] = (dD * D).sum((-1, -2))
        dS = a * dD
    return dq, dk, dv, dg, db, dS


def _exact_norm(st):
    case = st["case"]
    G = case["groups"]
    part = lambda x: x.double().reshape(-1, G, x.shape[-1] // G)  # noqa: E731
    x, w, b = part(st["x"]), part(st["weight"]), part(st["bias"])
    var, mean = torch.var_mean(x, -1, correction=0, keepdim=True)
    s = torch.sqrt(var + EPS)
    xh = (x - mean) / s
    y = (xh * w + b).flatten(1)
    if not case["grad"]:
        return y
    dy = part(st["dy"])
    e = dy * w
    dx = (e - e.mean(-1, keepdim=True) - xh * (e * xh).mean(-1, keepdim=True)) / s
    return y, dx.flatten(1), (dy * xh).sum(0).flatten(), dy.sum(0).flatten()

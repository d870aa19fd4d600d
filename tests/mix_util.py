"""The selective scan, the short convolution and the block norm from their definitions in
64 bits, on the CPU, and the tolerances of their tests.

Tolerances (rel-L2 over an output; E = 2^-24).  References get the very values the GPU got, so
what remains is the rounding of the result, at most half a step (2^-8 of the value for bf16, E
for fp32), and the fp32 arithmetic.

Scan.  Per token a state is multiplied by e^(delta A) and added to: delta is good to 8 E (two
exponentials' and a logarithm's last places, and their products), the product delta A and its
exponential to |delta A| 9 E + 2 E of the factor.  |delta A| e^(-|delta A|) is below 0.4, so a
factor's error is at most 6 E of what was there, the update adds 2 roundings and delta's own
8 E: 16 E per token, of states whose earlier parts have decayed meanwhile; over n tokens at
most 16 n E of the sum of the terms' sizes.  That sum is up to sqrt(min(n, 1 / decay)) times the
state's own size for terms of random signs; the tests' steps and decays leave less than 3 of it on
average, and not all roundings lean the same way: 16 n E covers both.  y adds a sum
over S states: S E.  Gradients run over the same factors once more and through delta's slope:
twice that; the weights' sums over all tokens add one rounding per token.

Convolution: W products and sums, the activation (sigmoid: 4 E; its slope multiplies it by at
most 2): (2 W + 10) E, twice that for gradients, and a rounding per token for the sums over
tokens.

Block norm: sums over C channels, at most C E of their terms' sizes, through mean, variance (2
C) and both norms (4 C), in the backward once more (8 C).  dx-like results of a norm take differences
of their terms, see `grow` where it is used.
"""
import torch

E = 2.0 ** -24


def half_step(dt):
    return 2.0 ** -8 if dt == torch.bfloat16 else E


def rel(x, ref):
    x, ref = x.detach().double().cpu(), ref.detach().double().cpu()
    assert x.shape == ref.shape, (x.shape, ref.shape)
    assert torch.equal(torch.isnan(x), torch.isnan(ref)), "NaN in other places"
    x, ref = torch.nan_to_num(x), torch.nan_to_num(ref)
    n = ref.norm().item()
    return (x - ref).norm().item() / n if n > 0 else x.norm().item()


# ------------------------------------------------------------------ selective scan
def scan_tol(steps, S, dtype, tokens=0, grad=False):
    return half_step(dtype) + (2 if grad else 1) * (16 * steps + S + 16) * E + tokens * E


def make_scan(B, T, C, S, G, dtype, seed=0, N=None, z=True, D=True, bias=True, h0=True):
    """Seeded inputs on the CPU: a dict of x, dt, A, b, c, D, z, dt_bias, h0, dy, dhT."""
    gen = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    N = N or B
    p = dict(x=rn(B, T, C).to(dtype), dt=(rn(B, T, C) - 2).to(dtype), A=-torch.exp(0.7 * rn(C, S)),
             b=rn(B, T, G, S).to(dtype), c=rn(B, T, G, S).to(dtype))
    p["D"] = 1 + 0.3 * rn(C) if D else None
    p["z"] = rn(B, T, C).to(dtype) if z else None
    p["dt_bias"] = 0.5 * rn(C) if bias else None
    p["h0"] = rn(N, C, S) if h0 else None
    p["dy"] = rn(B, T, C).to(dtype)
    p["dhT"] = rn(N, C, S) if h0 else None
    return p


INS = ("x", "dt", "A", "b", "c", "D", "z", "dt_bias", "h0")
GRADS = ("dx", "ddt", "dA", "db", "dc", "dD", "dz", "ddt_bias", "dh0")


def ref_scan(v, softplus=True, cu=None, N=None):
    """Token by token, differentiable; v: a dict of doubles -> y (rows outside sequences 0), hT."""
    x, A = v["x"], v["A"]
    B, T, C = x.shape
    S, per = A.shape[1], C // v["b"].shape[2]
    d = v["dt"] + (0 if v["dt_bias"] is None else v["dt_bias"])
    if softplus:
        d = torch.logaddexp(d, torch.zeros_like(d))
    b, c = (v[n].repeat_interleave(per, 2) for n in ("b", "c"))
    spans = [(slice(None), 0, T, slice(None))] if cu is None else \
        [(slice(0, 1), a, e, slice(n, n + 1)) for n, (a, e) in enumerate(zip(cu, cu[1:]))]
    N = B if cu is None else len(cu) - 1
    h0 = x.new_zeros(N, C, S) if v["h0"] is None else v["h0"]
    zero = x.new_zeros(x.shape[0], C)
    ys, hs = [zero] * T, []
    for rows, t0, t1, ns in spans:
        h = h0[ns]
        for t in range(t0, t1):
            h = torch.exp(d[rows, t, :, None] * A) * h + (d[rows, t] * x[rows, t])[..., None] * b[rows, t]
            ys[t] = (h * c[rows, t]).sum(-1)
            if v["D"] is not None:
                ys[t] = ys[t] + v["D"] * x[rows, t]
            if v["z"] is not None:
                ys[t] = ys[t] * v["z"][rows, t] * torch.sigmoid(v["z"][rows, t])
        hs.append(h)
    return torch.stack(ys, 1), torch.cat(hs)


def ref_scan_grads(p, softplus=True, cu=None, dev="cpu"):
    """(y, hT) and a dict of gradients (formed on `dev`, where elementary operations are quicker for many channels)."""
    p = {n: None if t is None else t.to(dev) for n, t in p.items()}
    v = {n: None if p[n] is None else p[n].double().requires_grad_() for n in INS}
    y, hT = ref_scan(v, softplus, cu)
    outs, cots = [y], [p["dy"].double()]
    if p["dhT"] is not None:
        outs.append(hT)
        cots.append(p["dhT"].double())
    outs, cots = zip(*[(o, g) for o, g in zip(outs, cots) if o.requires_grad])     # y of empty sequences has none
    it = iter(torch.autograd.grad(outs, [v[n] for n in INS if v[n] is not None], cots, allow_unused=True))
    grads = {g: None if v[n] is None else next(it) for n, g in zip(INS, GRADS)}
    for n, g in zip(INS, GRADS):
        if v[n] is not None and grads[g] is None:
            grads[g] = torch.zeros_like(v[n])
    return y.detach(), hT.detach(), grads


# ------------------------------------------------------------------ convolution
def conv_tol(W, dtype, tokens=0, grad=False):
    return half_step(dtype) + (2 if grad else 1) * (2 * W + 10) * E + tokens * E


def make_conv(B, T, C, W, dtype, seed=0, N=None, bias=True, h0=True, wdtype=torch.float32):
    gen = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    N = N or B
    return dict(x=rn(B, T, C).to(dtype), weight=rn(C, W).to(wdtype), bias=(0.5 * rn(C)).to(wdtype) if bias else None,
                h0=rn(N, W - 1, C).to(dtype) if h0 else None, dy=rn(B, T, C).to(dtype),
                dhT=rn(N, W - 1, C).to(dtype) if h0 else None)


def ref_conv(v, silu=True, cu=None):
    """Differentiable; rows outside sequences 0 -> y, hT."""
    x, w = v["x"], v["weight"]
    (B, T, C), W = x.shape, w.shape[1]
    spans = [(slice(None), 0, T, slice(None))] if cu is None else \
        [(slice(0, 1), a, e, slice(n, n + 1)) for n, (a, e) in enumerate(zip(cu, cu[1:]))]
    N = B if cu is None else len(cu) - 1
    h0 = x.new_zeros(N, W - 1, C) if v["h0"] is None else v["h0"]
    ys, hs, at = [], [], 0
    for rows, t0, t1, ns in spans:
        ext = torch.cat([h0[ns], x[rows, t0:t1]], 1)
        s = sum(ext[:, j:j + t1 - t0] * w[:, j] for j in range(W))
        if v["bias"] is not None:
            s = s + v["bias"]
        ys += [x.new_zeros(ext.shape[0], t0 - at, C), s * torch.sigmoid(s) if silu else s]
        hs.append(ext[:, t1 - t0:])
        at = t1
    ys.append(x.new_zeros(x.shape[0] if cu is None else 1, T - at, C))
    return torch.cat(ys, 1), torch.cat(hs)


def ref_conv_grads(p, silu=True, cu=None):
    names = ("x", "weight", "bias", "h0")
    v = {n: None if p[n] is None else p[n].double().requires_grad_() for n in names}
    y, hT = ref_conv(v, silu, cu)
    outs, cots = [y], [p["dy"].double()]
    if p["dhT"] is not None:
        outs.append(hT)
        cots.append(p["dhT"].double())
    leaves = [v[n] for n in names if v[n] is not None]
    it = iter(torch.autograd.grad(outs, leaves, cots, allow_unused=True))
    got = {}
    for n, g in zip(names, ("dx", "dweight", "dbias", "dh0")):
        if v[n] is not None:
            d = next(it)
            got[g] = torch.zeros_like(v[n]) if d is None else d
    return y.detach(), hT.detach(), got


# ------------------------------------------------------------------ block norm
WS = ("weight", "bias", "scale", "weight2", "bias2")


def ref_rn(v, groups=1, norm="layer", norm2=None, act="silu", eps=1e-5, eps2=1e-5):
    """Differentiable; v: a dict of doubles -> r, h."""
    def normed(t, kind, e):
        if kind == "layer":
            t = t - t.mean(-1, keepdim=True)
        return t / torch.sqrt((t * t).mean(-1, keepdim=True) + e)

    u = normed(v["o"].unflatten(-1, (groups, -1)), norm, eps).flatten(-2)
    u = u if v["weight"] is None else u * v["weight"]
    u = u if v["bias"] is None else u + v["bias"]
    if v["gate"] is not None:
        s = torch.sigmoid(v["gate"])
        u = u * (v["gate"] * s if act == "silu" else s)
    u = u if v["scale"] is None else u * v["scale"]
    r = u if v["res"] is None else v["res"] + u
    if norm2 is None:
        return r, None
    h = normed(r, norm2, eps2)
    h = h if v["weight2"] is None else h * v["weight2"]
    return r, h if v["bias2"] is None else h + v["bias2"]

"""The gated delta rule and the layer norm from their definitions in 64 bits, on
the CPU, and the tolerances of their tests.

Tolerances.  A reference is computed from the very values the GPU got, so what
remains is the rounding of the result, at most half a step (2^-8 of the value for
bf16, 2^-24 for fp32), and the fp32 arithmetic in between.  Per chunk a value of o or of the state
passes through sums over K, over 64 tokens (R to U), and over 64 tokens again: an
fp32 sum of n terms is off by at most n 2^-24 of the sum of its terms' sizes, so
(K + 128) 2^-24 relative for well-scaled terms; states decay from chunk to chunk, and the
delta rule removes errors along k as it removes values, so chunks do not
add up.  The gradients pass the same sums twice, once more for the row sums
(another V): 2 (K + 128) + V, all of it times 2^-24 (rel-L2 over an output).
"""
import torch


def tol_fwd(K, dtype):
    return (2.0 ** -8 if dtype == torch.bfloat16 else 0.0) + (K + 128) * 2.0 ** -24


def tol_bwd(K, V, dtype):
    return (2.0 ** -8 if dtype == torch.bfloat16 else 0.0) + (2 * (K + 128) + V) * 2.0 ** -24


def rel(x, ref):
    x, ref = x.detach().double().cpu(), ref.detach().double().cpu()
    assert x.shape == ref.shape
    assert torch.equal(torch.isnan(x), torch.isnan(ref)), "NaN in other places"
    x, ref = torch.nan_to_num(x), torch.nan_to_num(ref)
    n = ref.norm().item()
    return (x - ref).norm().item() / n if n > 0 else x.norm().item()


def make(B, T, Hk, H, K, V, dtype, seed=0, N=None, h0=True, lean=0.4):
    """Seeded inputs (q, k, v, g, beta, h0, do, dhT) on the CPU."""
    gen = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    unit = lambda x: x / x.norm(dim=-1, keepdim=True)  # noqa: E731
    q = unit(rn(B, T, Hk, K)).to(dtype)
    k = unit(rn(B, T, Hk, K) + lean * rn(1, 1, Hk, K)).to(dtype)
    v = rn(B, T, H, V).to(dtype)
    g = -torch.exp(1.5 * rn(H) - 2) * torch.nn.functional.softplus(rn(B, T, H))
    beta = torch.sigmoid(rn(B, T, H))
    N = N or B
    s0 = 0.1 * rn(N, H, V, K) if h0 else None
    do = rn(B, T, H, V).to(dtype)
    dhT = 0.1 * rn(N, H, V, K) if h0 else None
    return q, k, v, g, beta, s0, do, dhT


def ref_dense(q, k, v, g, beta, h0, scale):
    """Token by token in 64 bits, differentiable.  (B, T, ...) -> o, final state."""
    H = v.shape[2]
    q, k = (x.repeat_interleave(H // x.shape[2], 2) for x in (q, k))
    S, os = h0, []
    for t in range(q.shape[1]):
        S = S * torch.exp(g[:, t])[..., None, None]
        u = beta[:, t, :, None] * (v[:, t] - (S * k[:, t, :, None, :]).sum(-1))
        S = S + u[..., None] * k[:, t, :, None, :]
        os.append(scale * (S * q[:, t, :, None, :]).sum(-1))
    return torch.stack(os, 1), S


def reference(q, k, v, g, beta, h0=None, do=None, dhT=None, cu=None, scale=None):
    """{o, hT} and, given do, {dq, dk, dv, dg, dbeta, dh0} in 64 bits; tokens
    outside the packed sequences have zeros."""
    B, T, Hk, K = q.shape
    H, V = v.shape[2:]
    scale = K ** -0.5 if scale is None else scale
    N = B if cu is None else len(cu) - 1
    leaves = [x.double().clone().requires_grad_() for x in (q, k, v, g, beta)]
    s0 = torch.zeros(N, H, V, K, dtype=torch.float64) if h0 is None else h0.double().clone()
    s0.requires_grad_()
    if cu is None:
        o, hT = ref_dense(*leaves, s0, scale)
    else:
        parts, last, at = [], [], 0
        for n in range(N):
            a, b = cu[n], cu[n + 1]
            parts.append(torch.zeros(1, a - at, H, V, dtype=torch.float64))
            at = b
            if a == b:
                last.append(s0[n:n + 1])
                continue
            on, sn = ref_dense(*[x[:, a:b] for x in leaves], s0[n:n + 1], scale)
            parts.append(on)
            last.append(sn)
        parts.append(torch.zeros(1, T - at, H, V, dtype=torch.float64))
        o, hT = torch.cat(parts, 1), torch.cat(last)
    out = {"o": o.detach(), "hT": hT.detach()}
    if do is not None:
        loss = (o * do.double()).sum()
        if dhT is not None:
            loss = loss + (hT * dhT.double()).sum()
        grads = torch.autograd.grad(loss, [*leaves, s0], allow_unused=True)
        for n, x, like in zip(("dq", "dk", "dv", "dg", "dbeta", "dh0"), grads, [*leaves, s0]):
            out[n] = torch.zeros_like(like) if x is None else x
    return out


def ref_norm(x, weight, bias, groups, eps, dy=None):
    """{y} and, given dy, {dx, dweight, dbias} in 64 bits; x (rows, C)."""
    x = x.double().clone().requires_grad_()
    C = x.shape[1]
    w = torch.ones(C, dtype=torch.float64) if weight is None else weight.double().clone()
    b = torch.zeros(C, dtype=torch.float64) if bias is None else bias.double().clone()
    w.requires_grad_()
    b.requires_grad_()
    p = x.view(x.shape[0], groups, -1)
    c = p - p.mean(-1, keepdim=True)
    xh = c / torch.sqrt((c * c).mean(-1, keepdim=True) + eps)
    y = xh.reshape(x.shape) * w + b
    out = {"y": y.detach()}
    if dy is not None:
        out["dx"], out["dweight"], out["dbias"] = torch.autograd.grad(y, [x, w, b], dy.double())
    return out

"""The multi-head operators in 64 bits, step by step from their definitions
(torch on the CPU), their gradients by the chain rule written out, seeded
inputs, and the comparison the tests use.

Bounds of the comparison, by the type a result is stored in.  A float32
result is made of products whose factors are exact or carry float32 rounding
(2^-24 each) and of float32 sums of at most some hundred terms a stage, so its
error relative to the result's 2-norm stays near 1e-6; 2e-5 leaves room for
the steps' exponentials.  A bfloat16 result is rounded once (2^-9, about
1.7e-3 in the 2-norm), and the matrix products behind it may round one operand
of each of two products the same way: sqrt(3) 1.7e-3 = 2.9e-3; the bound is
5e-3.  Single elements: 10 times the bound of the 2-norm, relative to the
larger of the element and the root mean square.
A sum over all tokens (dA, dD, ddelta_bias) may cancel, so its error is held
relative to the root of its terms' squares where that is larger.
"""
import numpy as np
import torch

F64 = torch.float64
REL = {torch.float32: 2e-5, torch.bfloat16: 5e-3}


def check(name, got, ref, scale=None):
    """`scale`: what the error is relative to where it exceeds |ref| (a sum's
    terms in the 2-norm, element by element)."""
    rel = REL[got.dtype]
    g, r = got.detach().double().cpu(), ref.double()
    assert g.shape == r.shape, (name, g.shape, r.shape)
    assert torch.isfinite(g).all(), f"{name}: not finite"
    e = (g - r).abs()
    s = r.abs() if scale is None else torch.maximum(r.abs(), scale.double())
    norm = float(s.norm())
    assert float(e.norm()) <= rel * norm + 1e-30, (name, float(e.norm()) / max(norm, 1e-300), rel)
    rms = norm / max(1, s.numel()) ** 0.5
    bad = e > 10 * rel * torch.clamp(s, min=rms) + 1e-30
    assert not bad.any(), (name, float((e / torch.clamp(s, min=rms)).max()), 10 * rel)


def steps(raw, A, softplus, disc):
    dt = torch.logaddexp(raw, torch.zeros_like(raw)) if softplus else raw
    x = dt * A
    safe = torch.where(A == 0, torch.ones_like(A), A)
    w = torch.where(A == 0, dt, torch.expm1(x) / safe) if disc == "zoh" else dt
    return dt, torch.exp(x), w


def rep(t, H):
    """(..., groups, N) -> (..., heads, N)."""
    return t.repeat_interleave(H // t.shape[-2], -2)


def scan_fwd(u, delta, A, B, C, D=None, delta_bias=None, h0=None, reset=None, softplus=True,
             disc="zoh"):
    """out, last state, and the states before every step."""
    b, L, H, P = u.shape
    raw = delta if delta_bias is None else delta + delta_bias
    dt, a, w = steps(raw, A, softplus, disc)
    if reset is not None:
        a = torch.where(reset.bool().unsqueeze(-1), torch.zeros_like(a), a)
    h = torch.zeros(b, H, P, B.shape[-1], dtype=F64) if h0 is None else h0
    Bh, Ch = rep(B, H), rep(C, H)
    out, hs = torch.zeros_like(u), []
    for t in range(L):
        hs.append(h)
        h = a[:, t, :, None, None] * h + torch.einsum("bh,bhp,bhn->bhpn", w[:, t], u[:, t], Bh[:, t])
        out[:, t] = torch.einsum("bhpn,bhn->bhp", h, Ch[:, t])
    if D is not None:
        out = out + D[:, None] * u
    return out, h, hs


def scan_bwd(u, delta, A, B, C, D, delta_bias, dout, h0=None, dlast=None, reset=None,
             softplus=True, disc="zoh"):
    """Gradients, and the scales of the sums over all tokens."""
    b, L, H, P = u.shape
    G, N = B.shape[-2:]
    raw = delta if delta_bias is None else delta + delta_bias
    dt, a, w = steps(raw, A, softplus, disc)
    if reset is not None:
        a = torch.where(reset.bool().unsqueeze(-1), torch.zeros_like(a), a)
    _, last, hs = scan_fwd(u, delta, A, B, C, None, delta_bias, h0, reset, softplus, disc)
    hs = hs[1:] + [last]
    Bh, Ch = rep(B, H), rep(C, H)
    g = torch.zeros_like(last) if dlast is None else dlast
    du, dBh, dCh = torch.zeros_like(u), torch.zeros_like(Bh), torch.zeros_like(Ch)
    dlog, dw = torch.zeros_like(dt), torch.zeros_like(dt)
    before = [torch.zeros_like(last) if h0 is None else h0] + hs[:-1]
    for t in reversed(range(L)):
        g = g + torch.einsum("bhp,bhn->bhpn", dout[:, t], Ch[:, t])
        dCh[:, t] = torch.einsum("bhpn,bhp->bhn", hs[t], dout[:, t])
        gB = torch.einsum("bhpn,bhn->bhp", g, Bh[:, t])
        du[:, t] = w[:, t, :, None] * gB
        dBh[:, t] = torch.einsum("bhpn,bhp->bhn", g, u[:, t]) * w[:, t, :, None]
        dw[:, t] = (gB * u[:, t]).sum(-1)
        g = a[:, t, :, None, None] * g
        dlog[:, t] = (g * before[t]).sum((-1, -2))
    if disc == "zoh":
        x = dt * A
        by_dt = torch.exp(x)
        series = dt * dt * (0.5 + x / 3 + x * x / 8)
        safe = torch.where(A == 0, torch.ones_like(A), A)
        by_A = torch.where(x.abs() < 1e-5, series, (dt * by_dt - torch.expm1(x) / safe) / safe)
    else:
        by_dt, by_A = torch.ones_like(dt), torch.zeros_like(dt)
    ddelta = (A * dlog + dw * by_dt) * (torch.sigmoid(raw) if softplus else 1.0)
    tA, tD = dt * dlog + dw * by_A, (u * dout).sum(-1)
    res = dict(du=du if D is None else du + D[:, None] * dout, ddelta=ddelta, dA=tA.sum((0, 1)),
               dB=dBh.unflatten(-2, (G, H // G)).sum(-2), dC=dCh.unflatten(-2, (G, H // G)).sum(-2))
    terms = lambda t: t.square().sum((0, 1)).sqrt()  # noqa: E731
    scale = dict(dA=terms(tA), dD=terms(tD), ddelta_bias=terms(ddelta))
    if D is not None:
        res["dD"] = tD.sum((0, 1))
    if delta_bias is not None:
        res["ddelta_bias"] = ddelta.sum((0, 1))
    if h0 is not None:
        res["dh0"] = g
    return res, scale


def conv_fwd(x, w, b=None, window=None, reset=None):
    """out and the window to continue from."""
    n, L, dim = x.shape
    W = w.shape[1]
    hist = torch.zeros(n, W - 1, dim, dtype=F64) if window is None else window.clone()
    out = torch.zeros_like(x)
    for t in range(L):
        if reset is not None:
            hist = torch.where(reset[:, t].bool()[:, None, None], torch.zeros_like(hist), hist)
        taps = torch.cat([hist, x[:, t:t + 1]], 1)
        pre = (taps * w.T).sum(1) + (0 if b is None else b)
        out[:, t] = pre * torch.sigmoid(pre)
        hist = taps[:, 1:]
    return out, hist


def norm_fwd(x, z, weight, groups, eps, gate_first):
    g = 1.0 if z is None else z * torch.sigmoid(z)
    v = x * g if gate_first else x
    v = v.unflatten(-1, (groups, -1))
    y = (v / torch.sqrt(v.square().mean(-1, keepdim=True) + eps)).flatten(-2)
    y = y if weight is None else y * weight
    return y if gate_first else y * g


def autograd(fn, leaves, dout):
    """Gradients of sum(fn(leaves) dout) for the given leaves, in 64 bits."""
    vs = [None if v is None else v.detach().clone().requires_grad_(True) for v in leaves]
    live = [v for v in vs if v is not None]
    got = iter(torch.autograd.grad(fn(*vs), live, dout))
    return [None if v is None else next(got) for v in vs]


class Inputs:
    """Seeded tensors, rounded to `dtype` first so that both sides see the same values."""

    def __init__(self, seed, dtype):
        self.r, self.dtype = np.random.default_rng([20, seed]), dtype

    def seq(self, *shape, scale=1.0):
        x = torch.from_numpy(self.r.standard_normal(shape) * scale)
        return x.to(self.dtype).double()

    def f32(self, *shape, scale=1.0):
        return torch.from_numpy(self.r.standard_normal(shape) * scale).float().double()

    def uniform(self, lo, hi, *shape):
        return torch.from_numpy(self.r.uniform(lo, hi, shape)).float().double()

    def flags(self, batch, L, kind):
        f = np.zeros((batch, L), np.uint8)
        if kind == "random":
            f = (self.r.random((batch, L)) < 0.04).astype(np.uint8)
        elif kind == "every":
            f[:] = 1
        elif kind == "edges":       # first, last and the steps around multiples of 32
            f[:, 0] = f[:, -1] = 1
            f[:, 31::32] = 1
            f[:, 64::64] = 1
        return torch.from_numpy(f)


def scan_inputs(seed, dtype, batch, L, H, P, G, N, h0=False, reset=None, A="init"):
    r = Inputs(seed, dtype)
    a = -r.uniform(1.0, 16.0, H)
    if A == "mixed":           # a growing head, one without decay, a nearly still one
        a[0::3], a[1::3] = 0.01, 0.0
        a[2::3] = -1e-4
    return dict(u=r.seq(batch, L, H, P), delta=r.seq(batch, L, H), A=a, B=r.seq(batch, L, G, N),
                C=r.seq(batch, L, G, N), D=r.f32(H), delta_bias=r.uniform(-6.9, -2.25, H),
                h0=r.f32(batch, H, P, N) if h0 else None,
                reset=None if reset is None else r.flags(batch, L, reset),
                dout=r.seq(batch, L, H, P), dlast=r.f32(batch, H, P, N))

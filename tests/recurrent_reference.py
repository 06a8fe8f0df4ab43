"""The gated linear recurrence and the residual norm in 64 bits, step by step from
their definitions (torch on the CPU), their gradients by the chain rule written
out, seeded inputs, and the comparison the tests use.

Bounds of the comparison, by the type a result is stored in.  float32: a step's
decay is off by at most 2^-22 relative (its exponent's rounding and one unit of
the exponential), and the inputs here, A <= -1/20 and gates of unit variance,
forget within some 40 steps, so that the states are off by 40 2^-22 = 1e-5 if
all the errors point one way; what follows is a handful of products of 2^-24
each, and sums of at most some thousand terms in parts of at most a hundred.
2e-5 relative to the 2-norm, and for single elements ten times that relative to
the larger of the element and the root mean square (a gradient is the difference
of two terms).  bfloat16 and e4m3: that, and half a step of the type (2^-8,
2^-4) of each element for its one rounding; below the type's smallest normal
value half of its smallest step.  A sum over tokens (dA, dweight) is held
relative to the sum of its terms' absolute values: each is within the bound.
"""
import torch

F64 = torch.float64
REL = 2e-5
HALF = {torch.float32: 0.0, torch.bfloat16: 2.0 ** -8, torch.float8_e4m3fn: 2.0 ** -4}
LEAST = {torch.float32: 0.0, torch.bfloat16: 2.0 ** -134, torch.float8_e4m3fn: 2.0 ** -10}


def check(name, got, ref, scale=None, rel=REL):
    """`scale`: what the error is relative to where it exceeds |ref|, element by element."""
    half, least = HALF[got.dtype], LEAST[got.dtype]
    g, r = got.detach().double().cpu(), ref.double().cpu()
    assert g.shape == r.shape, (name, g.shape, r.shape)
    assert torch.isfinite(g).all(), f"{name}: not finite"
    e = (g - r).abs()
    s = r.abs() if scale is None else torch.maximum(r.abs(), scale.double())
    norm = float(s.norm())
    # half a step is relative to the rounded value, itself within 1 + half of the true one
    allowed = (half * (1 + half) + rel) * norm + least * s.numel() ** 0.5 + 1e-37
    assert float(e.norm()) <= allowed, (name, float(e.norm()) / max(norm, 1e-300))
    rms = norm / max(1, s.numel()) ** 0.5
    bad = e > half * (1 + half) * r.abs() + 10 * rel * torch.clamp(s, min=rms) + least + 1e-37
    assert not bad.any(), (name, int(bad.sum()), float((e / torch.clamp(s, min=rms)).max()))


def sig(v):
    return 1 / (1 + torch.exp(-v))


def stored(t, dtype):
    """Values that `dtype` holds, in 64 bits."""
    return t.float().to(dtype).double()


def rec_inputs(seed, dtype, batch, L, dim, z=True, h0=True, reset=None):
    r = torch.Generator().manual_seed(seed)
    n = lambda *s: stored(torch.randn(*s, generator=r), dtype)  # noqa: E731
    f = lambda *s: torch.randn(*s, generator=r).double()  # noqa: E731
    i = dict(x=n(batch, L, dim), r=n(batch, L, dim), i=n(batch, L, dim),
             A=-(0.05 + 4 * torch.rand(dim, generator=r)).double(),
             z=n(batch, L, dim) if z else None, h0=f(batch, dim) if h0 else None,
             dout=n(batch, L, dim), dlast=f(batch, dim), reset=None)
    if reset == "random":
        i["reset"] = (torch.rand(batch, L, generator=r) < 0.05).to(torch.uint8)
    elif reset == "every":
        i["reset"] = torch.ones(batch, L, dtype=torch.uint8)
    elif reset == "edges":
        i["reset"] = torch.zeros(batch, L, dtype=torch.uint8)
        for t in (0, 15, 16, 63, 64, 127, 128, 1024, L - 1):
            if t < L:
                i["reset"][t % batch, t] = 1
    return i


def rec_fwd(x, r, i, A, z=None, h0=None, reset=None):
    """out, last state, and the states before every step."""
    b, L, d = x.shape
    a = torch.exp(A * sig(r))
    v = torch.sqrt(-torch.expm1(2 * A * sig(r))) * sig(i) * x
    h = torch.zeros(b, d, dtype=x.dtype) if h0 is None else h0
    before, states = [], []
    for t in range(L):
        before.append(h)
        into = a[:, t] * h
        if reset is not None:
            into = torch.where(reset[:, t, None] != 0, torch.zeros((), dtype=x.dtype), into)
        h = into + v[:, t]
        states.append(h)
    states = torch.stack(states, 1)
    return (states if z is None else states * z * sig(z)), h, torch.stack(before, 1)


def rec_bwd(x, r, i, A, z, dout, h0=None, dlast=None, reset=None):
    """The gradients, and for dA the sum of its terms' absolute values."""
    b, L, d = x.shape
    _, _, before = rec_fwd(x, r, i, A, z, h0, reset)
    sr, si = sig(r), sig(i)
    a = torch.exp(A * sr)
    m = torch.sqrt(-torch.expm1(2 * A * sr))
    kept = a if reset is None else torch.where(reset.unsqueeze(-1) != 0,
                                               torch.zeros((), dtype=x.dtype), a)
    hk = torch.where(kept == 0, torch.zeros((), dtype=x.dtype), kept * before)
    got = {}
    dh = dout
    if z is not None:
        sz = sig(z)
        got["dz"] = dout * (hk + m * si * x) * sz * (1 + z * (1 - sz))
        dh = dout * z * sz
    g = torch.zeros_like(x)
    after = torch.zeros(b, d, dtype=x.dtype) if dlast is None else dlast
    for t in reversed(range(L)):
        g[:, t] = dh[:, t] + after
        after = kept[:, t] * g[:, t]
    if h0 is not None:
        got["dh0"] = after
    got["dx"] = g * m * si
    got["di"] = g * m * x * si * (1 - si)
    dlog = g * (hk - si * x * a * a / m)
    got["dr"] = dlog * A * sr * (1 - sr)
    got["dA"] = (dlog * sr).sum((0, 1))
    return got, {"dA": (g.abs() * (hk.abs() + (si * x * a * a / m).abs()) * sr).sum((0, 1))}


def norm_inputs(seed, dtype, res_dtype, *shape, residual=True, weight=True):
    r = torch.Generator().manual_seed(seed)
    n = lambda dt, *s: stored(torch.randn(*s, generator=r), dt)  # noqa: E731
    return dict(x=n(dtype, *shape), residual=2 * n(res_dtype, *shape) if residual else None,
                weight=1 + 0.3 * torch.randn(shape[-1], generator=r).float().double()
                if weight else None, dout=n(dtype, *shape), dres=n(res_dtype, *shape))


def norm_fwd(x, residual, weight, eps, res_dtype):
    """out, res as it is kept, and the exact sum."""
    total = x if residual is None else x + residual
    res = total if residual is None else total.float().to(res_dtype).double()
    y = res / torch.sqrt(res.square().mean(-1, keepdim=True) + eps)
    return (y if weight is None else y * weight), res, total


def norm_terms(res, weight, dout, dres, eps):
    """The sum of the absolute values of the terms that norm_bwd's d is made of.  d may
    be a small difference of them (with one column it is inner eps / root^3, of
    two terms of |inner| / root that agree in all but eps / root^2), each rounded
    to 2^-24 of itself: d's error is relative to them, not to d."""
    root = torch.sqrt(res.square().mean(-1, keepdim=True) + eps)
    inner = dout if weight is None else dout * weight
    mean = (inner * res / root).abs().mean(-1, keepdim=True)
    terms = (inner.abs() + (res / root).abs() * mean) / root
    return terms if dres is None else terms + dres.abs()


def norm_bwd(res, weight, dout, dres, eps):
    n = res.shape[-1]
    root = torch.sqrt(res.square().mean(-1, keepdim=True) + eps)
    hat = res / root
    inner = dout if weight is None else dout * weight
    d = (inner - hat * (inner * hat).sum(-1, keepdim=True) / n) / root
    if dres is not None:
        d = d + dres
    flat = (dout * hat).reshape(-1, n)
    return d, flat.sum(0), flat.abs().sum(0)

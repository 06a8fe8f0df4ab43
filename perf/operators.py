"""What is measured of the multi-head operators: the token-major mixer that
reads a joined projection, convolves it, scans it with one decay a head and
normalises it under a gate; for prompts, for training and token by token.

Every case is one call of a public operator (the token cases: the convolution's
and the scan's single-token forms, which always run together).  `run` computes
it in elementary torch operations in 32 bits, or, where `own` is true, calls
scan_selective_fwd_amd.  Layouts: u (batch, L, heads, P), delta (batch, L,
heads), B, C (batch, L, groups, N), states (batch, heads, P, N) float32; x of
the convolution (batch, L, dim), its window (batch, W - 1, dim); rows of the
norm (rows, dim).
"""
import math

import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
BIAS_LO, BIAS_HI = math.log(math.expm1(0.001)), math.log(math.expm1(0.1))
PLAIN_CHUNK = 128


def _ms():
    import scan_selective_fwd_amd as ms
    return ms


# --------------------------------------------------------------------------- cases

def _scan(name, kind, batch, L, heads, P, N, groups, dtype, disc, h0, packed):
    c = dict(kind=kind, batch=batch, L=L, heads=heads, P=P, N=N, groups=groups, dtype=dtype,
             disc=disc, h0=h0, packed=packed)
    return dict(c, name=name) if name else c


def _token(name, batch, heads, P, N, groups, dtype, disc, slots):
    c = dict(kind="token", batch=batch, heads=heads, P=P, N=N, groups=groups, dtype=dtype,
             disc=disc, slots=slots)
    return dict(c, name=name) if name else c


def _conv(name, kind, batch, L, dim, W, dtype, window, packed):
    c = dict(kind=kind, batch=batch, L=L, dim=dim, W=W, dtype=dtype, window=window,
             packed=packed)
    return dict(c, name=name) if name else c


def _norm(name, kind, rows, dim, groups, dtype, gate_first):
    c = dict(kind=kind, rows=rows, dim=dim, groups=groups, dtype=dtype, gate_first=gate_first)
    return dict(c, name=name) if name else c


def listed():
    return [
        # the next piece of one user's prompt, continuing from its state: latency counts
        _scan("prompt-piece", "scan_fwd", 1, 200, 24, 64, 128, 1, "bf16", "euler", True, False),
        # a batch of prompts at the benchmark layer's width (8 x 2048 x 1536)
        _scan("prompt-batch", "scan_fwd", 8, 2048, 24, 64, 128, 1, "bf16", "euler", False, False),
        # one very long document: few channels, all the work along the sequence
        _scan("prompt-long", "scan_fwd", 1, 131072, 24, 64, 128, 1, "bf16", "zoh", False, False),
        # packed ragged prompts in float32, sizes that fill no tile, two groups
        _scan("prompt-packed-f32", "scan_fwd", 3, 1000, 10, 48, 80, 2, "f32", "zoh", True, True),
        # the backward of a wide training layer (2 x 2048 x 5120)
        _scan("train-wide", "scan_bwd", 2, 2048, 80, 64, 128, 1, "bf16", "euler", False, False),
        # packed training rows in float32, four groups, with the entering state's gradient
        _scan("train-packed-f32", "scan_bwd", 4, 777, 16, 64, 64, 4, "f32", "zoh", True, True),
        # one token of one user: the smallest call
        _token("token-one", 1, 24, 64, 128, 1, "bf16", "euler", False),
        # one token for each of 256 users, states picked from a pool by slot
        _token("token-pool", 256, 80, 64, 128, 1, "bf16", "euler", True),
        # the convolution of a batch of prompts, handing its window on to decoding
        _conv("conv-prompt", "conv_fwd", 8, 2048, 1792, 4, "bf16", True, False),
        # its backward in packed training rows
        _conv("conv-train", "conv_bwd", 2, 2047, 5376, 4, "bf16", False, True),
        # the gated norm of a batch of prompts
        _norm("norm-prompt", "norm_fwd", 16384, 1536, 1, "bf16", True),
        # its backward in training, eight groups a row
        _norm("norm-train", "norm_bwd", 4096, 5120, 8, "bf16", True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(dim, step):  # one width is left out
    return dim + step if dim == 3 * 1024 else dim


def _sizes(rng):
    """A head layout: sizes that fill the tiles half of the time, else odd ones."""
    if rng.random() < 0.5:
        P, N = rng.choice([32, 64, 64, 128]), rng.choice([16, 64, 128, 128, 256])
    else:
        P, N = rng.randint(9, 100), rng.randint(9, 200)
    groups = rng.choice([1, 1, 2, 4])
    heads = groups * rng.randint(1, 32 // groups)
    return P, N, groups, heads


def _limit(L, per_token, most):
    return max(1, min(L, int(most / per_token)))


def draw(rng):
    kind = rng.choice(["scan_fwd", "scan_fwd", "scan_fwd", "scan_bwd", "scan_bwd", "token",
                       "conv_fwd", "conv_bwd", "norm_fwd", "norm_bwd"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if kind in ("scan_fwd", "scan_bwd"):
        P, N, groups, heads = _sizes(rng)
        batch = rng.randint(1, 6)
        fwd = kind == "scan_fwd"
        L = _log(rng, 1, 40000 if fwd else 4000)
        # bounds the products of the recurrence and the plain form's chunk matrices
        L = _limit(L, batch * heads * max(P * N, 1700), 5e9 if fwd else 1.2e9)
        return _scan(None, kind, batch, L, heads, P, N, groups, dtype,
                     rng.choice(["zoh", "euler"]), rng.random() < 0.5, rng.random() < 0.4)
    if kind == "token":
        P, N, groups, heads = _sizes(rng)
        return _token(None, _log(rng, 1, 200), heads, P, N, groups, dtype,
                      rng.choice(["zoh", "euler"]), rng.random() < 0.5)
    if kind in ("conv_fwd", "conv_bwd"):
        dim, W = _width(_log(rng, 17, 4500), 1), rng.choice([2, 3, 4, 4])
        batch = rng.randint(1, 8)
        L = _limit(_log(rng, 1, 20000), batch * dim, 2e7)
        return _conv(None, kind, batch, L, dim, W, dtype, rng.random() < 0.5,
                     rng.random() < 0.4)
    groups = rng.choice([1, 1, 2, 8])
    dim = _width(groups * _log(rng, 16, 6000 // groups), groups)
    rows = _limit(_log(rng, 1, 30000), dim, 2e7)
    return _norm(None, kind, rows, dim, groups, dtype, rng.random() < 0.7)


# --------------------------------------------------------------------------- inputs

class _Draw:
    def __init__(self, seed):
        self.g = torch.Generator(device=DEV)
        self.g.manual_seed(seed)

    def normal(self, *shape, dtype=torch.float32, scale=1.0):
        x = torch.randn(*shape, generator=self.g, device=DEV, dtype=torch.float32)
        return (x * scale if scale != 1.0 else x).to(dtype)

    def uniform(self, lo, hi, *shape):
        return torch.rand(*shape, generator=self.g, device=DEV) * (hi - lo) + lo

    def flags(self, batch, L):
        """Starts of packed sequences, a few hundred steps apart."""
        return (torch.rand(batch, L, generator=self.g, device=DEV) < 1 / 200).to(torch.uint8)


def _head_weights(r, heads):
    """A = -1..-16 a head, the skip weight, the step bias of steps 0.001..0.1."""
    return dict(A=-r.uniform(1.0, 16.0, heads), D=r.normal(heads),
                delta_bias=r.uniform(BIAS_LO, BIAS_HI, heads))


def prepare(case, seed):
    c, r = case, _Draw(seed)
    s = {"case": c}
    dt = DTYPES[c["dtype"]]
    k = c["kind"]
    if k in ("scan_fwd", "scan_bwd"):
        b, L, H, P, N, G = (c[n] for n in ("batch", "L", "heads", "P", "N", "groups"))
        # u, B, C are what the convolution wrote: parts of one row a token
        x = r.normal(b, L, H * P + 2 * G * N, dtype=dt)
        s["u"] = x[..., :H * P].unflatten(-1, (H, P))
        s["B"] = x[..., H * P:H * P + G * N].unflatten(-1, (G, N))
        s["C"] = x[..., H * P + G * N:].unflatten(-1, (G, N))
        s["delta"] = r.normal(b, L, H, dtype=dt)
        s.update(_head_weights(r, H))
        s["h0"] = r.normal(b, H, P, N) if c["h0"] else None
        s["reset"] = r.flags(b, L) if c["packed"] else None
        if k == "scan_bwd":
            s["dout"] = r.normal(b, L, H, P, dtype=dt)
    elif k == "token":
        b, H, P, N, G = (c[n] for n in ("batch", "heads", "P", "N", "groups"))
        dim, W = H * P + 2 * G * N, 4
        pool = 2 * b if c["slots"] else b
        s["x"] = r.normal(b, dim, dtype=dt)
        s["w"] = r.normal(dim, W, scale=0.5)
        s["b"] = r.normal(dim, scale=0.5)
        s["window"] = r.normal(pool, W - 1, dim, dtype=dt)
        s["state"] = r.normal(pool, H, P, N)
        s["delta"] = r.normal(b, H, dtype=dt)
        s.update(_head_weights(r, H))
        s["slots"] = None
        if c["slots"]:
            s["slots"] = torch.randperm(pool, generator=r.g, device=DEV)[:b].to(torch.int32)
    elif k in ("conv_fwd", "conv_bwd"):
        b, L, dim, W = c["batch"], c["L"], c["dim"], c["W"]
        s["x"] = r.normal(b, L, dim, dtype=dt)
        s["w"] = r.normal(dim, W, scale=0.5)
        s["b"] = r.normal(dim, scale=0.5)
        s["window"] = r.normal(b, W - 1, dim, dtype=dt) if c["window"] else None
        s["reset"] = r.flags(b, L) if c["packed"] else None
        if k == "conv_bwd":
            s["dout"] = r.normal(b, L, dim, dtype=dt)
    else:
        s["x"] = r.normal(c["rows"], c["dim"], dtype=dt)
        s["z"] = r.normal(c["rows"], c["dim"], dtype=dt)
        s["weight"] = 1.0 + r.normal(c["dim"], scale=0.2)
        if k == "norm_bwd":
            s["dout"] = r.normal(c["rows"], c["dim"], dtype=dt)
    return s


# --------------------------------------------------------------------------- work

def work(case):
    c = case
    e = 2 if c["dtype"] == "bf16" else 4
    k = c["kind"]
    if k in ("scan_fwd", "scan_bwd"):
        b, L, H, P, N, G = (c[n] for n in ("batch", "L", "heads", "P", "N", "groups"))
        seq = b * L * (H * P + H + 2 * G * N) * e + (b * L if c["packed"] else 0)
        st, out = b * H * P * N * 4, b * L * H * P * e
        if k == "scan_fwd":
            # in: the sequences, h0; out: out, the last state.  A state's two
            # products a step: the update and the output's contraction
            return {"bytes": seq + out + st * (2 if c["h0"] else 1) + 3 * H * 4,
                    "flops": 4.0 * b * L * H * P * N}
        # in: the sequences, dout, h0; out: their gradients.  Five products a
        # step: the state, the adjoint, and dC, dB, du
        return {"bytes": seq + out + b * L * (H * P + H + 2 * G * N) * e
                + (2 * st if c["h0"] else 0) + 6 * H * 4,
                "flops": 10.0 * b * L * H * P * N}
    if k == "token":
        b, H, P, N, G = (c[n] for n in ("batch", "heads", "P", "N", "groups"))
        dim, W = H * P + 2 * G * N, 4
        return {"bytes": 2 * b * H * P * N * 4 + b * dim * e * (1 + 2 * (W - 1))
                + b * H * (P + 1) * e + dim * (W + 1) * 4 + 3 * H * 4,
                "flops": b * (5.0 * H * P * N + 2.0 * dim * W)}
    if k in ("conv_fwd", "conv_bwd"):
        n = c["batch"] * c["L"] * c["dim"]
        extra = c["dim"] * (c["W"] + 1) * 4 + (c["batch"] * c["L"] if c["packed"] else 0)
        win = c["batch"] * (c["W"] - 1) * c["dim"] * e
        if k == "conv_fwd":
            return {"bytes": 2 * n * e + extra + win * (2 if c["window"] else 1),
                    "flops": n * (2.0 * c["W"] + 4)}
        return {"bytes": 3 * n * e + 2 * extra + (2 * win if c["window"] else 0),
                "flops": n * (6.0 * c["W"] + 10)}
    n = c["rows"] * c["dim"]
    if k == "norm_fwd":
        return {"bytes": 3 * n * e + c["dim"] * 4, "flops": 10.0 * n}
    return {"bytes": 5 * n * e + 2 * c["dim"] * 4, "flops": 25.0 * n}


# --------------------------------------------------------------------------- plain forms

def _steps(delta, A, bias, disc, softplus=torch.nn.functional.softplus):
    """The step's log decay a = delta A and input weight w of every (token, head)."""
    d = softplus(delta + bias, threshold=60.0)
    a = d * A
    return a, (torch.expm1(a) / A if disc == "zoh" else d)


def _pairwise(a):
    """T[..., i, j] = a_{j+1} + ... + a_i for i >= j and -inf above: sums of
    the terms themselves, not differences of running totals."""
    n = a.shape[-1]
    at = torch.arange(n, device=a.device)
    t = a.unsqueeze(-1).expand(*a.shape, n)
    t = torch.where(at[:, None] > at[None, :], t, torch.zeros((), device=a.device)).cumsum(-2)
    return torch.where(at[:, None] >= at[None, :], t, torch.full((), -math.inf, device=a.device))


def _plain_scan(u, delta, A, B, C, D, bias, h0, reset, disc):
    """out, last state: within chunks as masked products, over chunks as one
    product with the matrix of decays between them."""
    b, L, H, P = u.shape
    G, N = B.shape[2:]
    Q = min(PLAIN_CHUNK, L)
    nc = -(-L // Q)
    pad = nc * Q - L
    a, w = _steps(delta, A, bias, disc)

    def chunks(t):
        t = torch.nn.functional.pad(t, [0, 0] * (t.dim() - 2) + [0, pad])
        return t.unflatten(1, (nc, Q)).transpose(2, 3) if t.dim() > 2 else t.unflatten(1, (nc, Q))

    # sequence number of each token; h0 is number 0's
    ids = torch.zeros(b, nc * Q, device=u.device)
    if reset is not None:
        ids[:, :L] = reset.float().cumsum(1)
        ids[:, L:] = ids[:, L - 1:L]
    ids = ids.unflatten(1, (nc, Q))                                   # b c q
    at = chunks(a)                                                    # b c h q
    x = chunks(u * w.unsqueeze(-1))                                   # b c h q p
    Bc = chunks(B).repeat_interleave(H // G, 2)                       # b c h q n
    Cc = chunks(C).repeat_interleave(H // G, 2)
    same = (ids.unsqueeze(-1) == ids.unsqueeze(-2)).unsqueeze(2)      # b c 1 q s
    decay = torch.exp(_pairwise(at)) * same
    out = ((Cc @ Bc.transpose(-1, -2)) * decay) @ x
    # what each chunk adds to the state at its end, and h0 before all of them
    add = (x * decay[..., -1, :, None]).transpose(-1, -2) @ Bc        # b c h p n
    first = torch.zeros(b, 1, H, P, N, device=u.device) if h0 is None else h0.unsqueeze(1)
    add = torch.cat([first, add], 1).transpose(1, 2)                  # b h c+1 p n
    end_id = torch.cat([torch.zeros(b, 1, device=u.device), ids[..., -1]], 1)
    total = torch.nn.functional.pad(at.sum(-1), [0, 0, 1, 0]).transpose(1, 2)   # b h c+1
    between = torch.exp(_pairwise(total)) * (end_id.unsqueeze(-1) == end_id.unsqueeze(-2)).unsqueeze(1)
    states = (between @ add.flatten(-2)).unflatten(-1, (P, N)).transpose(1, 2)  # b c+1 h p n
    into = torch.exp(at.cumsum(-1)) * (ids == end_id[:, :-1, None]).unsqueeze(2)
    out = out + (Cc @ states[:, :-1].transpose(-1, -2)) * into.unsqueeze(-1)
    out = out.transpose(2, 3).reshape(b, nc * Q, H, P)[:, :L] + D[:, None] * u
    return out, states[:, -1]


def _plain_conv(x, w, b, window, reset):
    """silu of the causal sum over the last W tokens of the same sequence."""
    B_, L, dim = x.shape
    W = w.shape[1]
    head = torch.zeros(B_, W - 1, dim, device=x.device) if window is None else window
    xx = torch.cat([head, x], 1)
    ids = torch.zeros(B_, L + W - 1, device=x.device)
    if reset is not None:
        ids[:, W - 1:] = reset.float().cumsum(1)
    taps = xx.unfold(1, W, 1)                                         # b l dim w
    same = ids.unfold(1, W, 1) == ids[:, W - 1:, None]                # b l w
    pre = (torch.where(same.unsqueeze(2), taps, torch.zeros((), device=x.device)) * w).sum(-1) + b
    return pre * torch.sigmoid(pre), xx


def _window_after(xx, reset, W):
    """The last W - 1 inputs of the sequence that goes on: what decoding continues from."""
    tail = xx[:, -(W - 1):]
    if reset is None:
        return tail.contiguous()
    ids = torch.zeros(xx.shape[:2], device=xx.device)
    ids[:, W - 1:] = reset.float().cumsum(1)
    return torch.where((ids[:, -(W - 1):] == ids[:, -1:]).unsqueeze(-1), tail,
                       torch.zeros((), device=xx.device, dtype=xx.dtype))


def _plain_norm(x, z, weight, groups, gate_first, eps=1e-5):
    gate = z * torch.sigmoid(z)
    v = (x * gate if gate_first else x).unflatten(-1, (groups, -1))
    y = (v * torch.rsqrt(v.square().mean(-1, keepdim=True) + eps)).flatten(-2) * weight
    return y if gate_first else y * gate


def _leaf(t):
    return None if t is None else t.float().detach().requires_grad_(True)


def _grads(outs, douts, leaves, like):
    """Gradients of the named leaves, each rounded once to its tensor's type."""
    names = [n for n in leaves if leaves[n] is not None]
    g = torch.autograd.grad(outs, [leaves[n] for n in names], douts)
    return {"d" + n: v.to(like[n].dtype) for n, v in zip(names, g)}


def _run_plain(s):
    c = s["case"]
    k = c["kind"]
    f = lambda n: None if s[n] is None else s[n].float()  # noqa: E731
    if k == "scan_fwd":
        out, last = _plain_scan(f("u"), f("delta"), s["A"], f("B"), f("C"), s["D"],
                                s["delta_bias"], s["h0"], s["reset"], c["disc"])
        return {"out": out.to(s["u"].dtype), "last_state": last}
    if k == "scan_bwd":
        v = {n: _leaf(s[n]) for n in ("u", "delta", "A", "B", "C", "D", "delta_bias", "h0")}
        out, _ = _plain_scan(v["u"], v["delta"], v["A"], v["B"], v["C"], v["D"], v["delta_bias"],
                             v["h0"], s["reset"], c["disc"])
        return _grads(out, f("dout"), v, s)
    if k == "token":
        H, P, N, G = c["heads"], c["P"], c["N"], c["groups"]
        at = slice(None) if s["slots"] is None else s["slots"].long()
        y, xx = _plain_conv(f("x").unsqueeze(1), s["w"], s["b"], s["window"][at].float(), None)
        s["window"][at] = xx[:, 1:].to(s["window"].dtype)
        y = y[:, 0].to(s["x"].dtype).float()
        u, B, C = y.split([H * P, G * N, G * N], -1)
        u = u.unflatten(-1, (H, P))
        B = B.unflatten(-1, (G, N)).repeat_interleave(H // G, 1)
        C = C.unflatten(-1, (G, N)).repeat_interleave(H // G, 1)
        a, w = _steps(f("delta"), s["A"], s["delta_bias"], c["disc"])
        h = s["state"][at] * torch.exp(a)[..., None, None] \
            + (u * w.unsqueeze(-1)).unsqueeze(-1) * B.unsqueeze(2)
        s["state"][at] = h
        out = (h * C.unsqueeze(2)).sum(-1) + s["D"][:, None] * u
        return {"out": out.to(s["x"].dtype), "state": s["state"], "window": s["window"]}
    if k == "conv_fwd":
        y, xx = _plain_conv(f("x"), s["w"], s["b"], f("window"), s["reset"])
        return {"out": y.to(s["x"].dtype),
                "window": _window_after(xx, s["reset"], c["W"]).to(s["x"].dtype)}
    if k == "conv_bwd":
        v = {n: _leaf(s[n]) for n in ("x", "w", "b", "window")}
        y, _ = _plain_conv(v["x"], v["w"], v["b"], v["window"], s["reset"])
        return _grads(y, f("dout"), v, s)
    if k == "norm_fwd":
        y = _plain_norm(f("x"), f("z"), s["weight"], c["groups"], c["gate_first"])
        return {"out": y.to(s["x"].dtype)}
    v = {n: _leaf(s[n]) for n in ("x", "z", "weight")}
    y = _plain_norm(v["x"], v["z"], v["weight"], c["groups"], c["gate_first"])
    return _grads(y, f("dout"), v, s)


# --------------------------------------------------------------------------- the framework's calls

def _run_own(s):
    ms, c = _ms(), s["case"]
    k = c["kind"]
    if k == "scan_fwd":
        out, last = ms.heads_scan_fwd(s["u"], s["delta"], s["A"], s["B"], s["C"], s["D"],
                                      s["delta_bias"], s["h0"], disc=c["disc"], reset=s["reset"],
                                      return_last_state=True)
        return {"out": out, "last_state": last}
    if k == "scan_bwd":
        return ms.heads_scan_bwd(s["u"], s["delta"], s["A"], s["B"], s["C"], s["D"],
                                 s["delta_bias"], s["dout"], s["h0"], disc=c["disc"],
                                 reset=s["reset"])
    if k == "token":
        H, P, N, G = c["heads"], c["P"], c["N"], c["groups"]
        y = ms.conv1d_tokens_update(s["x"], s["window"], s["w"], s["b"], slots=s["slots"])
        u = y[:, :H * P].unflatten(-1, (H, P))
        B = y[:, H * P:H * P + G * N].unflatten(-1, (G, N))
        C = y[:, H * P + G * N:].unflatten(-1, (G, N))
        out = ms.heads_state_update(s["state"], u, s["delta"], s["A"], B, C, s["D"],
                                    s["delta_bias"], disc=c["disc"], slots=s["slots"])
        return {"out": out, "state": s["state"], "window": s["window"]}
    if k == "conv_fwd":
        out, window = ms.conv1d_tokens_fwd(s["x"], s["w"], s["b"], window=s["window"],
                                           reset=s["reset"], return_window=True)
        return {"out": out, "window": window}
    if k == "conv_bwd":
        return ms.conv1d_tokens_bwd(s["x"], s["w"], s["b"], s["dout"], window=s["window"],
                                    reset=s["reset"])
    if k == "norm_fwd":
        return {"out": ms.gated_norm_fwd(s["x"], s["z"], s["weight"], groups=c["groups"],
                                         gate_first=c["gate_first"])}
    return ms.gated_norm_bwd(s["x"], s["z"], s["weight"], s["dout"], groups=c["groups"],
                             gate_first=c["gate_first"])


def run(state):
    return _run_own(state) if own else _run_plain(state)


# --------------------------------------------------------------------------- 64 bits

class _Recurrence:
    """The scan step by step in 64 bits, from its definition."""

    def __init__(self, s):
        c = s["case"]
        d = lambda n: None if s[n] is None else s[n].double()  # noqa: E731
        self.u, self.B, self.C, self.A, self.D = d("u"), d("B"), d("C"), d("A"), d("D")
        b, L, H, P = self.u.shape
        self.rep = H // self.B.shape[2]
        raw = d("delta") + d("delta_bias")
        self.raw = raw
        self.dt = torch.logaddexp(raw, torch.zeros_like(raw))
        self.keep = torch.ones(b, L, 1, dtype=torch.float64, device=DEV)
        if s["reset"] is not None:
            self.keep = 1.0 - s["reset"].double().unsqueeze(-1)
        self.decay = torch.exp(self.dt * self.A) * self.keep
        self.zoh = c["disc"] == "zoh"
        self.w = torch.expm1(self.dt * self.A) / self.A if self.zoh else self.dt
        self.h0 = d("h0")
        if self.h0 is None:
            self.h0 = torch.zeros(b, H, P, self.B.shape[3], dtype=torch.float64, device=DEV)

    def row(self, t, t_at):
        return t[:, t_at].repeat_interleave(self.rep, 1)

    def step(self, h, t):
        x = self.u[:, t] * self.w[:, t].unsqueeze(-1)
        return h.mul(self.decay[:, t, :, None, None]).addcmul_(x.unsqueeze(-1),
                                                               self.row(self.B, t).unsqueeze(2))


def _exact_scan_fwd(s):
    r = _Recurrence(s)
    h, out = r.h0, torch.empty_like(r.u)
    for t in range(r.u.shape[1]):
        h = r.step(h, t)
        out[:, t] = (h @ r.row(r.C, t).unsqueeze(-1)).squeeze(-1)
    return {"out": out + r.D[:, None] * r.u, "last_state": h}


def _exact_scan_bwd(s):
    """The chain rule of the recurrence, backwards in time; the states are
    made again from every 64th."""
    r, dy = _Recurrence(s), s["dout"].double()
    b, L, H, P = r.u.shape
    G, N = r.B.shape[2:]
    marks, h = [], r.h0
    for t in range(L):
        if t % 64 == 0:
            marks.append(h)
        h = r.step(h, t)
    z = lambda *n: torch.zeros(*n, dtype=torch.float64, device=DEV)  # noqa: E731
    du, dB, dC = r.D[:, None] * dy, z(b, L, G, N), z(b, L, G, N)
    dlog, dw = z(b, L, H), z(b, L, H)
    g = torch.zeros_like(r.h0)
    for t0 in reversed(range(0, L, 64)):
        hs = [marks[t0 // 64]]
        for t in range(t0, min(L, t0 + 64)):
            hs.append(r.step(hs[-1], t))
        for t in reversed(range(t0, min(L, t0 + 64))):
            g = g.addcmul(dy[:, t].unsqueeze(-1), r.row(r.C, t).unsqueeze(2))
            dC[:, t] = (dy[:, t].unsqueeze(2) @ hs[t - t0 + 1]).squeeze(2).unflatten(1, (G, -1)).sum(2)
            gB = (g @ r.row(r.B, t).unsqueeze(-1)).squeeze(-1)
            du[:, t] += gB * r.w[:, t].unsqueeze(-1)
            dw[:, t] = (gB * r.u[:, t]).sum(-1)
            xw = r.u[:, t] * r.w[:, t].unsqueeze(-1)
            dB[:, t] = (xw.unsqueeze(2) @ g).squeeze(2).unflatten(1, (G, -1)).sum(2)
            g = g * r.decay[:, t, :, None, None]
            dlog[:, t] = (g * hs[t - t0]).sum((-1, -2))
    x = r.dt * r.A
    if r.zoh:
        ddt = dlog * r.A + dw * torch.exp(x)
        # d/dA of (e^{dt A} - 1) / A
        dA = dlog * r.dt + dw * (r.dt * torch.exp(x) - r.w) / r.A
    else:
        ddt, dA = dlog * r.A + dw, dlog * r.dt
    ddelta = ddt * torch.sigmoid(r.raw)
    got = {"du": du, "ddelta": ddelta, "dA": dA.sum((0, 1)), "dB": dB, "dC": dC,
           "dD": (dy * r.u).sum((0, 1, 3)), "ddelta_bias": ddelta.sum((0, 1))}
    if s["h0"] is not None:
        got["dh0"] = g
    return got


def _exact_conv(s, upto=None):
    """The convolution tap by tap in 64 bits: pre, and the input before it."""
    x, w, b = s["x"].double(), s["w"].double(), s["b"].double()
    n, L, dim = x.shape
    W = w.shape[1]
    xx = torch.cat([torch.zeros(n, W - 1, dim, dtype=x.dtype, device=DEV)
                    if s["window"] is None else s["window"].double(), x], 1)
    seq = torch.zeros(n, L + W - 1, dtype=torch.int64, device=DEV)
    if s["reset"] is not None:
        seq[:, W - 1:] = s["reset"].long().cumsum(1)
    ok = [(seq[:, j:j + L] == seq[:, W - 1:]).double().unsqueeze(-1) for j in range(W)]
    pre = b + sum(ok[j] * xx[:, j:j + L] * w[:, j] for j in range(W))
    return pre, xx, ok, seq


def _exact_norm(s):
    c = s["case"]
    x, z, w = s["x"].double(), s["z"].double(), s["weight"].double()
    sg = 1 / (1 + torch.exp(-z))
    gate = z * sg
    v = (x * gate if c["gate_first"] else x).unflatten(-1, (c["groups"], -1))
    r = 1 / torch.sqrt((v * v).mean(-1, keepdim=True) + 1e-5)
    return x, z, w, sg, gate, v, r


def exact(case, seed):
    s = prepare(case, seed)
    k = case["kind"]
    if k in ("scan_fwd", "scan_bwd"):
        # a step is a handful of launches on the whole state
        state = case["batch"] * case["heads"] * case["P"] * case["N"]
        cost = case["L"] * max(40e-6 if k == "scan_fwd" else 250e-6,
                               state * (5e-11 if k == "scan_fwd" else 2e-10))
        if cost > 12:
            return None
        return _exact_scan_fwd(s) if k == "scan_fwd" else _exact_scan_bwd(s)
    if k == "token":
        c = case
        H, P, N, G = c["heads"], c["P"], c["N"], c["groups"]
        at = torch.arange(c["batch"], device=DEV) if s["slots"] is None else s["slots"].long()
        one = {"x": s["x"].unsqueeze(1), "w": s["w"], "b": s["b"], "window": s["window"][at],
               "reset": None}
        pre, xx, _, _ = _exact_conv(one)
        # the scan reads the convolution's output in its stored type
        y = (pre / (1 + torch.exp(-pre)))[:, 0].float().to(s["x"].dtype)
        v = dict(s, reset=None, u=y[:, None, :H * P].unflatten(-1, (H, P)),
                 B=y[:, None, H * P:H * P + G * N].unflatten(-1, (G, N)),
                 C=y[:, None, H * P + G * N:].unflatten(-1, (G, N)),
                 delta=s["delta"].unsqueeze(1), h0=s["state"][at])
        got = _exact_scan_fwd(v)
        state, window = s["state"].double(), s["window"].double()
        state[at], window[at] = got["last_state"], xx[:, 1:]
        return {"out": got["out"][:, 0], "state": state, "window": window}
    if k in ("conv_fwd", "conv_bwd"):
        pre, xx, ok, seq = _exact_conv(s)
        L, W = case["L"], case["W"]
        sg = 1 / (1 + torch.exp(-pre))
        if k == "conv_fwd":
            live = (seq[:, L:] == seq[:, -1:]).double().unsqueeze(-1)
            return {"out": pre * sg, "window": xx[:, L:] * live}
        dpre = s["dout"].double() * sg * (1 + pre * (1 - sg))
        dxx, dw = torch.zeros_like(xx), []
        for j in range(W):
            dxx[:, j:j + L] += ok[j] * dpre * s["w"][:, j].double()
            dw.append((ok[j] * dpre * xx[:, j:j + L]).sum((0, 1)))
        got = {"dx": dxx[:, W - 1:], "dw": torch.stack(dw, 1), "db": dpre.sum((0, 1))}
        if s["window"] is not None:
            got["dwindow"] = dxx[:, :W - 1]
        return got
    x, z, w, sg, gate, v, r = _exact_norm(s)
    first = case["gate_first"]
    hat = (v * r).flatten(-2)
    if k == "norm_fwd":
        return {"out": hat * w if first else hat * w * gate}
    dy = s["dout"].double()
    dhat = (dy * w if first else dy * w * gate).unflatten(-1, (case["groups"], -1))
    dv = (r * (dhat - v * r * r * (dhat * v).mean(-1, keepdim=True))).flatten(-2)
    dgate = dv * x if first else dy * w * hat
    return {"dx": dv * gate if first else dv, "dz": dgate * sg * (1 + z * (1 - sg)),
            "dweight": (dy * hat if first else dy * hat * gate).sum(0)}

"""What is measured of the recurrent block's operators: the gated linear
recurrence (prompts, training, single tokens) and the root-mean-square norm with
the residual's addition that opens each block (in the activations' type or in
8 bits, and its backward).

Every case is one pass through a public operator; a training pass of the
recurrence is its forward and its backward.  `run` computes it in elementary
torch operations in 32 bits, or, where `own` is true, calls
scan_selective_fwd_amd.  Layouts: x, r, i, z, out (batch, L, dim), A (dim,),
states (batch, dim) or a pool (pool, dim) float32; rows of the norm (rows, dim).

The recurrence, channel by channel, with s(v) = 1 / (1 + exp(-v)):

    a_t = exp(A s(r_t)),   h_t = a_t h_{t-1} + sqrt(1 - a_t^2) s(i_t) x_t
    out_t = h_t            (times z_t s(z_t) where z is given)

A flagged step starts another sequence: the state before it is left out.  The
norm: res = x + residual, kept in the residual's type, and of what is kept
out = res / sqrt(mean(res^2) + eps) * weight; in 8 bits (e4m3) out is divided by
its row's scale max|out| / 448.
"""
import math

import torch

own = False

DEV = "cuda"
EPS = 1e-5
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
FP8, FP8_MAX, SCALE_FLOOR = torch.float8_e4m3fn, 448.0, 2.0 ** -100


def _ms():
    import scan_selective_fwd_amd as ms
    return ms


# --------------------------------------------------------------------------- cases

def _rec(name, kind, batch, L, dim, dtype, gate, h0, packed):
    c = dict(kind=kind, batch=batch, L=L, dim=dim, dtype=dtype, gate=gate, h0=h0, packed=packed)
    return dict(c, name=name) if name else c


def _token(name, batch, dim, dtype, gate, slots):
    c = dict(kind="rec_token", batch=batch, dim=dim, dtype=dtype, gate=gate, slots=slots)
    return dict(c, name=name) if name else c


def _norm(name, kind, rows, dim, dtype, res_dtype):
    c = dict(kind=kind, rows=rows, dim=dim, dtype=dtype, res_dtype=res_dtype)
    return dict(c, name=name) if name else c


def listed():
    return [
        # the next piece of one user's prompt, continuing from its state: latency counts
        _rec("rec-piece", "rec_fwd", 1, 200, 1536, "bf16", False, True, False),
        # a batch of prompts at the benchmark layer's width, the block's gate on the output
        _rec("rec-batch", "rec_fwd", 8, 2048, 1536, "bf16", True, False, False),
        # one very long document: few channels, all the work along the sequence
        _rec("rec-long", "rec_fwd", 1, 131072, 1536, "bf16", False, False, False),
        # packed ragged prompts in float32, an odd width
        _rec("rec-packed-f32", "rec_fwd", 3, 1000, 1003, "f32", True, True, True),
        # a training pass of a wide layer (2 x 2048 x 5120)
        _rec("rec-train", "rec_train", 2, 2048, 5120, "bf16", True, False, False),
        # packed training rows in float32, with the entering state's gradient
        _rec("rec-train-packed-f32", "rec_train", 4, 777, 1025, "f32", False, True, True),
        # one token for each of 256 users, states picked from a pool by slot
        _token("rec-token-pool", 256, 5120, "bf16", True, True),
        # one token of one user's block: the smallest call
        _norm("norm-token", "norm_fwd", 1, 1536, "bf16", "bf16"),
        # a batch of prompts
        _norm("norm-prompt", "norm_fwd", 16384, 1536, "bf16", "bf16"),
        # a batch of prompts in 8 bits, the residual stream in float32
        _norm("norm-prompt-8bit", "norm_fp8", 4096, 5120, "bf16", "f32"),
        # a batch of single tokens in 8 bits, an odd width
        _norm("norm-token-8bit", "norm_fp8", 129, 2047, "bf16", "bf16"),
        # the backward in training
        _norm("norm-train", "norm_bwd", 4096, 5120, "bf16", "bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _limit(n, per, most):
    return max(1, min(n, int(most / per)))


def _dim(rng, lo, hi):
    """A width that fills whole cache lines half of the time, else any."""
    dim = _log(rng, lo, hi)
    return max(64, dim // 64 * 64) if rng.random() < 0.5 else dim


def draw(rng):
    kind = rng.choice(["rec_fwd", "rec_fwd", "rec_train", "rec_train", "rec_token", "norm_fwd",
                       "norm_fp8", "norm_bwd"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    half = lambda: rng.random() < 0.5  # noqa: E731
    if kind in ("rec_fwd", "rec_train"):
        fwd = kind == "rec_fwd"
        dim, batch = _dim(rng, 17, 6000), rng.randint(1, 9)
        L = _limit(_log(rng, 1, 60000 if fwd else 8000), batch * dim, 1e8 if fwd else 2e7)
        return _rec(None, kind, batch, L, dim, dtype, half(), half(), rng.random() < 0.4)
    if kind == "rec_token":
        return _token(None, _log(rng, 1, 512), _dim(rng, 17, 8000), dtype, half(), half())
    dim = _dim(rng, 17, 12000)
    rows = _limit(_log(rng, 1, 30000), dim, 2.5e7)
    return _norm(None, kind, rows, dim, dtype, "f32" if dtype == "f32" or half() else "bf16")


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


def _decay(r, dim):
    """A of channels that keep between 0.9 and 0.999 of the state at an eighth of the gate."""
    return 8.0 * torch.log(r.uniform(0.9, 0.999, dim))


def prepare(case, seed):
    c, r = case, _Draw(seed)
    s = {"case": c}
    dt = DTYPES[c["dtype"]]
    k = c["kind"]
    if k in ("rec_fwd", "rec_train"):
        b, L, d = c["batch"], c["L"], c["dim"]
        s["x"] = r.normal(b, L, d, dtype=dt)
        gates = r.normal(b, L, 2 * d, dtype=dt)      # one projection writes both gates
        s["r"], s["i"] = gates[..., :d], gates[..., d:]
        s["A"] = _decay(r, d)
        s["z"] = r.normal(b, L, d, dtype=dt) if c["gate"] else None
        s["h0"] = r.normal(b, d) if c["h0"] else None
        s["reset"] = r.flags(b, L) if c["packed"] else None
        if k == "rec_train":
            s["dout"] = r.normal(b, L, d, dtype=dt)
    elif k == "rec_token":
        b, d = c["batch"], c["dim"]
        pool = 2 * b if c["slots"] else b
        s["x"] = r.normal(b, d, dtype=dt)
        gates = r.normal(b, 2 * d, dtype=dt)
        s["r"], s["i"] = gates[..., :d], gates[..., d:]
        s["A"] = _decay(r, d)
        s["z"] = r.normal(b, d, dtype=dt) if c["gate"] else None
        s["state"] = r.normal(pool, d)
        s["slots"] = None
        if c["slots"]:
            s["slots"] = torch.randperm(pool, generator=r.g, device=DEV)[:b].to(torch.int32)
    else:
        rows, d, rt = c["rows"], c["dim"], DTYPES[c["res_dtype"]]
        s["weight"] = 1.0 + r.normal(d, scale=0.2)
        # a residual stream some blocks deep against one block's output
        s["residual"] = r.normal(rows, d, dtype=rt, scale=3.0)
        if k == "norm_bwd":
            s["dout"] = r.normal(rows, d, dtype=dt)
            s["dres"] = r.normal(rows, d, dtype=rt)
        else:
            s["x"] = r.normal(rows, d, dtype=dt)
    return s


# --------------------------------------------------------------------------- work

def work(case):
    c = case
    e = 2 if c["dtype"] == "bf16" else 4
    k = c["kind"]
    if k in ("rec_fwd", "rec_train"):
        n, st = c["batch"] * c["L"] * c["dim"], c["batch"] * c["dim"] * 4
        ins = 4 if c["gate"] else 3
        flags = c["batch"] * c["L"] if c["packed"] else 0
        fwd = {"bytes": n * e * (ins + 1) + flags + st * (2 if c["h0"] else 1) + c["dim"] * 4,
               "flops": n * (25.0 if c["gate"] else 20.0)}
        if k == "rec_fwd":
            return fwd
        # the backward reads the inputs and dout, and writes a gradient for each input
        return {"bytes": fwd["bytes"] + n * e * (2 * ins + 1) + flags
                + (2 * st if c["h0"] else 0) + 2 * c["dim"] * 4, "flops": 3.5 * fwd["flops"]}
    if k == "rec_token":
        n = c["batch"] * c["dim"]
        return {"bytes": n * (8 + e * (5 if c["gate"] else 4)) + c["dim"] * 4
                + (4 * c["batch"] if c["slots"] else 0), "flops": 25.0 * n}
    n, er = c["rows"] * c["dim"], 2 if c["res_dtype"] == "bf16" else 4
    if k == "norm_bwd":   # in: res, dout, dres; out: dx, and dresidual where it has another type
        return {"bytes": n * (2 * er + 2 * e + (er if er != e else 0)) + 2 * c["dim"] * 4,
                "flops": 12.0 * n}
    out = e if k == "norm_fwd" else 1
    return {"bytes": n * (e + 2 * er + out) + c["dim"] * 4
            + (c["rows"] * 4 if k == "norm_fp8" else 0),
            "flops": n * (5.0 if k == "norm_fwd" else 8.0)}


# --------------------------------------------------------------------------- plain forms

def _plain_step(x, r, i, A):
    """Decay and input of every step."""
    y = A * torch.sigmoid(r)
    return torch.exp(y), torch.sqrt(-torch.expm1(2.0 * y)) * torch.sigmoid(i) * x


def _plain_recurrence(x, r, i, A, z, h0, reset):
    """out, last state: the steps' affine maps joined over 1, 2, 4, ... steps."""
    L = x.shape[1]
    a, h = _plain_step(x, r, i, A)
    if reset is not None:
        a = torch.where(reset.unsqueeze(-1) != 0, torch.zeros((), device=a.device), a)
    if h0 is not None:
        h = torch.cat([h[:, :1] + a[:, :1] * h0.unsqueeze(1), h[:, 1:]], 1)
    k = 1
    while k < L:
        h = torch.cat([h[:, :k], h[:, k:] + a[:, k:] * h[:, :-k]], 1)
        a = torch.cat([a[:, :k], a[:, k:] * a[:, :-k]], 1)
        k *= 2
    return (h if z is None else h * (z * torch.sigmoid(z))), h[:, -1]


def _plain_norm(s):
    """The sum as the stream keeps it, and its norm."""
    res = (s["x"].float() + s["residual"].float()).to(s["residual"].dtype)
    v = res.float()
    return res, v * torch.rsqrt(v.square().mean(-1, keepdim=True) + EPS) * s["weight"]


def _run_plain(s):
    c = s["case"]
    k = c["kind"]
    f = lambda n: None if s[n] is None else s[n].float()  # noqa: E731
    if k == "rec_fwd":
        out, last = _plain_recurrence(f("x"), f("r"), f("i"), s["A"], f("z"), s["h0"], s["reset"])
        return {"out": out.to(s["x"].dtype), "last_state": last.contiguous()}
    if k == "rec_train":
        v = {n: s[n].float().detach().requires_grad_(True)
             for n in ("x", "r", "i", "A", "z", "h0") if s[n] is not None}
        out, _ = _plain_recurrence(v["x"], v["r"], v["i"], v["A"], v.get("z"), v.get("h0"),
                                   s["reset"])
        g = torch.autograd.grad(out, list(v.values()), f("dout"))
        return dict({"d" + n: d.to(s[n].dtype) for n, d in zip(v, g)},
                    out=out.detach().to(s["x"].dtype))
    if k == "rec_token":
        at = slice(None) if s["slots"] is None else s["slots"].long()
        a, v = _plain_step(f("x"), f("r"), f("i"), s["A"])
        h = a * s["state"][at] + v
        s["state"][at] = h
        if s["z"] is not None:
            h = h * (f("z") * torch.sigmoid(f("z")))
        return {"out": h.to(s["x"].dtype), "state": s["state"]}
    if k == "norm_fwd":
        res, y = _plain_norm(s)
        return {"out": y.to(s["x"].dtype), "residual": res}
    if k == "norm_fp8":
        res, y = _plain_norm(s)
        scale = y.abs().amax(-1, keepdim=True).clamp_min(SCALE_FLOOR) / FP8_MAX
        return {"out": (y / scale).to(FP8), "scale": scale.squeeze(-1), "residual": res}
    v, dy = f("residual"), f("dout")
    r = torch.rsqrt(v.square().mean(-1, keepdim=True) + EPS)
    dhat = dy * s["weight"]
    d = f("dres") + r * (dhat - v * (r * r * (dhat * v).mean(-1, keepdim=True)))
    return {"dx": d.to(s["dout"].dtype), "dresidual": d.to(s["residual"].dtype),
            "dweight": (dy * v * r).sum(0)}


# --------------------------------------------------------------------------- the framework's calls

def _run_own(s):
    ms, c = _ms(), s["case"]
    k = c["kind"]
    if k == "rec_fwd":
        out, last = ms.gated_recurrence_fwd(s["x"], s["r"], s["i"], s["A"], s["z"], s["h0"],
                                            reset=s["reset"], return_last_state=True)
        return {"out": out, "last_state": last}
    if k == "rec_train":
        kept = torch.empty(ms.gated_recurrence_checkpoint_shape(c["batch"], c["L"], c["dim"]),
                           dtype=torch.float32, device=DEV)
        out = ms.gated_recurrence_fwd(s["x"], s["r"], s["i"], s["A"], s["z"], s["h0"],
                                      reset=s["reset"], checkpoints=kept)
        g = ms.gated_recurrence_bwd(s["x"], s["r"], s["i"], s["A"], s["z"], s["dout"], s["h0"],
                                    reset=s["reset"], checkpoints=kept)
        return dict(g, out=out)
    if k == "rec_token":
        out = ms.gated_recurrence_update(s["state"], s["x"], s["r"], s["i"], s["A"], s["z"],
                                         slots=s["slots"])
        return {"out": out, "state": s["state"]}
    if k == "norm_fwd":
        out, res = ms.residual_norm_fwd(s["x"], s["residual"], s["weight"], eps=EPS)
        return {"out": out, "residual": res}
    if k == "norm_fp8":
        out, scale, res = ms.residual_norm_fp8(s["x"], s["residual"], s["weight"], eps=EPS)
        return {"out": out, "scale": scale, "residual": res}
    return ms.residual_norm_bwd(s["residual"], s["weight"], s["dout"], s["dres"], eps=EPS)


def run(state):
    return _run_own(state) if own else _run_plain(state)


# --------------------------------------------------------------------------- 64 bits

def _sig(v):
    return 1.0 / (1.0 + torch.exp(-v))


class _Steps:
    """The factors of every step, step by step in 64 bits."""

    def __init__(self, s):
        d = lambda n: None if s.get(n) is None else s[n].double()  # noqa: E731
        self.x, self.A, self.z = d("x"), d("A"), d("z")
        self.r, self.i = _sig(d("r")), _sig(d("i"))
        y = self.A * self.r
        self.a = torch.exp(y)
        self.m = torch.sqrt((1.0 - self.a) * (1.0 + self.a))
        self.v = self.m * self.i * self.x
        self.kept = self.a      # what of the state before goes on
        if s.get("reset") is not None:
            self.kept = self.a * (s["reset"] == 0).double().unsqueeze(-1)

    def states(self, h0):
        """The state before each step, and the last."""
        L = self.x.shape[1]
        h = torch.zeros_like(self.x[:, 0]) if h0 is None else h0.double()
        before = torch.empty_like(self.v)
        for t in range(L):
            before[:, t] = h
            h = self.kept[:, t] * h + self.v[:, t]
        return before, h


def _exact_recurrence(s, train):
    q = _Steps(s)
    before, last = q.states(s["h0"])
    h = q.kept * before + q.v
    gate = 1.0 if q.z is None else q.z * _sig(q.z)
    if not train:
        return {"out": h * gate, "last_state": last}
    dy = s["dout"].double()
    got = {"out": h * gate}
    if q.z is not None:
        sz = _sig(q.z)
        got["dz"] = dy * h * sz * (1.0 + q.z * (1.0 - sz))
    g = torch.empty_like(h)                    # gradient at each state
    after = torch.zeros_like(last)
    for t in reversed(range(h.shape[1])):
        g[:, t] = dy[:, t] * (gate if q.z is None else gate[:, t]) + after
        after = q.kept[:, t] * g[:, t]
    if s["h0"] is not None:
        got["dh0"] = after
    got["dx"] = g * q.m * q.i
    got["di"] = g * q.m * q.x * q.i * (1.0 - q.i)
    dlog = g * (q.kept * before - q.i * q.x * q.a * q.a / q.m)   # at log a
    got["dr"] = dlog * q.A * q.r * (1.0 - q.r)
    got["dA"] = (dlog * q.r).sum((0, 1))
    return got


def exact(case, seed):
    s = prepare(case, seed)
    k = case["kind"]
    if k in ("rec_fwd", "rec_train"):
        return _exact_recurrence(s, k == "rec_train")
    if k == "rec_token":
        at = torch.arange(case["batch"], device=DEV) if s["slots"] is None else s["slots"].long()
        q = _Steps(s)
        state = s["state"].double()
        h = q.a * state[at] + q.v
        state[at] = h
        return {"out": h if q.z is None else h * q.z * _sig(q.z), "state": state}
    w, res = s["weight"].double(), s["residual"].double()
    if k != "norm_bwd":
        total = res + s["x"].double()
        res = total.to(s["residual"].dtype).double()     # the norm is of what is kept
    root = torch.sqrt((res * res).sum(-1, keepdim=True) / case["dim"] + EPS)
    if k == "norm_fwd":
        return {"out": res / root * w, "residual": total}
    if k == "norm_fp8":
        y = res / root * w
        scale = y.abs().max(-1, keepdim=True).values / FP8_MAX
        return {"out": y / scale, "scale": scale.squeeze(-1), "residual": total}
    dy = s["dout"].double()
    hat = res / root
    inner = dy * w
    d = (inner - hat * (inner * hat).sum(-1, keepdim=True) / case["dim"]) / root
    d = d + s["dres"].double()
    return {"dx": d, "dresidual": d, "dweight": (dy * hat).sum(0)}

"""The recurrent block's operators together: a block of them against the 64-bit
reference, whole prompts against pieces and single tokens, captured into graphs and
replayed, on other streams, and the example."""
import os
import sys

import pytest
import torch

import recurrent_reference as R

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                                "examples"))
F32 = torch.float32


@pytest.fixture(scope="module")
def ms():
    import scan_selective_fwd_amd as m
    assert torch.cuda.is_available()
    return m


def block(ms, p, x, stream, h0=None, reset=None, **kw):
    """norm -> gates -> recurrence -> norm, with weights p; returns out, stream, state."""
    y, s = ms.residual_norm(x, stream, p["w1"])
    u, r, i, z = (y.unsqueeze(-2) * p["mix"]).unbind(-2)
    h, last = ms.gated_recurrence(u.contiguous(), r, i, p["A"], z, h0, reset=reset,
                                  return_last_state=True)
    out, s = ms.residual_norm(h, s, p["w2"])
    return out, s, last


def reference(p, x, stream, h0, reset):
    """The same in 64 bits on the CPU, differentiable."""
    def norm(v, w):
        return v / torch.sqrt(v.square().mean(-1, keepdim=True) + 1e-5) * w
    s = x + stream
    y = norm(s, p["w1"])
    u, r, i, z = (y.unsqueeze(-2) * p["mix"]).unbind(-2)
    a = torch.exp(p["A"] * torch.sigmoid(r))
    v = torch.sqrt(1 - a * a) * torch.sigmoid(i) * u
    h, hs = h0, []
    for t in range(x.shape[1]):
        keep = a[:, t] * (reset[:, t, None] == 0)
        h = keep * h + v[:, t]
        hs.append(h)
    s = s + torch.stack(hs, 1) * z * torch.sigmoid(z)
    return norm(s, p["w2"]), s, h


def weights(dim, seed=1):
    g = torch.Generator().manual_seed(seed)
    f = lambda *s: torch.randn(*s, generator=g).double()  # noqa: E731
    return dict(w1=1 + 0.2 * f(dim), w2=1 + 0.2 * f(dim), mix=f(4, dim),
                A=-(0.05 + 4 * torch.rand(dim, generator=g)).double())


def inputs(batch, L, dim, seed=2):
    g = torch.Generator().manual_seed(seed)
    f = lambda *s: torch.randn(*s, generator=g).float().double()  # noqa: E731
    return dict(x=f(batch, L, dim), stream=f(batch, L, dim), h0=f(batch, dim)), \
        (torch.rand(batch, L, generator=g) < 0.02).to(torch.uint8)


@pytest.mark.parametrize("size", [(1, 1, 32), (2, 100, 96), (2, 700, 130)])
def test_a_block_and_its_gradients(ms, size):
    """float32: each stage is within the bound of its own test, the second norm divides
    by a root mean square of about 1; four stages' bounds together."""
    p, (i, reset) = weights(size[2]), inputs(*size)
    cpu = {k: v.clone().requires_grad_(True) for k, v in {**p, **i}.items()}
    gpu = {k: v.float().cuda().requires_grad_(True) for k, v in {**p, **i}.items()}
    ref = reference({k: cpu[k] for k in p}, cpu["x"], cpu["stream"], cpu["h0"], reset)
    got = block(ms, {k: gpu[k] for k in p}, gpu["x"], gpu["stream"], gpu["h0"], reset.cuda())
    g = torch.Generator().manual_seed(3)
    douts = [torch.randn(t.shape, generator=g).double() for t in ref]
    for name, a, b in zip(("out", "stream", "state"), got, ref):
        R.check(name, a, b.detach(), rel=4 * R.REL)
    da = torch.autograd.grad(got, list(gpu.values()), [d.float().cuda() for d in douts])
    db = torch.autograd.grad(ref, list(cpu.values()), douts)
    for name, a, b in zip(gpu, da, db):
        # a weight's gradient is a sum over batch * L terms that may cancel: relative to
        # the root of their number times a term's size, which the others' size gives
        scale = None if name in i else torch.full_like(b, (size[0] * size[1]) ** 0.5
                                                       * float(db[0].abs().max().clamp(max=10)))
        R.check("d" + name, a, b, scale, rel=4 * R.REL)


@pytest.mark.parametrize("dtype", [F32, torch.bfloat16])
def test_prompt_pieces_and_tokens(ms, dtype):
    """Whole, in pieces through the state, and token by token over pools with slots, norm
    and recurrence together; the stream in float32 is carried in place by the steps."""
    p = {k: v.float().cuda() for k, v in weights(160).items()}
    i, _ = inputs(3, 620, 160)
    x, stream = i["x"].to(dtype).cuda(), i["stream"].float().cuda()
    mix = p["mix"].to(dtype)

    def mixer(y, call):
        u, r, z, g = (y.unsqueeze(-2) * mix).unbind(-2)
        return call(u.contiguous(), r.contiguous(), g.contiguous(), z.contiguous())
    y, _ = ms.residual_norm_fwd(x, stream, p["w1"])
    whole, last = mixer(y, lambda u, r, g, z: ms.gated_recurrence_fwd(
        u, r, g, p["A"], z, return_last_state=True))
    outs, state = [], None
    for a, b in ((0, 300), (300, 557), (557, 600)):
        y, _ = ms.residual_norm_fwd(x[:, a:b], stream[:, a:b], p["w1"])
        o, state = mixer(y, lambda u, r, g, z: ms.gated_recurrence_fwd(
            u, r, g, p["A"], z, state, return_last_state=True))
        outs.append(o)
    pool = torch.zeros(7, 160, device="cuda")
    slots = torch.tensor([5, 0, 3], dtype=torch.int32, device="cuda")
    pool[slots.long()] = state
    for t in range(600, 620):
        s = stream[:, t].contiguous()
        y, kept = ms.residual_norm_fwd(x[:, t], s, p["w1"], residual_out=s)
        assert kept is s
        outs.append(mixer(y, lambda u, r, g, z: ms.gated_recurrence_update(
            pool, u, r, g, p["A"], z, slots=slots))[:, None])
    # the norm and the gates are of the same bits; the states differ by float32's order
    R.check("out", torch.cat(outs, 1), whole.double().cpu(),
            whole.double().cpu().abs() * (1 + 2 * R.HALF[dtype] / R.REL))
    R.check("state", pool[slots.long()], last.double().cpu())
    assert not pool[[1, 2, 4, 6]].any()


def test_eight_bits_stand_for_the_norm(ms):
    """The 8-bit output times its scale is the norm's within half a step, and a product of
    it is the products' sum."""
    x = torch.randn(64, 512, device="cuda").bfloat16()
    stream = torch.randn(64, 512, device="cuda")
    w = 1 + 0.1 * torch.randn(512, device="cuda")
    y, s = ms.residual_norm_fwd(x, stream, w)
    q, scale, s8 = ms.residual_norm_fp8(x, stream, w)
    assert torch.equal(s, s8)
    back = q.float() * scale[:, None]
    # half a step of e4m3, at least that of its smallest values, and half one of bfloat16
    assert ((back - y.float()).abs() <= (2.0 ** -4 + 2.0 ** -8) * 1.01 * y.float().abs()
            + 2.0 ** -10 * scale[:, None] * 1.01).all()
    m = torch.randn(512, 48, device="cuda")
    exact = back.double().cpu() @ m.double().cpu()
    mine = (q.double().cpu() @ m.double().cpu()) * scale.double().cpu()[:, None]
    assert ((exact - mine).abs() <= 1e-6 * back.double().cpu().abs() @ m.double().cpu().abs()).all()


def run_all(ms, s):
    """One training pass and one token step through every operator, into fixed tensors."""
    out, res = ms.residual_norm_fwd(s["x"], s["stream"], s["w"], out=s["y"], residual_out=s["res"])
    ms.residual_norm_fp8(s["x"], s["stream"], s["w"], out=s["q"], scale=s["scale"],
                         residual_out=s["res8"])
    ms.gated_recurrence_fwd(s["y"], s["r"], s["i"], s["A"], s["z"], s["h0"], reset=s["flags"],
                            return_last_state=True, out=s["h"], last_state=s["last"],
                            checkpoints=s["ck"], workspace=s["ws"])
    g = ms.gated_recurrence_bwd(s["y"], s["r"], s["i"], s["A"], s["z"], s["dout"], s["h0"],
                                dlast_state=s["last"], reset=s["flags"], checkpoints=s["ck"],
                                workspace=s["ws"])
    n = ms.residual_norm_bwd(res, s["w"], g["dx"], s["dres"], workspace=s["ws"])
    t = ms.gated_recurrence_update(s["pool"], s["y"][:, 0], s["r"][:, 0], s["i"][:, 0], s["A"],
                                   slots=s["slots"])
    return [s["y"], s["res"], s["q"].view(torch.uint8), s["scale"], s["h"], s["last"], s["ck"],
            *g.values(), n["dx"], n["dresidual"], n["dweight"], t, s["pool"]]


def graph_state(ms, L, dim, seed):
    torch.manual_seed(seed)
    b, bf = 2, torch.bfloat16
    r = lambda *s, dt=bf: torch.randn(*s, device="cuda").to(dt)  # noqa: E731
    e = lambda *s, dt=bf: torch.empty(*s, device="cuda", dtype=dt)  # noqa: E731
    s = dict(x=r(b, L, dim), stream=r(b, L, dim, dt=F32), w=1 + r(dim, dt=F32) / 5,
             r=r(b, L, dim), i=r(b, L, dim), z=r(b, L, dim), A=-torch.rand(dim, device="cuda") - .05,
             h0=r(b, dim, dt=F32), dout=r(b, L, dim), dres=r(b, L, dim, dt=F32),
             flags=(torch.rand(b, L, device="cuda") < 0.01).to(torch.uint8),
             y=e(b, L, dim), res=e(b, L, dim, dt=F32), res8=e(b, L, dim, dt=F32),
             q=e(b, L, dim, dt=torch.float8_e4m3fn), scale=e(b, L, dt=F32), h=e(b, L, dim),
             last=e(b, dim, dt=F32), ck=e(ms.gated_recurrence_checkpoint_shape(b, L, dim), dt=F32),
             pool=r(5, dim, dt=F32), slots=torch.tensor([3, 1], dtype=torch.int32, device="cuda"))
    n = max(ms.gated_recurrence_fwd_workspace_bytes(b, L, dim, bf),
            ms.gated_recurrence_bwd_workspace_bytes(b, L, dim, bf), 1 << 22)
    s["ws"] = torch.empty(n, dtype=torch.uint8, device="cuda")
    return s


@pytest.mark.parametrize("size", [(100, 96), (700, 130), (2500, 64)])
def test_captured_and_replayed(ms, size):
    """Two graphs that share a workspace, replayed in turn with eager work between; new
    inputs are copied into the captured tensors."""
    states = [graph_state(ms, *size, seed) for seed in (1, 2)]
    states[1]["ws"] = states[0]["ws"]
    graphs, outs = [], []
    for s in states:
        pool = s["pool"].clone()
        stream = torch.cuda.Stream()
        stream.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(stream):
            run_all(ms, s)
        torch.cuda.current_stream().wait_stream(stream)
        s["pool"].copy_(pool)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(run_all(ms, s))
        graphs.append(g)
    for turn in range(4):
        for s, g, out in zip(states, graphs, outs):
            torch.manual_seed(10 + turn)
            for k in ("x", "r", "i", "dout"):
                s[k].copy_(torch.randn(s[k].shape, device="cuda"))
            before = s["pool"].clone()
            g.replay()
            torch.cuda.synchronize()
            got = [t.clone() for t in out]
            eager = dict(s, **{k: torch.empty_like(s[k]) for k in ("y", "res", "res8", "q", "scale",
                                                                   "h", "last", "ck", "ws")},
                         pool=before)
            want = run_all(ms, eager)
            assert all(torch.equal(a, b) for a, b in zip(got, want)), (turn, size)


def test_two_streams_at_once(ms):
    """Calls on two streams, each with its own workspace, and on a stream that is not the
    inputs' own."""
    states = [graph_state(ms, 1500, 200, seed) for seed in (3, 4)]
    want = [[t.clone() for t in run_all(ms, dict(s, pool=s["pool"].clone()))] for s in states]
    streams = [torch.cuda.Stream() for _ in states]
    torch.cuda.synchronize()
    for _ in range(5):
        got = []
        for s, stream in zip(states, streams):
            with torch.cuda.stream(stream):
                got.append(run_all(ms, dict(s, pool=s["pool"].clone())))
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_example():
    import recurrent_block as ex
    far, losses = ex.main()
    assert far < 2 * 2.0 ** -8      # bfloat16 roundings between the stages
    assert all(v == v and abs(v) < 1e6 for v in losses)
    torch.manual_seed(1)
    blk = ex.RecurrentBlock(64, 96)
    x = torch.randn(2, 150, 64, device="cuda").bfloat16().requires_grad_(True)
    stream = torch.randn(2, 150, 64, device="cuda", requires_grad=True)
    reset = torch.zeros(2, 150, dtype=torch.uint8, device="cuda")
    reset[0, 70] = 1
    out, kept = blk(x, stream, reset)
    (out.float().square().sum() + kept.sum()).backward()
    for t in (x, stream, *blk.parameters()):
        assert t.grad is not None and torch.isfinite(t.grad).all() and t.grad.any()
    # what is before a flag gets nothing from behind it
    (g,) = torch.autograd.grad(blk(x, stream, reset)[0][0, 70:].float().sum(), x)
    assert not g[0, :70].any() and g[0, 70:].any()

"""The recurrent block's operators at sizes where a kernel's variant begins and where a
launch ends, and comparisons of two calls that are as narrow as their roundings allow."""
import pytest
import torch

import recurrent_reference as R

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
TYPES = {"f32": (torch.float32, torch.float32), "bf16": (BF, BF), "mixed": (BF, torch.float32)}
EPS = 1e-5


@pytest.fixture(scope="module")
def ms():
    import scan_selective_fwd_amd as m
    assert torch.cuda.is_available()
    return m


def two_calls(name, a, b):
    """Two results within check's bounds of one truth: each is off by R.REL of the norm, a
    single element by ten times that of the larger of it and the root mean square, and
    by half a step of its type."""
    half = R.HALF[a.dtype]
    assert a.dtype == b.dtype and a.shape == b.shape
    rms = float(b.double().square().mean().sqrt())
    assert rms > 0 and rms < float("inf")
    for p, q in zip(a.reshape(-1).split(1 << 26), b.reshape(-1).split(1 << 26)):
        p, q = p.double(), q.double()
        size, e = torch.maximum(p.abs(), q.abs()), (p - q).abs()
        bad = ~(e <= 2 * half * (1 + half) * size + 20 * R.REL * torch.clamp(size, min=rms))
        assert not bad.any(), (name, int(bad.sum()), float(e.max()))
        assert float(e.norm()) <= (2 * half * (1 + half) + 2 * R.REL) * max(
            float(size.norm()), rms * p.numel() ** 0.5), name


@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("dim", [1544, 2048, 3501, 6136, 6144])
def test_norm_widths_of_every_variant(ms, dim, types):
    """The widths that other tests' lists step over: the last of those that a wave takes in
    groups of eight, those of four and of six groups of four a thread."""
    t = TYPES[types]
    i = R.norm_inputs(31, *t, 9, dim)
    kind = dict(x=t[0], dout=t[0], residual=t[1], dres=t[1], weight=torch.float32)
    g = {k: v.to(kind[k]).cuda() for k, v in i.items()}
    out, res = ms.residual_norm_fwd(g["x"], g["residual"], g["weight"], eps=EPS)
    o8, scale, res8 = ms.residual_norm_fp8(g["x"], g["residual"], g["weight"], eps=EPS)
    assert torch.equal(res, res8)
    R.check("res", res, i["x"] + i["residual"], rel=2.0 ** -24)
    y = R.norm_fwd(res.double().cpu(), None, i["weight"], EPS, t[1])[0]
    R.check("out", out, y)
    R.check("scale", scale, y.abs().amax(-1) / 448)
    R.check("out8", o8, y / scale.double().cpu().unsqueeze(-1))
    got = ms.residual_norm_bwd(g["residual"], g["weight"], g["dout"], g["dres"], eps=EPS)
    d, dw, dw_abs = R.norm_bwd(i["residual"], i["weight"], i["dout"], i["dres"], EPS)
    terms = R.norm_terms(i["residual"], i["weight"], i["dout"], i["dres"], EPS)
    R.check("dx", got["dx"], d, terms)
    R.check("dresidual", got["dresidual"], d, terms)
    R.check("dweight", got["dweight"], dw, dw_abs)


@pytest.mark.parametrize("dtype", [torch.float32, BF])
def test_prompt_pieces_and_tokens(ms, dtype):
    """A prompt whole against its pieces and single tokens, over a pool by slots."""
    i = R.rec_inputs(32, dtype, 3, 620, 160, h0=False)
    x, r, g, z = (i[k].to(dtype).cuda() for k in ("x", "r", "i", "z"))
    A = i["A"].float().cuda()
    whole, last = ms.gated_recurrence_fwd(x, r, g, A, z, return_last_state=True)
    outs, state = [], None
    for a, b in ((0, 300), (300, 557), (557, 600)):
        o, state = ms.gated_recurrence_fwd(x[:, a:b], r[:, a:b], g[:, a:b], A, z[:, a:b], state,
                                           return_last_state=True)
        outs.append(o)
    pool = torch.zeros(7, 160, device="cuda")
    slots = torch.tensor([5, 0, 3], dtype=torch.int32, device="cuda")
    pool[slots.long()] = state
    for t in range(600, 620):
        outs.append(ms.gated_recurrence_update(pool, x[:, t], r[:, t], g[:, t], A, z[:, t],
                                               slots=slots)[:, None])
    two_calls("out", torch.cat(outs, 1), whole)
    two_calls("state", pool[slots.long()], last)


def normal(n, dim, seed):
    """(n, dim) bfloat16, drawn anew row by row."""
    g = torch.Generator("cuda").manual_seed(seed)
    out = torch.empty(n, dim, dtype=BF, device="cuda")
    for at in range(0, n, 1 << 16):
        part = out[at:at + (1 << 16)]
        part.copy_(torch.randn(part.shape, device="cuda", generator=g))
    return out


def test_one_long_sequence_in_two_parts(ms):
    """1.45M steps of 1536 channels: outputs, states and all gradients against two calls, the
    state carried from the first to the second and its gradient back."""
    L, dim, cut = 1_450_001, 1536, 1_000_003
    assert L * dim > 2 ** 31 and cut * dim < 2 ** 31
    x, r, i, dout = (normal(L, dim, 50 + k).unsqueeze(0) for k in range(4))
    A = -(0.05 + 4 * torch.rand(dim, device="cuda", generator=torch.Generator("cuda").manual_seed(9)))
    a, b = (lambda t: t[:, :cut].contiguous()), (lambda t: t[:, cut:].contiguous())
    out, last = ms.gated_recurrence_fwd(x, r, i, A, return_last_state=True)
    o1, state = ms.gated_recurrence_fwd(a(x), a(r), a(i), A, return_last_state=True)
    two_calls("out", out[:, :cut], o1)
    o2, l2 = ms.gated_recurrence_fwd(b(x), b(r), b(i), A, None, state, return_last_state=True)
    two_calls("out", out[:, cut:], o2)
    two_calls("last", last, l2)
    del out, o1, o2
    g = ms.gated_recurrence_bwd(x, r, i, A, None, dout)
    g2 = ms.gated_recurrence_bwd(b(x), b(r), b(i), A, None, b(dout), state)
    g1 = ms.gated_recurrence_bwd(a(x), a(r), a(i), A, None, a(dout), dlast_state=g2["dh0"])
    for k in ("dx", "dr", "di"):
        two_calls(k, g[k][:, :cut], g1[k])
        two_calls(k, g[k][:, cut:], g2[k])
    # dA's terms are those of dr over A (1 - s(r)); the two ways differ in them by float32's
    # order, with signs that are each other's own beyond the some 40 steps that a state
    # lives: eight times the root of their squares' sum
    squares = torch.zeros(dim, device="cuda", dtype=torch.float64)
    for at in range(0, L, 1 << 17):
        s = slice(at, at + (1 << 17))
        squares += (g["dr"][0, s].float() / (A * torch.sigmoid(-r[0, s].float()))).double().square().sum(0)
    far = (g["dA"].double() - (g1["dA"].double() + g2["dA"].double())).abs()
    assert (far <= 8 * 40 ** 0.5 * R.REL * squares.sqrt()).all(), float((far / squares.sqrt()).max())


def test_dweight_of_many_rows(ms):
    """1.45M rows of 1536 against the sum in 64 bits.  A block adds some 2800 rows in float32
    and the blocks' sums are added after: each addition is off by half a step of a partial
    sum, the terms by some 2^-22 of themselves, with signs of their own: eight times the
    root of the squares' sum, with partial sums of the terms' random walk."""
    n, dim = 1_450_000, 1536
    assert n * dim > 2 ** 31
    res, dout = normal(n, dim, 61), normal(n, dim, 62)
    w = 1 + 0.1 * torch.randn(dim, device="cuda")
    got = ms.residual_norm_bwd(res, w, dout, eps=EPS)["dweight"].double()
    want, squares = (torch.zeros(dim, device="cuda", dtype=torch.float64) for _ in range(2))
    for at in range(0, n, 1 << 16):
        x, dy = res[at:at + (1 << 16)].double(), dout[at:at + (1 << 16)].double()
        term = dy * x / torch.sqrt(x.square().mean(-1, keepdim=True) + EPS)
        want += term.sum(0)
        squares += term.square().sum(0)
    blocks = 512
    steps = n / blocks
    walk = n * (squares / n) * steps / 2            # the partial sums' squares, added up
    tops = 32 * squares + 16 * squares              # those of the sums over blocks
    allowed = 8 * (2.0 ** -24 * (walk + tops).sqrt() + 2.0 ** -22 * squares.sqrt())
    assert ((got - want).abs() <= allowed).all(), float(((got - want).abs() / allowed).max())

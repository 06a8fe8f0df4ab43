"""The recurrent block's operators where offsets pass 2^31 elements: one long sequence,
many rows, a large pool; and many short sequences.  What is compared lies behind the
border, against the same call on a part of the inputs that does not reach it."""
import pytest
import torch

import recurrent_reference as R

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module")
def ms():
    import scan_selective_fwd_amd as m
    assert torch.cuda.is_available()
    return m


def rows(n, dim, seed):
    """(n, dim) bfloat16, a block of random rows over and over with a row number mixed in."""
    g = torch.Generator("cuda").manual_seed(seed)
    base = torch.randn(8192, dim, device="cuda", generator=g).to(BF)
    out = base.repeat(-(-n // 8192), 1)[:n]
    out[:, 0] = torch.randn(n, device="cuda", generator=g).to(BF)
    return out


def test_one_long_sequence(ms):
    """1.45M steps of 1536 channels: the outputs of the last 5000 against those of a call
    that begins there, from the state that the first part leaves; the gradients of the
    last steps the same way."""
    L, dim, tail = 1_450_001, 1536, 5000
    assert L * dim > 2 ** 31
    x, r, i = (rows(L, dim, k).unsqueeze(0) for k in range(3))
    A = -(0.05 + 4 * torch.rand(dim, device="cuda", generator=torch.Generator("cuda").manual_seed(9)))
    ck = torch.empty(ms.gated_recurrence_checkpoint_shape(1, L, dim), device="cuda")
    out, last = ms.gated_recurrence_fwd(x, r, i, A, return_last_state=True, checkpoints=ck)
    cut = L - tail
    part = lambda t: t[:, cut:]  # noqa: E731
    _, state = ms.gated_recurrence_fwd(x[:, :cut], r[:, :cut], i[:, :cut], A,
                                       return_last_state=True)
    o2, l2 = ms.gated_recurrence_fwd(part(x), part(r), part(i), A, None, state,
                                     return_last_state=True)
    # two roundings of values that agree to float32's order
    R.check("out", part(out), o2.double().cpu(), o2.double().cpu().abs() * (1 + 2 ** -7 / R.REL))
    R.check("last", last, l2.double().cpu())
    del state
    dout = rows(L, dim, 4).unsqueeze(0)
    g = ms.gated_recurrence_bwd(x, r, i, A, None, dout, checkpoints=ck)
    _, state = ms.gated_recurrence_fwd(x[:, :cut], r[:, :cut], i[:, :cut], A,
                                       return_last_state=True)
    g2 = ms.gated_recurrence_bwd(part(x), part(r), part(i), A, None, part(dout).contiguous(), state)
    for k in ("dx", "dr", "di"):
        want = g2[k].double().cpu()
        R.check(k, part(g[k]), want, want.abs() * (1 + 2 ** -7 / R.REL))
    assert torch.isfinite(g["dA"]).all()


def test_many_rows(ms):
    """1.45M rows of 1536 through the norm: those behind 2^31 elements have the bits that
    they have alone."""
    n, dim, tail = 1_450_000, 1536, 3000
    x, res = rows(n, dim, 5), rows(n, dim, 6)
    w = 1 + 0.1 * torch.randn(dim, device="cuda")
    for call in (ms.residual_norm_fwd, ms.residual_norm_fp8):
        a, b = call(x, res, w), call(x[-tail:], res[-tail:], w)
        for p, q in zip(a, b):
            assert torch.equal(p[-tail:].float(), q.float())
        del a, b
    a = ms.residual_norm_bwd(res, w, x)
    b = ms.residual_norm_bwd(res[-tail:], w, x[-tail:])
    assert torch.equal(a["dx"][-tail:], b["dx"]) and torch.isfinite(a["dweight"]).all()


def test_a_large_pool(ms):
    pool = torch.zeros(1_450_000, 1536, device="cuda")
    slots = torch.tensor([1_449_999, 3, 1_400_000], dtype=torch.int32, device="cuda")
    pool[slots.long()] = torch.randn(3, 1536, device="cuda")
    small = pool[slots.long()].clone()
    x, r, i = (torch.randn(3, 1536, device="cuda").to(BF) for _ in range(3))
    A = -torch.rand(1536, device="cuda")
    got = ms.gated_recurrence_update(pool, x, r, i, A, slots=slots)
    want = ms.gated_recurrence_update(small, x, r, i, A)
    assert torch.equal(got, want) and torch.equal(pool[slots.long()], small)


@pytest.mark.parametrize("batch,L,dim", [(70_000, 1, 40), (70_000, 3, 3), (300, 300, 64)])
def test_many_sequences(ms, batch, L, dim):
    i = R.rec_inputs(31, torch.float32, 50, L, dim)
    g = {k: v.float().cuda() for k, v in i.items() if v is not None}
    n = batch // 50
    many = {k: v if k == "A" else v.repeat(n, *[1] * (v.dim() - 1)) for k, v in g.items()}
    call = lambda s: ms.gated_recurrence_fwd(s["x"], s["r"], s["i"], s["A"], s["z"], s["h0"],  # noqa: E731
                                             return_last_state=True)
    for a, b in zip(call(many), call(g)):
        assert torch.equal(a, b.repeat(n, *[1] * (b.dim() - 1)))
    back = lambda s: ms.gated_recurrence_bwd(s["x"], s["r"], s["i"], s["A"], s["z"], s["dout"],  # noqa: E731
                                             s["h0"], dlast_state=s["dlast"])
    a, b = back(many), back(g)
    for k in b:
        if k != "dA":
            assert torch.equal(a[k], b[k].repeat(n, *[1] * (b[k].dim() - 1))), k
    _, terms = R.rec_bwd(i["x"], i["r"], i["i"], i["A"], i["z"], i["dout"], i["h0"], i["dlast"])
    R.check("dA", a["dA"], n * b["dA"].double().cpu(), n * terms["dA"])

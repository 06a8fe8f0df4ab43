"""The residual norm on the GPU against the 64-bit reference: widths around every
variant's border, the residual in both types, views, 8 bits with scales, values
that are not finite, and what is refused."""
import pytest
import torch

import recurrent_reference as R

pytestmark = pytest.mark.gpu

TYPES = {"f32": (torch.float32, torch.float32), "bf16": (torch.bfloat16, torch.bfloat16),
         "mixed": (torch.bfloat16, torch.float32)}
# (rows, dim): one value, odd widths, around the wave's and the block's reach
SIZES = [(1, 1), (3, 2), (2, 7), (5, 64), (1, 257), (4, 512), (3, 520), (2, 1003), (7, 1024),
         (130, 1536), (1, 2047), (3, 2056), (2, 4096), (3, 5120), (2, 8192), (1, 8200), (2, 16384),
         (1, 33000), (700, 96)]
EPS = 1e-5


@pytest.fixture(scope="module")
def ms():
    import scan_selective_fwd_amd as m
    assert torch.cuda.is_available()
    return m


def dev(i, types):
    kind = dict(x=types[0], dout=types[0], residual=types[1], dres=types[1], weight=torch.float32)
    return {k: None if v is None else v.to(kind[k]).cuda() for k, v in i.items()}


def check_res(got, total, res_dtype):
    R.check("res", got, total, rel=2.0 ** -24)      # one rounding of an exact sum, twice


@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("size", SIZES)
def test_forward(ms, size, types):
    t = TYPES[types]
    i = R.norm_inputs(1, *t, *size, weight=size[0] != 3)
    g = dev(i, t)
    out, res = ms.residual_norm_fwd(g["x"], g["residual"], g["weight"], eps=EPS)
    assert out.dtype == t[0] and res.dtype == t[1]
    y, _, total = R.norm_fwd(i["x"], i["residual"], i["weight"], EPS, t[1])
    check_res(res, total, t[1])
    y = R.norm_fwd(res.double().cpu(), None, i["weight"], EPS, t[1])[0]   # of what is kept
    R.check("out", out, y)
    # alone: the norm of x, and x goes on as the stream
    out, res = ms.residual_norm_fwd(g["x"], None, g["weight"], eps=EPS)
    assert res is g["x"]
    R.check("out", out, R.norm_fwd(i["x"], None, i["weight"], EPS, t[1])[0])


def check_fp8(out, scale, y):
    """out against y over its own scale: half a step of e4m3; the scale in float32."""
    amax = y.abs().amax(-1)
    R.check("scale", scale, torch.clamp_min(amax, 2.0 ** -100) / 448)
    assert out.dtype == torch.float8_e4m3fn and float(out.float().abs().max()) <= 448
    R.check("out8", out, y / scale.double().cpu().unsqueeze(-1))


@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("size", SIZES)
def test_eight_bits(ms, size, types):
    t = TYPES[types]
    i = R.norm_inputs(2, *t, *size, weight=size[0] != 3)
    g = dev(i, t)
    out, scale, res = ms.residual_norm_fp8(g["x"], g["residual"], g["weight"], eps=EPS)
    assert scale.shape == (size[0],) and scale.dtype == torch.float32 and res.dtype == t[1]
    check_res(res, i["x"] + i["residual"], t[1])
    check_fp8(out, scale, R.norm_fwd(res.double().cpu(), None, i["weight"], EPS, t[1])[0])
    top = out.float().abs().amax(-1)
    assert (top == 448).all()       # each row reaches the type's largest value
    out, scale, res = ms.residual_norm_fp8(g["x"], None, g["weight"], eps=EPS)
    assert res is g["x"]
    check_fp8(out, scale, R.norm_fwd(i["x"], None, i["weight"], EPS, t[1])[0])


@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("size", SIZES + [(1500, 33), (513, 2048)])
def test_backward(ms, size, types):
    t = TYPES[types]
    i = R.norm_inputs(3, *t, *size, weight=size[0] != 3)
    g = dev(i, t)
    res = g["residual"]
    for dres in (None, "dres"):
        got = ms.residual_norm_bwd(res, g["weight"], g["dout"], dres and g[dres], eps=EPS)
        d, dw, dw_abs = R.norm_bwd(i["residual"], i["weight"], i["dout"], dres and i[dres], EPS)
        assert got["dx"].dtype == t[0] and got["dresidual"].dtype == t[1]
        assert (got["dresidual"] is got["dx"]) == (t[0] == t[1])
        terms = R.norm_terms(i["residual"], i["weight"], i["dout"], dres and i[dres], EPS)
        R.check("dx", got["dx"], d, terms)
        R.check("dresidual", got["dresidual"], d, terms)
        assert ("dweight" in got) == (g["weight"] is not None)
        if g["weight"] is not None:
            R.check("dweight", got["dweight"], dw, dw_abs)


@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("dim,off", [(64, 0), (64, 1), (1024, 8), (1024, 3), (33, 5), (2056, 8)])
def test_views_of_wider_rows(ms, dim, off, types):
    t = TYPES[types]
    i = R.norm_inputs(4, *t, 2, 9, dim)
    g = dev(i, t)
    v = dict(g)
    for k in ("x", "residual"):
        wide = torch.full((2, 9, dim + 16 + off), 7.0, dtype=g[k].dtype, device="cuda")
        wide[..., off:off + dim] = g[k]
        v[k] = wide[..., off:off + dim]
    # against the reference: the dense call's results are rounded as these are, so that the
    # two may differ by two half steps
    out, res = ms.residual_norm_fwd(v["x"], v["residual"], g["weight"])
    assert torch.equal(res, ms.residual_norm_fwd(g["x"], g["residual"], g["weight"])[1])
    y = R.norm_fwd(res.double().cpu(), None, i["weight"], EPS, t[1])[0]
    R.check("out", out, y)
    o8, scale, again = ms.residual_norm_fp8(v["x"], v["residual"], g["weight"])
    assert scale.shape == (2, 9) and torch.equal(again, res)
    check_fp8(o8, scale, y)
    got = ms.residual_norm_bwd(v["residual"], g["weight"], g["dout"], g["dres"])
    d, dw, dw_abs = R.norm_bwd(i["residual"], i["weight"], i["dout"], i["dres"], EPS)
    terms = R.norm_terms(i["residual"], i["weight"], i["dout"], i["dres"], EPS)
    R.check("dx", got["dx"], d, terms)
    R.check("dresidual", got["dresidual"], d, terms)
    R.check("dweight", got["dweight"], dw, dw_abs)
    # parts of batch rows, together with dense ones, and one row for every row
    dense = lambda t: t.contiguous()  # noqa: E731
    for a, b in ((g["x"][:, 2:7], dense(g["residual"][:, 2:7])),
                 (dense(g["x"][:, ::2]), g["residual"][:, ::2]),
                 (g["x"][:, 3:5], g["residual"][:, 1:3]),
                 (g["x"][:1, :1].expand(2, 9, dim), g["residual"])):
        for call in (ms.residual_norm_fwd, ms.residual_norm_fp8):
            for p, q in zip(call(a, b, g["weight"]), call(dense(a), dense(b), g["weight"])):
                assert torch.equal(p.float(), q.float())
    part, dpart = g["residual"][:, 2:7], dense(g["dout"][:, 2:7])
    p, q = (ms.residual_norm_bwd(r, g["weight"], dpart) for r in (part, dense(part)))
    assert all(torch.equal(p[k], q[k]) for k in p)
    for bad in (g["x"].unsqueeze(0).expand(3, 2, 9, dim).transpose(0, 2), g["x"].transpose(1, 2)):
        with pytest.raises(ValueError):     # no two strides say this
            ms.residual_norm_fwd(bad)
    row = g["x"][0, :1].expand(9, dim)
    a, _ = ms.residual_norm_fwd(row, g["residual"][0], g["weight"])
    b, _ = ms.residual_norm_fwd(row.contiguous(), g["residual"][0], g["weight"])
    assert torch.equal(a, b)


@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("dim", [33, 1536, 12288])
def test_the_stream_in_place(ms, dim, types):
    t = TYPES[types]
    g = dev(R.norm_inputs(5, *t, 6, dim), t)
    out, res = ms.residual_norm_fwd(g["x"], g["residual"], g["weight"])
    stream = g["residual"].clone()
    again, kept = ms.residual_norm_fwd(g["x"], stream, g["weight"], residual_out=stream)
    assert kept is stream and torch.equal(stream, res) and torch.equal(again, out)
    o8, s8, res = ms.residual_norm_fp8(g["x"], g["residual"], g["weight"])
    stream = g["residual"].clone()
    again, s, _ = ms.residual_norm_fp8(g["x"], stream, g["weight"], residual_out=stream)
    assert torch.equal(stream, res) and torch.equal(again.view(torch.uint8), o8.view(torch.uint8))
    assert torch.equal(s, s8)


@pytest.mark.parametrize("dim", [5, 256, 2048, 9000])
def test_rows_of_zeros_and_of_extremes(ms, dim):
    x = torch.zeros(5, dim, device="cuda")
    x[1] = 1e-20                    # squares vanish beside eps
    x[2] = 1e18                     # their squares' sum is near the type's end
    x[3, 0] = -3e38
    x[3] *= 1e-19
    x[4, -1] = 2.5
    out, _ = ms.residual_norm_fwd(x)
    ref, _, _ = R.norm_fwd(x.double().cpu(), None, None, EPS, torch.float32)
    for k in range(5):
        R.check(f"row {k}", out[k], ref[k])
    o8, scale, _ = ms.residual_norm_fp8(x)
    assert not o8[0].float().any()
    assert abs(float(scale[0]) * 448 * 2.0 ** 100 - 1) <= 2.0 ** -24     # one division's rounding
    for k in range(1, 5):
        R.check(f"scale {k}", scale[k], ref[k].abs().max() / 448)
        R.check(f"row {k}", o8[k], ref[k] / float(scale[k]))
    out, _ = ms.residual_norm_fwd(torch.zeros(2, dim, device="cuda"), eps=0.0)
    assert torch.isnan(out).all()           # 0 / 0, as the formula says
    dout = torch.randn(5, dim, device="cuda")
    got = ms.residual_norm_bwd(x, None, dout)["dx"]
    d, _, _ = R.norm_bwd(x.double().cpu(), None, dout.double().cpu(), None, EPS)
    for k in (0, 1, 4):
        R.check(f"dx {k}", got[k], d[k])


@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("dim", [40, 1536, 2051])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_non_finite_values_stay_in_their_row(ms, value, dim, types):
    t = TYPES[types]
    g = dev(R.norm_inputs(6, *t, 9, dim), t)
    bad = g["x"].clone()
    bad[4, 3] = value
    rest = [k for k in range(9) if k != 4]
    for call in (ms.residual_norm_fwd, ms.residual_norm_fp8):
        a, b = call(bad, g["residual"], g["weight"]), call(g["x"], g["residual"], g["weight"])
        for p, q in zip(a, b):
            p, q = p.float(), q.float()
            assert torch.equal(p[rest], q[rest])
        assert torch.isnan(a[0][4, 3].float())        # inf / inf
        if value != value:
            assert torch.isnan(a[0][4].float()).all()
        else:
            assert not a[0][4].float().nan_to_num().any()
    res = g["residual"].clone()
    res[4, 3] = value
    a = ms.residual_norm_bwd(res, g["weight"], g["dout"], g["dres"])
    b = ms.residual_norm_bwd(g["residual"], g["weight"], g["dout"], g["dres"])
    assert torch.equal(a["dx"][rest], b["dx"][rest]) and torch.isnan(a["dx"][4, 3])


def test_gradients_through_autograd(ms):
    for t in TYPES.values():
        i = R.norm_inputs(7, *t, 3, 5, 96)
        g = dev(i, t)
        leaf = {k: g[k].clone().requires_grad_(True) for k in ("x", "residual", "weight")}
        out, res = ms.residual_norm(leaf["x"], leaf["residual"], leaf["weight"])
        got = torch.autograd.grad([out, res], list(leaf.values()), [g["dout"], g["dres"]],
                                  retain_graph=True)
        d, dw, dw_abs = R.norm_bwd(res.detach().double().cpu(), i["weight"], i["dout"], i["dres"],
                                   EPS)
        R.check("dx", got[0], d)
        R.check("dresidual", got[1], d)
        R.check("dweight", got[2], dw, dw_abs)
        # through one of the two outputs
        got = torch.autograd.grad(out, list(leaf.values()), g["dout"], retain_graph=True)
        d, _, _ = R.norm_bwd(res.detach().double().cpu(), i["weight"], i["dout"], None, EPS)
        R.check("dx", got[0], d)
        got = torch.autograd.grad(res, list(leaf.values()), g["dres"])
        R.check("dx", got[0], i["dres"])
        R.check("dresidual", got[1], i["dres"])
        assert not got[2].any()
        # x as both: its gradient is twice that at the sum
        x = g["x"].to(t[1]).requires_grad_(True)
        out, res = ms.residual_norm(x, x, leaf["weight"])
        out.backward(g["dout"].to(t[1]))
        d, _, _ = R.norm_bwd(res.detach().double().cpu(), i["weight"], i["dout"], None, EPS)
        R.check("dx", x.grad, 2 * d, d.abs() * 4, rel=2 * R.REL)
        # alone, and the stream goes on from x
        x = g["x"].clone().requires_grad_(True)
        out, res = ms.residual_norm(x, None, g["weight"])
        (dx,) = torch.autograd.grad(out, x, g["dout"], create_graph=True)
        d, _, _ = R.norm_bwd(i["x"], i["weight"], i["dout"], None, EPS)
        R.check("dx", dx, d)
        with pytest.raises(RuntimeError):
            torch.autograd.grad(dx.float().square().sum() + x.float().sum(), x)


def test_gradients_against_differences(ms):
    """Along random directions, central differences of the float32 forward: the loss's
    rounding, 1e-6 of its terms' root sum of squares over a step of 2 2^-6."""
    t = TYPES["f32"]
    g = dev(R.norm_inputs(8, *t, 6, 200), t)
    h = 2.0 ** -6

    def loss(x, w):
        out, res = ms.residual_norm_fwd(x, g["residual"], w)
        return float((out.double() * g["dout"].double()).sum()
                     + (res.double() * g["dres"].double()).sum())
    _, res = ms.residual_norm_fwd(g["x"], g["residual"], g["weight"])
    got = ms.residual_norm_bwd(res, g["weight"], g["dout"], g["dres"])
    u, v = torch.randn(6, 200, device="cuda"), torch.randn(200, device="cuda")
    for d, have in (((u, 0 * v), (got["dx"] * u).double()),
                    ((0 * u, v), (got["dweight"] * v).double())):
        want = (loss(g["x"] + h * d[0], g["weight"] + h * d[1])
                - loss(g["x"] - h * d[0], g["weight"] - h * d[1])) / (2 * h)
        assert abs(want - float(have.sum())) < 2e-3 * float(have.norm())


@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("dim", [33, 1536, 9000])
def test_outputs_are_overwritten_and_equal_calls_give_equal_bits(ms, dim, types):
    t = TYPES[types]
    g = dev(R.norm_inputs(9, *t, 700, dim), t)

    def padded(n, dtype):
        flat = torch.full((n + 128,), 77.0, device="cuda").to(dtype)
        return flat, flat[64:64 + n]
    out_, out = padded(700 * dim, t[0])
    res_, res = padded(700 * dim, t[1])
    a = ms.residual_norm_fwd(g["x"], g["residual"], g["weight"], out=out.view(700, dim),
                             residual_out=res.view(700, dim))
    b = ms.residual_norm_fwd(g["x"], g["residual"], g["weight"])
    assert all(torch.equal(p, q) for p, q in zip(a, b))
    o8_, o8 = padded(700 * dim, torch.float8_e4m3fn)
    s_, s = padded(700, torch.float32)
    a = ms.residual_norm_fp8(g["x"], g["residual"], g["weight"], out=o8.view(700, dim), scale=s)
    b = ms.residual_norm_fp8(g["x"], g["residual"], g["weight"])
    assert all(torch.equal(p.float(), q.float()) for p, q in zip(a, b))
    for flat in (out_, res_, o8_, s_):
        edge = flat[:64].float()
        assert (edge == edge[0]).all() and (flat[-64:].float() == edge[0]).all()
    a = ms.residual_norm_bwd(res.view(700, dim), g["weight"], g["dout"], g["dres"])
    ws = torch.full((64 << 20,), 0xA5, dtype=torch.uint8, device="cuda")
    for _ in range(3):
        b = ms.residual_norm_bwd(res.view(700, dim), g["weight"], g["dout"], g["dres"],
                                 workspace=ws)
        assert all(torch.equal(a[k], b[k]) for k in a)


def test_refusals(ms):
    t = TYPES["bf16"]
    g = dev(R.norm_inputs(10, *t, 4, 16), t)
    f = ms.residual_norm_fwd
    for bad in ((g["x"].cpu(), g["residual"], None), (g["x"], g["residual"][:3], None),
                (g["x"], g["residual"], g["weight"][:15]), (g["x"][:, ::2], g["residual"][:, :8],
                                                            None)):
        with pytest.raises(ValueError):
            f(*bad)
    for bad in ((g["x"].half(), g["residual"], None), (g["x"], g["residual"].half(), None),
                (g["x"].float(), g["residual"], None),
                (g["x"], g["residual"], g["weight"].bfloat16())):
        with pytest.raises(TypeError):
            f(*bad)
    with pytest.raises(ValueError):
        f(g["x"], None, None, residual_out=torch.empty_like(g["x"]))
    with pytest.raises(ms.MambaScanError):
        f(g["x"], g["residual"], eps=-1.0)
    with pytest.raises(ms.MambaScanError):
        f(g["x"][:0], g["residual"][:0])
    with pytest.raises(ms.MambaScanError):      # out over an input
        f(g["x"], g["residual"], out=g["x"])
    with pytest.raises(ms.MambaScanError):      # a part of the stream
        both = torch.zeros(80, dtype=torch.bfloat16, device="cuda")
        f(g["x"], both[:64].view(4, 16), residual_out=both[16:].view(4, 16))
    with pytest.raises(TypeError):
        ms.residual_norm_fp8(g["x"], g["residual"], out=torch.empty_like(g["x"]))
    with pytest.raises(ValueError):
        ms.residual_norm_bwd(g["residual"], g["weight"], g["dout"][:3])
    with pytest.raises(TypeError):
        ms.residual_norm_bwd(g["residual"].double(), g["weight"], g["dout"])
    with pytest.raises(ValueError):
        ms.residual_norm_bwd(g["residual"], g["weight"], g["dout"], workspace=torch.empty(64))


@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("dim", [33, 1024])
def test_a_batch_broadcast_from_one(ms, dim, types):
    """Every batch row the same rows, in memory once: as x, as the residual, as both, and as
    the backward's res."""
    t = TYPES[types]
    g = dev(R.norm_inputs(11, *t, 3, 7, dim), t)
    one, two = g["x"][:1].expand(3, 7, dim), g["residual"][:1].expand(3, 7, dim)
    for x, res in ((one, None), (one, g["residual"]), (g["x"], two), (one, two)):
        full = None if res is None else res.contiguous()
        for call in (ms.residual_norm_fwd, ms.residual_norm_fp8):
            for p, q in zip(call(x, res, g["weight"]), call(x.contiguous(), full, g["weight"])):
                assert torch.equal(p.float(), q.float())
    p, q = (ms.residual_norm_bwd(r, g["weight"], g["dout"], g["dres"])
            for r in (two, two.contiguous()))
    assert all(torch.equal(p[k], q[k]) for k in p)


@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("dim", [1, 3, 4, 5, 7, 8, 9, 13, 63, 64, 65, 128, 129, 132, 255, 511,
                                 513, 770, 1025, 1537, 2046, 2049, 4099, 6001, 8191, 8194,
                                 16381, 16387])
def test_rows_that_start_anywhere(ms, dim, types):
    """Widths around whole groups: a row's last group ends with it, and nothing beside the
    rows is written."""
    t = TYPES[types]
    i = R.norm_inputs(12, *t, 5, dim)
    g = dev(i, t)

    def inside(like, dtype=None):     # a tensor between values that have to stay
        n, dtype = like.numel(), dtype or like.dtype
        wide = torch.full((n + 64,), 3.0, device="cuda").to(dtype)
        return wide, wide[32:32 + n].view(like.shape)

    for shift in (0, 1):              # with rows of whole groups too
        w, x = inside(torch.empty(5 * dim + shift, dtype=t[0], device="cuda"))
        x = x[shift:].view(5, dim).copy_(g["x"])
        (wo, out), (wr, kept), (w8, o8) = (inside(g["x"]), inside(g["residual"]),
                                           inside(g["x"], torch.float8_e4m3fn))
        kept.copy_(g["residual"])
        _, res = ms.residual_norm_fwd(x, kept, g["weight"], out=out, residual_out=kept)
        check_res(res, i["x"] + i["residual"], t[1])
        y = R.norm_fwd(res.double().cpu(), None, i["weight"], EPS, t[1])[0]
        R.check("out", out, y)
        kept.copy_(g["residual"])
        _, scale, again = ms.residual_norm_fp8(x, kept, g["weight"], out=o8, residual_out=kept)
        assert torch.equal(again, res)
        check_fp8(o8, scale, y)
        for wide in (wo, wr, w8):
            ends = torch.cat([wide[:32].float(), wide[-32:].float()])
            assert bool((ends == 3.0).all())
    got = ms.residual_norm_bwd(g["residual"], g["weight"], g["dout"], g["dres"])
    d, dw, dw_abs = R.norm_bwd(i["residual"], i["weight"], i["dout"], i["dres"], EPS)
    terms = R.norm_terms(i["residual"], i["weight"], i["dout"], i["dres"], EPS)
    R.check("dx", got["dx"], d, terms)
    R.check("dresidual", got["dresidual"], d, terms)
    R.check("dweight", got["dweight"], dw, dw_abs)

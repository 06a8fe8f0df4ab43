"""The residual norm where its statistics come near the ends of float32 or vanish: no eps,
and rows whose squares' or products' sums pass the type's range; and what its 8 bits
are rounded from."""
import pytest
import torch

import recurrent_reference as R

pytestmark = pytest.mark.gpu

TYPES = {"f32": (torch.float32, torch.float32), "bf16": (torch.bfloat16, torch.bfloat16),
         "mixed": (torch.bfloat16, torch.float32)}


@pytest.fixture(scope="module")
def ms():
    import scan_selective_fwd_amd as m
    assert torch.cuda.is_available()
    return m


def check_bwd(got, i, eps):
    d, dw, dw_abs = R.norm_bwd(i["residual"], i["weight"], i["dout"], i["dres"], eps)
    terms = R.norm_terms(i["residual"], i["weight"], i["dout"], i["dres"], eps)
    for k in ("dx", "dresidual"):
        R.check(k, got[k], d, terms)
    R.check("dweight", got["dweight"], dw, dw_abs)


@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("dim", [33, 256, 768, 1500])
@pytest.mark.parametrize("rows", [1, 5, 2050])
def test_backward_without_eps(ms, rows, dim, types):
    """No row is zero, so that every gradient is finite, also where the last pass over the
    rows leaves some of a block's teams without one."""
    t = TYPES[types]
    i = R.norm_inputs(21, *t, rows, dim)
    kind = dict(x=t[0], dout=t[0], residual=t[1], dres=t[1], weight=torch.float32)
    g = {k: v.to(kind[k]).cuda() for k, v in i.items()}
    check_bwd(ms.residual_norm_bwd(g["residual"], g["weight"], g["dout"], g["dres"], eps=0.0), i, 0.0)


def extreme_rows(dim, dtype):
    """Rows whose squares' sum leaves float32, or vanishes."""
    top = torch.finfo(torch.bfloat16).max            # what masks are made of; float32 has it too
    sign = 1.0 - 2.0 * (torch.arange(dim) % 3 == 0)
    x = torch.stack([sign * top, torch.full((dim,), -top), sign * 1e37, sign * 1e18, sign * 0,
                     sign * 1e-30, sign * 2.0 ** -120])
    x[4, dim // 2] = -3e19
    return R.stored(x, dtype)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("dim", [5, 64, 2048, 5120, 6001, 8191, 12000, 16392])
def test_forward_of_extreme_rows(ms, dim, dtype):
    """Every row is finite, and so is its norm.  eps = 0: also where the squares vanish."""
    x = extreme_rows(dim, dtype)
    w = 1 + 0.3 * torch.randn(dim, generator=torch.Generator().manual_seed(1)).double()
    w = w.float().double()
    for eps in (1e-5, 0.0):
        g = x.to(dtype).cuda()
        out, _ = ms.residual_norm_fwd(g, None, w.float().cuda(), eps=eps)
        o8, scale, _ = ms.residual_norm_fp8(g, None, w.float().cuda(), eps=eps)
        y, _, _ = R.norm_fwd(x, None, w, eps, dtype)
        for k in range(len(x)):
            R.check(f"row {k}", out[k], y[k])
            R.check(f"scale {k}", scale[k], torch.clamp_min(y[k].abs().max(), 2.0 ** -100) / 448)
            R.check(f"row {k} in 8 bits", o8[k], y[k] / scale[k].double().cpu())


@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("dim", [5, 256, 768, 2048, 6001, 8191, 12000, 16392])
def test_backward_of_extreme_rows(ms, dim, types):
    """The gradient at out is large where the row is, so that neither side of the
    comparison is lost below float32's normal values."""
    t = TYPES[types]
    x = extreme_rows(dim, t[1])
    i = R.norm_inputs(22, *t, len(x), dim)
    size = torch.tensor([1e20, 1e20, 1e25, 1e5, 1e5, 1, 1]).double()
    i.update(residual=x, dout=R.stored(i["dout"] * size[:, None], t[0]), dres=None)
    g = {k: v.to(d).cuda() for k, v, d in (("residual", i["residual"], t[1]),
                                           ("dout", i["dout"], t[0]),
                                           ("weight", i["weight"], torch.float32))}
    for eps in (1e-5, 0.0):
        got = ms.residual_norm_bwd(g["residual"], g["weight"], g["dout"], eps=eps)
        d, _, _ = R.norm_bwd(i["residual"], i["weight"], i["dout"], None, eps)
        terms = R.norm_terms(i["residual"], i["weight"], i["dout"], None, eps)
        for n in range(len(x)):
            one = {k: i[k][n:n + 1] for k in ("residual", "dout")}
            R.check(f"dx {n}", got["dx"][n], d[n], terms[n])
            R.check(f"dresidual {n}", got["dresidual"][n], d[n], terms[n])
            alone = ms.residual_norm_bwd(g["residual"][n:n + 1], g["weight"], g["dout"][n:n + 1],
                                         eps=eps)
            _, dw, dw_abs = R.norm_bwd(one["residual"], i["weight"], one["dout"], None, eps)
            R.check(f"dweight {n}", alone["dweight"], dw, dw_abs)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("dim", [40, 512, 1003, 2048, 6001, 16392])
def test_eight_bits_are_the_quotient_by_the_scale(ms, dim, dtype):
    """Bit by bit.  Quarters up to 7: their squares' sum is exact in any order, so that the
    float32 call's out is what the 8-bit call divides; over 7 / 448 many of them lie within
    a unit of float32 of the middle between two values of 8 bits."""
    r = torch.Generator().manual_seed(23)
    x = torch.randint(-28, 29, (300, dim), generator=r).float() / 4
    x[:, 0] = 7
    for w in (None, torch.randn(dim, generator=r).cuda()):
        y, _ = ms.residual_norm_fwd(x.cuda(), None, w)
        out, scale, _ = ms.residual_norm_fp8(x.to(dtype).cuda(), None, w)
        want = y.cpu().abs().amax(-1) / 448
        assert torch.equal(scale.cpu(), want)
        q = (y.cpu() / want[:, None]).to(torch.float8_e4m3fn)
        far = out.cpu().float() != q.float()
        assert not far.any(), (int(far.sum()), far.numel())

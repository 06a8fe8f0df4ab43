"""Gradients of the gated linear recurrence's gates where they are nearly open or nearly
shut, each element against its own size.  Every step is a sequence of its own, so that
dr and di are products, without a sum that would hide a small one behind large ones."""
import pytest
import torch

import recurrent_reference as R

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def ms():
    import scan_selective_fwd_amd as m
    assert torch.cuda.is_available()
    return m


def close(name, got, ref, gate, count, dtype):
    """Within (|gate| + count) 2^-23, and the one rounding to the type.  The exponential of a
    gate v is off by |v| 2^-23 (its exponent's two roundings) and one unit; `count`
    units 2^-23 are for the other factors and products, one by one below."""
    g, r = got.double().cpu(), ref
    half = R.HALF[dtype]
    allowed = ((gate.abs() + count) * 2.0 ** -23 + half * (1 + half)) * r.abs()
    bad = ~((g - r).abs() <= allowed)
    assert not bad.any(), (name, int(bad.sum()), float(((g - r).abs() / r.abs()).max()))


# The gate's complement: its exponential's unit, 1 + e, the reciprocal, their product: 3.
# m = sqrt(1 - a^2): the root 1; 1 - a^2 within 6 (its polynomial 1, the log decay 3.5 or,
# beyond its range, the decay's 4.5 times |y| a^2 / (1 - a^2) < 1), halved by the root: 3.
# The other gate 2.5 and four products: 2.  di: 3 + 4 + 2.5 + 2 < 16.
BY_I = 16
# dr has two decays, of 4.5 each where |A| <= 1, u (as above: 10), y / m^2 (y 4, 1 - a^2 6,
# the reciprocal 1), the complement 3 and four products: 3 + 9 + 10 + 11 + 2 < 48.
BY_R = 48


def run(ms, seed, dtype, size, r, i):
    n = R.rec_inputs(seed, DT[dtype], *size, z=False, h0=False, reset="every")
    g = torch.Generator().manual_seed(seed + 100)
    between = lambda lo, hi: R.stored(lo + (hi - lo) * torch.rand(*size, generator=g), DT[dtype])  # noqa: E731
    n.update(r=between(*r), i=between(*i), A=-(0.05 + 0.15 * torch.rand(size[2], generator=g)).double())
    dev = {k: v.to(DT[dtype]).cuda() for k, v in n.items() if k in ("x", "r", "i", "dout")}
    got = ms.gated_recurrence_bwd(dev["x"], dev["r"], dev["i"], n["A"].float().cuda(), None,
                                  dev["dout"], reset=n["reset"].cuda())
    n["A"] = n["A"].float().double()
    # 1 - s(v) as s(-v): in 64 bits the difference keeps too few digits from v = 20 on
    sr, si = R.sig(n["r"]), R.sig(n["i"])
    m = torch.sqrt(-torch.expm1(2 * n["A"] * sr))
    a2 = torch.exp(2 * n["A"] * sr)
    di = n["dout"] * m * n["x"] * si * R.sig(-n["i"])
    dr = -n["dout"] * si * n["x"] * a2 / m * n["A"] * sr * R.sig(-n["r"])
    return n, got, dr, di


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("size", [(70, 1, 66), (2, 100, 130), (2, 700, 33)])
def test_gates_nearly_open(ms, size, dtype):
    n, got, dr, di = run(ms, 41, dtype, size, (6, 30), (6, 30))
    close("di", got["di"], di, n["i"], BY_I, DT[dtype])
    close("dr", got["dr"], dr, n["r"], BY_R, DT[dtype])


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("size", [(70, 1, 66), (2, 100, 130), (2, 700, 33)])
def test_gates_nearly_shut(ms, size, dtype):
    """Log decays down to 2^-126, the smallest normal number, 1 - a^2 above it."""
    n, got, dr, di = run(ms, 42, dtype, size, (-84, -20), (-20, 2))
    # beside a gate's own exponential there is the other's: |r| at half in m, |i|
    close("di", got["di"], di, n["i"], BY_I + 42, DT[dtype])
    close("dr", got["dr"], dr, n["r"], BY_R + 20, DT[dtype])

"""How far the multi-head scan's results are from 64 bits.

A bfloat16 result is rounded once.  What it is made of carries 32 bits, or two
bfloat16 parts that keep 2^-17 of each operand: at most two such operands and
float32 sums, together below 2^-15 of the result's 2-norm, 4 % of the 8e-4 or
more that one rounding to bfloat16 leaves.  So a result's error is that of
rounding the exact one, times 1.05 at most.
"""
import pytest
import torch

import heads_reference as R
from test_gpu_heads import DT, check_bwd, dev, ms, ref_fwd, run_bwd, run_fwd  # noqa: F401

pytestmark = pytest.mark.gpu

# (batch, L, heads, P, groups, N): every width of the state, one to four heads a block
SIZES = [(2, 257, 4, 64, 2, 128), (1, 300, 2, 128, 1, 256), (3, 130, 6, 48, 3, 80),
         (1, 700, 8, 32, 1, 64), (2, 190, 8, 20, 2, 32), (1, 640, 1, 100, 1, 200),
         (2, 150, 8, 32, 1, 128), (1, 130, 5, 20, 1, 200), (1, 65, 4, 32, 1, 256)]
ROUNDED_ONCE = 1.05


def rounded_once(name, got, ref):
    assert got.dtype == torch.bfloat16
    least = (ref.to(torch.bfloat16).double() - ref).norm()
    e = (got.double().cpu() - ref).norm()
    assert float(e) <= ROUNDED_ONCE * float(least), (name, float(e / least))


@pytest.mark.parametrize("reset", [None, "random"])
@pytest.mark.parametrize("size", SIZES)
def test_bfloat16_out_is_rounded_once(ms, size, reset):  # noqa: F811
    i = R.scan_inputs(61, torch.bfloat16, *size, h0=True, reset=reset)
    for segments in (0, 1):
        out = run_fwd(ms, dev(i, torch.bfloat16), segments=segments)[0]
        rounded_once("out", out, ref_fwd(i)[0])


@pytest.mark.parametrize("reset", [None, "random"])
@pytest.mark.parametrize("size", SIZES)
def test_bfloat16_gradients_are_rounded_once(ms, size, reset):  # noqa: F811
    i = R.scan_inputs(62, torch.bfloat16, *size, h0=True, reset=reset)
    ref = R.scan_bwd(i["u"], i["delta"], i["A"], i["B"], i["C"], i["D"], i["delta_bias"],
                     i["dout"], i["h0"], i["dlast"], i["reset"])[0]
    for segments in (0, 1):
        got = run_bwd(ms, dev(i, torch.bfloat16), segments=segments)
        for k in ("du", "ddelta", "dB", "dC"):
            rounded_once(k, got[k], ref[k])


@pytest.mark.parametrize("size", SIZES)
def test_float32_of_the_same_sizes(ms, size):  # noqa: F811
    i = R.scan_inputs(64, torch.float32, *size, h0=True, reset="random")
    g = dev(i, torch.float32)
    out, last = run_fwd(ms, g)
    want, want_last = ref_fwd(i)
    R.check("out", out, want)
    R.check("last", last, want_last)
    check_bwd(run_bwd(ms, g), i)


def forgetting(seed, dtype, kind, softplus):
    """Steps that forget all that was before them among steps that keep nearly all:
    the log decays' sums are far below zero where weights are near 1."""
    b, L, H = 2, 200, 4
    i = R.scan_inputs(seed, dtype, b, L, H, 64, 1, 128)
    i["A"][:] = -16.0
    i["delta_bias"][:] = 0.0
    if kind == "alternating":
        dt = torch.full((b, L, H), 0.01, dtype=torch.float64)
        dt[:, ::2] = 8.0
    elif kind == "one in eight":
        dt = torch.full((b, L, H), 0.002, dtype=torch.float64)
        dt[:, 3::8] = 20.0
    else:
        dt = torch.nn.functional.softplus(R.Inputs(seed + 1, dtype).seq(b, L, H, scale=3.0))
    i["delta"] = (dt.expm1().log() if softplus else dt).to(dtype).double()
    return i


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("disc", ["zoh", "euler"])
@pytest.mark.parametrize("softplus", [True, False])
@pytest.mark.parametrize("kind", ["alternating", "one in eight", "spread"])
def test_out_under_forgetting_steps(ms, kind, softplus, disc, dtype):  # noqa: F811
    """float32: units of 2^-24 for the step (4), its exponent (2), the weight and its
    product (2), and the square root of the 160 terms that the two products sum (13)
    for the rounding of their sums, rounded up to 32 for all of them."""
    i = forgetting(63, DT[dtype], kind, softplus)
    out, last = run_fwd(ms, dev(i, DT[dtype]), softplus=softplus, disc=disc)
    want, want_last = ref_fwd(i, softplus=softplus, disc=disc)
    if dtype == "bf16":
        rounded_once("out", out, want)
    for name, x, y in (("out", out, want), ("last", last, want_last)):
        if x.dtype == torch.float32:
            e = float((x.double().cpu() - y).norm() / y.norm())
            assert e <= 32 * 2.0 ** -24, (name, e)

"""Infinities and NaN in the multi-head scan: how far they reach, against the
64-bit recurrence, in which 0 times one is NaN."""
import pytest
import torch

import heads_reference as R
from test_gpu_heads import DT, dev, ms, ref_fwd, run_bwd, run_fwd  # noqa: F401

pytestmark = pytest.mark.gpu

NAN, INF = float("nan"), float("inf")


def strong(dtype, L, reset=None):
    """Decays that underflow float32 within 20 steps."""
    i = R.scan_inputs(71, dtype, 2, L, 3, 40, 1, 48, h0=True, reset=reset)
    i["A"][:] = -16.0
    i["delta_bias"][:] = 0.5
    return i


def spoiled(i, what, at, value):
    i = dict(i, **{what: i[what].clone()})
    if what in ("h0", "dlast"):
        i[what][0, 1, 7, 5] = value
    elif what == "delta":
        i[what][0, at, 1] = value
    else:
        i[what][0, at].flatten()[9] = value
    return i


def ref_bwd(i):
    return R.scan_bwd(i["u"], i["delta"], i["A"], i["B"], i["C"], i["D"], i["delta_bias"],
                      i["dout"], i["h0"], i["dlast"], i["reset"])[0]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("value", [NAN, INF])
@pytest.mark.parametrize("what", ["u", "B", "C", "h0"])
def test_a_decay_that_underflows_keeps_them(ms, what, value, dtype):  # noqa: F811
    """One segment, several joined by the output pass, and by a pass of its own."""
    L = 700
    for reset in (None, "edges"):
        i = spoiled(strong(DT[dtype], L, reset), what, 10, value)
        want, want_last = (~torch.isfinite(x) for x in ref_fwd(i))
        if reset is not None:
            # a flag makes the state zero, where the reference multiplies it by zero
            number = i["reset"].long().cumsum(1)
            of = 0 if what == "h0" else number[0, 10]
            want &= (number == of)[:, :, None, None]
            want_last &= bool(number[0, -1] == of)
        elif what != "C":
            assert want[0, 10:].any((-1, -2)).all() and want_last.any()
        for segments in (0, 1, 5, 100):
            out, last = run_fwd(ms, dev(i, DT[dtype]), segments=segments)
            assert torch.equal(~torch.isfinite(out.cpu()), want), (segments, reset)
            assert torch.equal(~torch.isfinite(last.cpu()), want_last), (segments, reset)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("what,at", [("u", 10), ("B", 10), ("h0", 0), ("C", 690), ("dout", 690),
                                     ("dlast", 0)])
def test_a_decay_that_underflows_keeps_them_in_gradients(ms, what, at, dtype):  # noqa: F811
    """A gradient that the recurrence makes infinite or NaN is not finite here."""
    i = spoiled(strong(DT[dtype], 700), what, at, NAN)
    want = ref_bwd(i)
    for segments in (0, 1, 5):
        got = run_bwd(ms, dev(i, DT[dtype]), segments=segments)
        for k in want:
            lost = ~torch.isfinite(want[k]) & torch.isfinite(got[k].cpu())
            assert not lost.any(), (k, segments, int(lost.sum()), int((~torch.isfinite(want[k])).sum()))
            if want[k].dim() > 1:       # the other batch row's are finite
                assert torch.isfinite(got[k][1]).all(), (k, segments)


# flags inside chunks, at their borders and next to each other
STARTS = (3, 21, 40, 41, 64, 90, 128, 150)


def packed(dtype, L, H, P, G, N):
    i = R.scan_inputs(72, dtype, 2, L, H, P, G, N, h0=True, reset="random")
    i["reset"][:] = 0
    i["reset"][:, [s for s in STARTS if s < L]] = 1
    return i


@pytest.mark.parametrize("value", [NAN, INF, 3.0e38])
@pytest.mark.parametrize("what,at", [("u", 30), ("u", 40), ("dout", 50), ("B", 25), ("C", 63),
                                     ("delta", 45), ("u", 100), ("dout", 2), ("h0", 0),
                                     ("dlast", 0)])
def test_gradients_of_other_sequences_do_not_see_them(ms, what, at, value):  # noqa: F811
    """A non-finite value, or one whose products overflow, in one sequence of a packed
    row: the gradients at the other sequences' tokens are those of the clean inputs."""
    for dtype, size in ((torch.float32, (4, 40, 2, 24)), (torch.bfloat16, (4, 64, 1, 128)),
                        (torch.bfloat16, (3, 100, 1, 160)), (torch.bfloat16, (4, 32, 2, 48)),
                        (torch.float32, (2, 64, 1, 100))):
        L = 170
        i = packed(dtype, L, *size)
        want = ref_bwd(i)
        bad = spoiled(i, what, at, value)
        number = i["reset"].long().cumsum(1)[0]
        of = 0 if what == "h0" else int(number[-1]) if what == "dlast" else int(number[at])
        others = torch.nonzero(number != of).flatten()
        for segments in (0, 1):
            got = run_bwd(ms, dev(bad, dtype), segments=segments)
            for k in ("du", "ddelta", "dB", "dC"):
                R.check(k, got[k][0, others.cuda()], want[k][0, others])
                R.check(k, got[k][1], want[k][1])
            R.check("dh0", got["dh0"][1], want["dh0"][1])
            if of > 0:
                R.check("dh0", got["dh0"][0], want["dh0"][0])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_packed_gradients_with_them_are_those_of_the_sequences_alone(ms, dtype):  # noqa: F811
    """Also the spoiled sequence's: not finite where the recurrence over it is not."""
    L = 170
    i = packed(DT[dtype], L, 4, 64, 1, 128)
    for what, at in (("u", 45), ("dout", 50), ("B", 25), ("C", 63)):
        bad = spoiled(i, what, at, NAN)
        got = run_bwd(ms, dev(bad, DT[dtype]))
        begin = max(s for s in (0,) + STARTS if s <= at)
        end = min(s for s in STARTS + (L,) if s > at)
        part = dict(bad, h0=torch.zeros_like(bad["h0"]), dlast=torch.zeros_like(bad["dlast"]),
                    reset=None, **{n: bad[n][:, begin:end] for n in ("u", "delta", "B", "C", "dout")})
        want = ref_bwd(part)
        odd = {k: ~torch.isfinite(want[k][0]) for k in ("du", "ddelta", "dB", "dC")}
        assert any(o.any() for o in odd.values())
        for k, o in odd.items():
            assert not torch.isfinite(got[k][0, begin:end].cpu()[o]).any(), (what, k)

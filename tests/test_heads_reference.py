"""The 64-bit reference of the multi-head operators, on the CPU: its written-out
backward against central differences, the packed form against its pieces, the
scan against its convolution form and against the single-channel oracle."""
import numpy as np
import pytest
import torch

import heads_reference as R
import oracle

F64 = torch.float64
SCAN = ("u", "delta", "A", "B", "C", "D", "delta_bias", "h0")


def _loss(v, dout, dlast, reset, softplus, disc):
    out, last, _ = R.scan_fwd(v["u"], v["delta"], v["A"], v["B"], v["C"], v["D"], v["delta_bias"],
                              v["h0"], reset, softplus, disc)
    return float((out * dout).sum() + (last * dlast).sum())


@pytest.mark.parametrize("disc", ["zoh", "euler"])
@pytest.mark.parametrize("softplus", [True, False])
@pytest.mark.parametrize("reset", [None, "random", "edges"])
def test_scan_backward_against_differences(disc, softplus, reset):
    i = R.scan_inputs(1, torch.float32, 2, 40, 4, 3, 2, 5, h0=True, reset=reset)
    if not softplus:
        i["delta"] = i["delta"].abs() * 0.05
        i["delta_bias"] = i["delta_bias"].abs() * 0.01
    g, _ = R.scan_bwd(i["u"], i["delta"], i["A"], i["B"], i["C"], i["D"], i["delta_bias"],
                      i["dout"], i["h0"], i["dlast"], i["reset"], softplus, disc)
    r = np.random.default_rng(3)
    for name in SCAN:
        for _ in range(3):     # along random directions
            d = torch.from_numpy(r.standard_normal(i[name].shape))
            eps = 1e-6
            hi, lo = dict(i), dict(i)
            hi[name], lo[name] = i[name] + eps * d, i[name] - eps * d
            fd = (_loss(hi, i["dout"], i["dlast"], i["reset"], softplus, disc)
                  - _loss(lo, i["dout"], i["dlast"], i["reset"], softplus, disc)) / (2 * eps)
            an = float((g["d" + name] * d).sum())
            # rounding of two losses of some hundred / 2e-6, and the third derivative
            assert abs(fd - an) <= 1e-6 * max(1.0, abs(an)) + 1e-6, (name, fd, an)


def test_scan_matches_the_single_channel_oracle():
    """Every channel of a head is a channel of the S6 scan with A equal over its states."""
    b, L, H, P, N = 2, 50, 2, 3, 4
    i = R.scan_inputs(2, torch.float32, b, L, H, P, 1, N, h0=True)
    out, last, _ = R.scan_fwd(i["u"], i["delta"], i["A"], i["B"], i["C"], i["D"], i["delta_bias"],
                              i["h0"])
    chan = lambda t: np.ascontiguousarray(t.repeat_interleave(P, -1).numpy())  # noqa: E731
    seq = lambda t: np.ascontiguousarray(t.numpy())  # noqa: E731
    ref, ref_last = oracle.scan_fwd(
        seq(i["u"].flatten(2).transpose(1, 2)),
        seq(i["delta"].repeat_interleave(P, -1).transpose(1, 2)),
        seq(i["A"].repeat_interleave(P).unsqueeze(1).expand(H * P, N)),
        seq(i["B"][:, :, 0].transpose(1, 2)), seq(i["C"][:, :, 0].transpose(1, 2)), chan(i["D"]),
        None, chan(i["delta_bias"]), seq(i["h0"].flatten(1, 2)))
    assert np.abs(out.flatten(2).transpose(1, 2).numpy() - ref).max() <= 1e-12 * np.abs(ref).max()
    assert np.abs(last.flatten(1, 2).numpy() - ref_last).max() <= 1e-12 * np.abs(ref_last).max()


def test_packed_scan_equals_its_pieces():
    i = R.scan_inputs(4, torch.float32, 1, 60, 2, 3, 1, 4, reset="random")
    i["reset"][0, 17] = i["reset"][0, 44] = 1
    at = [0] + [t for t in range(1, 60) if i["reset"][0, t]] + [60]
    out, last, _ = R.scan_fwd(i["u"], i["delta"], i["A"], i["B"], i["C"], i["D"], i["delta_bias"],
                              reset=i["reset"])
    for a, b in zip(at, at[1:]):
        o, h, _ = R.scan_fwd(*(i[n][:, a:b] for n in ("u", "delta")), i["A"],
                             *(i[n][:, a:b] for n in ("B", "C")), i["D"], i["delta_bias"])
        # the vectorised exponentials may differ by an ulp with the memory layout
        assert torch.allclose(out[:, a:b], o, rtol=1e-12, atol=1e-14)
    assert torch.allclose(last, h, rtol=1e-12, atol=1e-14)


def test_conv_reference_against_numpy_convolve():
    r = R.Inputs(5, torch.float32)
    x, w, win = r.seq(1, 30, 2), r.f32(2, 4), r.seq(1, 3, 2)
    out, after = R.conv_fwd(x, w, None, win)
    for d in range(2):
        full = np.concatenate([win[0, :, d].numpy(), x[0, :, d].numpy()])
        pre = np.convolve(full, w[d].numpy()[::-1])[3:33]
        np.testing.assert_allclose(out[0, :, d].numpy(), pre / (1 + np.exp(-pre)), rtol=1e-12,
                                   atol=1e-14)
    assert torch.equal(after, x[:, -3:])


def test_norm_reference_has_unit_groups():
    r = R.Inputs(6, torch.float32)
    y = R.norm_fwd(r.seq(5, 24), r.seq(5, 24), None, 3, 0.0, True)
    ms = y.unflatten(-1, (3, 8)).square().mean(-1)
    assert torch.allclose(ms, torch.ones_like(ms), rtol=1e-12)

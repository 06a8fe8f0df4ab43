"""The norm's backward at rows of about the most channels that it takes."""
import pytest
import torch

import recurrent_reference as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ms():
    import scan_selective_fwd_amd as m
    assert torch.cuda.is_available()
    return m


def parts(*tensors):
    for at in range(0, tensors[0].numel(), 1 << 26):
        yield [t.reshape(-1)[at:at + (1 << 26)].double() for t in tensors]


@pytest.mark.parametrize("dim", [(1 << 28) - 64])
def test_dweight_of_the_widest_row(ms, dim):
    g = torch.Generator("cuda").manual_seed(2)
    res, dout = (torch.randn(1, dim, device="cuda", generator=g) for _ in range(2))
    w = 1 + 0.1 * torch.randn(dim, device="cuda", generator=g)
    got = ms.residual_norm_bwd(res, w, dout, eps=0.0)
    root = sum(float(v.square().sum()) for (v,) in parts(res))
    root = (root / dim) ** 0.5
    for dw, v, dy in parts(got["dweight"], res, dout):
        want = dy * v / root
        # dw is the one row's product, its root within some 2^-21: groups of four squares,
        # the joins over threads
        assert ((dw - want).abs() <= R.REL * want.abs()).all()

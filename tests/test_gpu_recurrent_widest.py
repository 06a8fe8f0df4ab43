"""The backward passes at the most channels that the recurrent block's operators take:
their sums over rows and tiles then need more than one launch (32 or 64 channels a block
of 1024 threads, and a launch has less than 2^32 threads)."""
import pytest
import torch

import recurrent_reference as R

pytestmark = pytest.mark.gpu
DIM = 1 << 28


@pytest.fixture(scope="module")
def ms():
    import scan_selective_fwd_amd as m
    assert torch.cuda.is_available()
    return m


def parts(*tensors):
    """In parts, the ends of the launches among them."""
    for at in range(0, tensors[0].numel(), 1 << 26):
        yield [t.reshape(-1)[at:at + (1 << 26)].double() for t in tensors]


def test_dA_of_the_widest_recurrence(ms):
    """One step: dA is dr / (A (1 - s(r))), channel by channel."""
    g = torch.Generator("cuda").manual_seed(1)
    x, r, i, dout = (torch.randn(1, 1, DIM, device="cuda", generator=g) for _ in range(4))
    A = -(0.05 + torch.rand(DIM, device="cuda", generator=g))
    got = ms.gated_recurrence_bwd(x, r, i, A, None, dout)
    for dA, dr, a, v in parts(got["dA"], got["dr"], A, r):
        want = dr / (a * torch.sigmoid(-v))
        # 1 - s(r) is within (|r| + 3) 2^-23, |r| < 7; the sum and the division by A 2^-23
        assert ((dA - want).abs() <= 12 * 2.0 ** -23 * want.abs()).all()


@pytest.mark.parametrize("dim", [(1 << 28) - 64, DIM])
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

"""The backward kernels have no derivative of their own: asking for a second one is
refused, where leaving it out would give a wrong gradient without a word."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def losses():
    import scan_selective_fwd_amd as ms
    r = lambda *s: torch.randn(*s, device="cuda")  # noqa: E731
    u = r(2, 24, 100).requires_grad_(True)
    yield u, lambda: ms.selective_scan(u, r(2, 24, 100), -torch.rand(24, 16, device="cuda"),
                                       r(2, 16, 100), r(2, 16, 100))
    h = r(2, 100, 4, 16).requires_grad_(True)
    yield h, lambda: ms.heads_scan(h, r(2, 100, 4), -torch.rand(4, device="cuda"),
                                   r(2, 100, 1, 16), r(2, 100, 1, 16))
    x = r(2, 100, 24).requires_grad_(True)
    yield x, lambda: ms.conv1d_tokens(x, r(24, 4))
    y = r(7, 48).requires_grad_(True)
    yield y, lambda: ms.gated_norm(y, r(7, 48))


@pytest.mark.parametrize("at", range(4))
def test_a_second_derivative_is_refused(at):
    leaf, call = list(losses())[at]
    (g,) = torch.autograd.grad(call().square().sum(), leaf, create_graph=True)
    assert torch.isfinite(g).all()
    with pytest.raises(RuntimeError):       # a penalty on the gradient beside another term
        torch.autograd.grad(g.square().sum() + leaf.sum(), leaf)

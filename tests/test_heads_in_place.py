"""What may not be written in place is refused (no GPU: before any launch)."""
from scan_selective_fwd_amd import _lib

P = 1 << 20            # a pointer that is never followed
INVALID = 8


def test_a_convolution_over_its_input_is_refused():
    """Its tokens read inputs that others' outputs would have replaced."""
    f = _lib.load().mamba_conv1d_tokens_fwd
    for W in (2, 4):
        assert f(P, 6400, 64, P, None, None, None, W, 1, 2, 64, 100, P, None, None) == INVALID


def test_a_window_that_is_its_successor_is_refused():
    f = _lib.load().mamba_conv1d_tokens_fwd
    assert f(P, 6400, 64, P, None, P, None, 4, 1, 2, 64, 100, 2 * P, P, None) == INVALID

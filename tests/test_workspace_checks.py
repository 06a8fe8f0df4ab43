"""The binding's check of a caller's workspace (no GPU: it comes before any launch)."""
import pytest
import torch

from scan_selective_fwd_amd import heads

GPU = torch.device("cuda", 0)


@pytest.mark.parametrize("workspace", [torch.empty(4096, dtype=torch.uint8),
                                       torch.empty(1024)])
def test_another_device_is_refused(workspace):
    """A host address would reach the kernels."""
    with pytest.raises(ValueError, match="is on cpu"):
        heads._workspace(4096, (1,), "a call", workspace, GPU)


def test_what_is_not_one_piece_is_refused():
    """One byte expanded counts as many elements as wanted."""
    cpu = torch.device("cpu")
    for w in (torch.empty(1, dtype=torch.uint8).expand(4096),
              torch.empty(8192, dtype=torch.uint8)[::2]):
        with pytest.raises(ValueError, match="contiguous"):
            heads._workspace(4096, (1,), "a call", w, cpu)


def test_what_is_not_a_tensor_is_refused():
    with pytest.raises(TypeError):
        heads._workspace(4096, (1,), "a call", 4096, GPU)


def test_a_large_enough_one_is_taken_and_a_smaller_one_left():
    cpu = torch.device("cpu")
    w = torch.empty(4096, dtype=torch.uint8)
    assert heads._workspace(4096, (1,), "a call", w, cpu) is w
    assert heads._workspace(16000, (1,), "a call", torch.empty(4000), cpu).numel() == 4000
    got = heads._workspace(4097, (1,), "a call", w, cpu)
    assert got is not w and got.numel() == 4097

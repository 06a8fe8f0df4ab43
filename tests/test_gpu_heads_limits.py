"""A norm of more rows than one launch holds (2^24 - 1 blocks of 256 threads)."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("off", [0, 1])
def test_norm_of_more_rows_than_a_launch_holds(off):
    """Four groups a block; rows on 16 bytes and off them."""
    import scan_selective_fwd_amd as ms
    rows, period = 4 * ((1 << 24) - 1) + 9, 1 << 12
    few = torch.randn(period, 8 + off, device="cuda").bfloat16()
    want = ms.gated_norm_fwd(few[:, :8], few[:, off:])
    wide = few.repeat(-(-rows // period), 1)[:rows]
    got = ms.gated_norm_fwd(wide[:, :8], wide[:, off:])
    torch.cuda.synchronize()
    for at in (0, rows // period // 2 * period, (rows // period - 1) * period):
        assert torch.equal(got[at:at + period], want)
    tail = rows % period
    assert torch.equal(got[rows - tail:], want[:tail])

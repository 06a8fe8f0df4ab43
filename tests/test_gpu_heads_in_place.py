"""A prompt whose last state takes h0's place."""
import pytest
import torch

import heads_reference as R
from test_gpu_heads import DT, dev, ms, run_fwd  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("size", [(2, 700, 4, 64, 2, 64), (1, 1500, 3, 100, 1, 200), (3, 65, 5, 20, 1, 7)])
def test_the_state_steps_in_place(ms, size, dtype):  # noqa: F811
    """In one segment, in several that the output pass joins, and in more."""
    i = R.scan_inputs(81, DT[dtype], *size, h0=True, reset="random")
    g = dev(i, DT[dtype])
    for segments in (0, 1, 3, 100):
        out, last = run_fwd(ms, g, segments=segments)
        state = g["h0"].clone()
        for _ in range(3):
            state.copy_(g["h0"])
            got, same = run_fwd(ms, dict(g, h0=state), segments=segments, last_state=state)
            assert same is state
            assert torch.equal(got, out) and torch.equal(state, last), segments


def test_a_last_state_over_a_part_of_h0_is_refused(ms):  # noqa: F811
    i = R.scan_inputs(82, torch.float32, 1, 90, 4, 16, 1, 16, h0=True)
    g = dev(i, torch.float32)
    two = torch.zeros(2 * 4 * 16 * 16, device="cuda")
    part = lambda at: two[at:at + 4 * 16 * 16].view(1, 4, 16, 16)  # noqa: E731
    for a, b in ((0, 256), (512, 0), (4, 0)):
        with pytest.raises(ms.MambaScanError):
            run_fwd(ms, dict(g, h0=part(a)), last_state=part(b))
    run_fwd(ms, dict(g, h0=part(0)), last_state=part(1024))

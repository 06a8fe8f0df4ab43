"""The example mixer: all multi-head operators run together."""
import os
import sys

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mixer_module():
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import heads_mixer
    return heads_mixer


def test_example_runs(mixer_module):
    far, losses = mixer_module.main()
    # bfloat16 activations: every stage rounds at 2^-9, and the pieces round at other places
    assert far < 2e-2
    assert losses[-1] < losses[0]


def test_pool_of_users(mixer_module):
    """Sequences of different lengths decode together from one pool, by slot."""
    torch.manual_seed(1)
    m = mixer_module.HeadsMixer(128, heads=4, headdim=32, dstate=64, groups=2,
                                dtype=torch.float32)
    lengths, pool = (5, 77, 130), 6
    x = torch.randn(3, 140, 128, device="cuda")
    window = torch.zeros(pool, 3, m.conv_cols, device="cuda")
    state = torch.zeros(pool, 4, 32, 64, device="cuda")
    slots = torch.tensor([4, 1, 3], dtype=torch.int32, device="cuda")
    for i, n in enumerate(lengths):
        _, (w, s) = m.prefill(x[i:i + 1, :n])
        window[slots[i].item()], state[slots[i].item()] = w[0], s[0]
    for k in range(8):
        xt = torch.stack([x[i, n + k] for i, n in enumerate(lengths)])
        out = m.step(xt, (window, state), slots)
        for i, n in enumerate(lengths):
            want = m(x[i:i + 1, :n + k + 1])[0, -1]
            # float32 through four stages and two library products of 128 and 512 terms
            assert float((out[i] - want).norm() / want.norm()) < 1e-4


def test_packed_rows_equal_their_sequences(mixer_module):
    torch.manual_seed(2)
    m = mixer_module.HeadsMixer(96, heads=4, headdim=32, dstate=32, dtype=torch.float32)
    x = torch.randn(1, 150, 96, device="cuda")
    reset = torch.zeros(1, 150, dtype=torch.bool, device="cuda")
    cuts = [0, 40, 41, 99, 150]
    for c in cuts[1:-1]:
        reset[0, c] = True
    out = m(x, reset)
    for a, b in zip(cuts, cuts[1:]):
        want = m(x[:, a:b])
        assert float((out[:, a:b] - want).norm() / want.norm()) < 1e-4
